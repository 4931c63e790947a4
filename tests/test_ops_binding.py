"""What the binding of the operators around a verification step refuses
before the library is called (CPU only)."""
import types

import pytest
import torch


@pytest.fixture(scope="module")
def sv():
    import rejection_sampling_verify_03_amd as m
    return m


U8 = torch.uint8


@pytest.mark.parametrize("codes,scales", [
    (torch.float8_e5m2, U8), (torch.float8_e4m3fnuz, U8), (torch.float8_e5m2fnuz, U8), (torch.int8, U8),
    (torch.bool, U8), (torch.bfloat16, U8), (torch.float8_e8m0fnu, U8), (U8, torch.int8), (U8, torch.bool),
    (U8, torch.float8_e4m3fn), (U8, torch.float32)])
def test_caches_of_other_types(sv, codes, scales):
    """Codes are e4m3 (or bytes) and scales exponent bytes: another 8-bit type
    would be read as what it is not."""
    k = torch.zeros(2, 16, 1, 64, dtype=U8).to(codes) if codes != torch.float8_e8m0fnu else \
        torch.zeros(2, 16, 1, 64, dtype=U8).view(codes)
    sc = torch.zeros(2, 1, 1, dtype=U8).to(scales)
    with pytest.raises(TypeError):
        sv.KVCache(k, k.clone(), sc, sc.clone())


# ctypes takes the lower 32 bits of what it is given
PAST = (2 ** 32 + 8, 2 ** 31, -2 ** 32 + 8)


def cache_on_cpu(sv):
    return types.SimpleNamespace(device=torch.device("cpu"), args=sv.SpecKVCache(), heads=2, head_dim=64, block_size=16)


@pytest.mark.parametrize("shape", [(1, 1, PAST[0]), (1, PAST[0], 8), (PAST[0], 1, 8), (1, 1, PAST[1])])
def test_logits_past_32_bits(sv, shape):
    x = torch.empty(shape, dtype=torch.bfloat16, device="meta")
    tokens = torch.empty(shape[:2], dtype=torch.int32, device="meta")
    out = sv.token_logprobs_outputs(*shape[:2], 3, "meta")
    for call in (lambda: sv.token_logprobs(x, tokens), lambda: sv.token_logprobs_args(x, tokens, None, out, None)):
        with pytest.raises(ValueError, match="32 bits"):
            call()
    assert sv.spec_logprobs_workspace_bytes(*shape, 3) == 0


@pytest.mark.parametrize("n", PAST[:2])
def test_entries_past_32_bits(sv, n):
    cache = cache_on_cpu(sv)
    slots = torch.empty(n, dtype=torch.int64, device="meta")
    key = torch.empty(n, 2, 64, dtype=torch.bfloat16, device="meta")
    cache.device = slots.device
    with pytest.raises(ValueError, match="32 bits"):
        sv.kv_write_args(cache, key, key, slots)
    with pytest.raises(ValueError, match="32 bits"):
        sv.kv_read(cache, slots)
    codes = torch.empty(1, 16, 1, 64, dtype=U8).expand(n, 16, 1, 64)
    with pytest.raises(ValueError, match="32 bits"):
        sv.KVCache(codes, codes, torch.empty(1, 1, 1, dtype=U8).expand(n, 1, 1),
                   torch.empty(1, 1, 1, dtype=U8).expand(n, 1, 1))


@pytest.mark.parametrize("n", PAST)
@pytest.mark.parametrize("name", ["max_q", "max_ctx", "window"])
def test_attention_bounds_past_32_bits(sv, name, n):
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    i32 = dict(dtype=torch.int32)
    kw = dict(max_q=2, max_ctx=32, scale=0.125, out=torch.zeros_like(q))
    args = (q, cache_on_cpu(sv), torch.zeros(2, 3, **i32), torch.zeros(3, **i32), torch.zeros(2, **i32))
    assert sv.kv_attention_args(*args, **kw).B == 2
    with pytest.raises(ValueError, match="32 bits"):
        sv.kv_attention_args(*args, **{**kw, name: n})


def test_attention_tables_past_32_bits(sv):
    q = torch.empty(2 ** 32 + 3, 4, 64, dtype=torch.bfloat16, device="meta")
    i32 = dict(dtype=torch.int32, device="meta")
    cache = cache_on_cpu(sv)
    cache.device = q.device
    kw = dict(max_q=2, max_ctx=32, scale=0.125)
    table, start, ctx = torch.empty(2, 3, **i32), torch.empty(3, **i32), torch.empty(2, **i32)
    with pytest.raises(ValueError, match="32 bits"):
        sv.kv_attention_args(q, cache, table, start, ctx, out=q, **kw)
    with pytest.raises(ValueError, match="32 bits"):
        sv.kv_attention_args(q[:3], cache, torch.empty(2, 2 ** 32 + 3, **i32), start, ctx, out=q[:3], **kw)


def test_writes_to_keys_and_values_in_one_place(sv):
    """Two owners of the same bytes: refused (one address for both; the
    launch is refused before anything is enqueued)."""
    P = 1 << 20
    for same in ("codes", "scales"):
        a = sv.SpecKVWriteArgs()
        c = a.cache
        c.num_blocks, c.block_size, c.scale_tokens, c.heads, c.head_dim = 10, 16, 16, 2, 64
        c.k_codes, c.v_codes, c.k_scales, c.v_scales = P, 2 * P, 3 * P, 4 * P
        c.block_stride, c.token_stride, c.head_stride = 2048, 128, 64
        c.scale_block_stride, c.scale_head_stride = 2, 1
        setattr(c, "v_" + same, getattr(c, "k_" + same))
        a.N, a.dtype, a.key, a.value, a.slots = 4, sv.SPEC_BF16, P, P, P
        assert sv.spec_kv_write_launch(a, None) == sv.SPEC_EINVAL
