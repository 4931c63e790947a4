"""The C ABI of the operators around a verification step, on the CPU: struct
layouts, workspace sizes, and every refusal before anything is enqueued (the
pointers here are never dereferenced); and the 64-bit oracle's 8-bit
conversion against torch's."""
import ctypes
import math
import subprocess
import os

import numpy as np
import pytest
import torch

import ops_oracle as oo

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20  # a well-aligned address that nothing reads


@pytest.fixture(scope="module")
def sv():
    import rejection_sampling_verify_03_amd as m
    return m


def test_struct_layouts_match_the_header(sv, tmp_path):
    pairs = (("spec_logprobs_args", sv.SpecLogprobsArgs), ("spec_kv_cache", sv.SpecKVCache),
             ("spec_kv_write_args", sv.SpecKVWriteArgs), ("spec_kv_read_args", sv.SpecKVReadArgs),
             ("spec_attn_args", sv.SpecAttnArgs))
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "spec_verify.h"', "int main(void) {"]
    want = []
    for cname, py in pairs:
        lines.append('printf("%%zu\\n", sizeof(%s));' % cname)
        want.append(ctypes.sizeof(py))
        for f, _ in py._fields_:
            lines.append('printf("%%zu\\n", offsetof(%s, %s));' % (cname, f))
            want.append(getattr(py, f).offset)
    lines.append('printf("%d\\n", SPEC_MAX_TOP); return 0; }')
    want.append(sv.SPEC_MAX_TOP)
    src, exe = tmp_path / "l.c", tmp_path / "l"
    src.write_text("\n".join(lines))
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == want


# ------------------------------------------------------------------ logprobs
def lp_args(sv, **kw):
    a = sv.SpecLogprobsArgs()
    a.B, a.R, a.V, a.dtype, a.top = 2, 3, 1000, sv.SPEC_BF16, 4
    a.logits, a.req_stride, a.row_stride, a.tokens, a.temperature = P, 3000, 1000, P, P
    a.logprobs, a.entropy, a.top_ids, a.top_logprobs, a.workspace = P, P, P, P, P
    a.workspace_bytes = 1 << 30
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), "SPEC_EINVAL"), (dict(R=-1), "SPEC_EINVAL"), (dict(V=0), "SPEC_EINVAL"),
    (dict(V=2 ** 31 - 1), "SPEC_EINVAL"), (dict(top=-1), "SPEC_EINVAL"), (dict(top=33), "SPEC_EINVAL"),
    (dict(dtype=2), "SPEC_EDTYPE"), (dict(logits=None), "SPEC_EINVAL"), (dict(tokens=None), "SPEC_EINVAL"),
    (dict(logprobs=None), "SPEC_EINVAL"), (dict(top_ids=None), "SPEC_EINVAL"), (dict(top_logprobs=None), "SPEC_EINVAL"),
    (dict(row_stride=999), "SPEC_EINVAL"), (dict(req_stride=2999), "SPEC_EINVAL"), (dict(req_stride=-3000), "SPEC_EINVAL"),
    (dict(workspace=None), "SPEC_EINVAL"), (dict(workspace=P + 8), "SPEC_EALIGN"), (dict(workspace_bytes=64), "SPEC_EWORKSPACE"),
    (dict(B=2 ** 16, R=2 ** 15, req_stride=0), "SPEC_EINVAL"), (dict(B=2 ** 16, R=300, req_stride=0), "SPEC_EINVAL")])
def test_logprobs_refusals(sv, kw, status):
    assert sv.spec_logprobs_launch(lp_args(sv, **kw), None) == getattr(sv, status)


def test_logprobs_of_nothing(sv):
    assert sv.spec_logprobs_launch(lp_args(sv, B=0, logits=None), None) == sv.SPEC_OK
    assert sv.spec_logprobs_launch(lp_args(sv, R=0, tokens=None), None) == sv.SPEC_OK
    assert sv.lib.spec_logprobs_launch(None, None) == sv.SPEC_EINVAL
    assert sv.spec_logprobs_workspace_bytes(2, 3, 1000, 0) > 0
    assert sv.spec_logprobs_workspace_bytes(2, 3, 1000, 1) > sv.spec_logprobs_workspace_bytes(2, 3, 1000, 0)
    for bad in ((-1, 1, 10, 0), (1, 1, 0, 0), (1, 1, 10, 33), (1, -1, 10, 0)):
        assert sv.spec_logprobs_workspace_bytes(*bad) == 0


# --------------------------------------------------------------------- cache
def cache_args(sv, **kw):
    c = sv.SpecKVCache()
    c.num_blocks, c.block_size, c.scale_tokens, c.heads, c.head_dim = 10, 16, 16, 2, 64
    c.k_codes = c.v_codes = c.k_scales = c.v_scales = P
    c.block_stride, c.token_stride, c.head_stride = 2048, 128, 64
    c.scale_block_stride, c.scale_head_stride = 2, 1
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_CACHES = [
    (dict(num_blocks=0), "SPEC_EINVAL"), (dict(block_size=8), "SPEC_EINVAL"), (dict(block_size=48), "SPEC_EINVAL"),
    (dict(block_size=2048), "SPEC_EINVAL"), (dict(scale_tokens=0), "SPEC_EINVAL"), (dict(scale_tokens=3), "SPEC_EINVAL"),
    (dict(scale_tokens=32), "SPEC_EINVAL"), (dict(heads=0), "SPEC_EINVAL"), (dict(heads=1025), "SPEC_EINVAL"),
    (dict(head_dim=0), "SPEC_EINVAL"), (dict(head_dim=72), "SPEC_EINVAL"), (dict(head_dim=272), "SPEC_EINVAL"),
    (dict(k_codes=None), "SPEC_EINVAL"), (dict(v_scales=None), "SPEC_EINVAL"), (dict(k_codes=P + 8), "SPEC_EALIGN"),
    (dict(token_stride=136), "SPEC_EALIGN"), (dict(block_stride=2056), "SPEC_EALIGN"),
    (dict(token_stride=64), "SPEC_EINVAL"), (dict(head_stride=48), "SPEC_EINVAL"), (dict(block_stride=1024), "SPEC_EINVAL"),
    (dict(token_stride=-128), "SPEC_EINVAL"), (dict(head_stride=2 ** 50), "SPEC_EINVAL"),
    (dict(scale_head_stride=0), "SPEC_EINVAL"), (dict(scale_block_stride=1), "SPEC_EINVAL")]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_cache_refusals(sv, kw, status):
    for call, struct in ((sv.spec_kv_write_launch, sv.SpecKVWriteArgs), (sv.spec_kv_read_launch, sv.SpecKVReadArgs)):
        a = struct()
        a.cache, a.N, a.dtype, a.key, a.value, a.slots = cache_args(sv, **kw), 4, sv.SPEC_BF16, P, P, P
        assert call(a, None) == getattr(sv, status)
    assert sv.spec_attn_launch(attn_args(sv, cache=cache_args(sv, **kw)), None) == getattr(sv, status)


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), "SPEC_EINVAL"), (dict(dtype=5), "SPEC_EDTYPE"), (dict(key=None), "SPEC_EINVAL"),
    (dict(value=None), "SPEC_EINVAL"), (dict(slots=None), "SPEC_EINVAL")])
def test_write_and_read_refusals(sv, kw, status):
    for call, struct in ((sv.spec_kv_write_launch, sv.SpecKVWriteArgs), (sv.spec_kv_read_launch, sv.SpecKVReadArgs)):
        a = struct()
        a.cache, a.N, a.dtype, a.key, a.value, a.slots = cache_args(sv), 4, sv.SPEC_BF16, P, P, P
        for k, v in kw.items():
            setattr(a, k, v)
        assert call(a, None) == getattr(sv, status)
        a = struct()
        a.cache, a.N = cache_args(sv), 0
        assert call(a, None) == sv.SPEC_OK
    for stride in ("k_token_stride", "k_head_stride", "v_token_stride", "v_head_stride"):
        a = sv.SpecKVWriteArgs()
        a.cache, a.N, a.dtype, a.key, a.value, a.slots = cache_args(sv), 4, sv.SPEC_BF16, P, P, P
        setattr(a, stride, -1)
        assert sv.spec_kv_write_launch(a, None) == sv.SPEC_EINVAL
    # grids past one dispatch of 2^32 work-items
    a = sv.SpecKVWriteArgs()
    a.cache, a.dtype, a.key, a.value, a.slots = cache_args(sv, heads=1024, token_stride=2 ** 16, block_stride=2 ** 20,
                                                           scale_block_stride=1024), sv.SPEC_BF16, P, P, P
    a.N = 2 ** 30
    assert sv.spec_kv_write_launch(a, None) == sv.SPEC_EINVAL
    r = sv.SpecKVReadArgs()
    r.cache, r.N, r.dtype, r.key, r.value, r.slots = a.cache, 2 ** 30, sv.SPEC_BF16, P, P, P
    assert sv.spec_kv_read_launch(r, None) == sv.SPEC_EINVAL
    assert sv.lib.spec_kv_write_launch(None, None) == sv.SPEC_EINVAL
    assert sv.lib.spec_kv_read_launch(None, None) == sv.SPEC_EINVAL


# ----------------------------------------------------------------- attention
def attn_args(sv, **kw):
    a = sv.SpecAttnArgs()
    a.cache, a.B, a.N, a.q_heads, a.max_q, a.max_ctx, a.window = cache_args(sv), 3, 6, 8, 2, 100, 0
    a.dtype, a.scale, a.q, a.q_token_stride, a.q_head_stride = sv.SPEC_BF16, 0.125, P, 512, 64
    a.q_start = a.ctx_len = a.block_table = a.out = a.lse = a.workspace = P
    a.bt_row_stride, a.max_blocks, a.workspace_bytes = 8, 7, 1 << 30
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), "SPEC_EINVAL"), (dict(N=-1), "SPEC_EINVAL"), (dict(q_heads=3), "SPEC_EINVAL"),
    (dict(q_heads=0), "SPEC_EINVAL"), (dict(q_heads=130), "SPEC_EINVAL"), (dict(max_q=0), "SPEC_EINVAL"),
    (dict(max_q=2 ** 24 + 1), "SPEC_EINVAL"), (dict(max_ctx=-1), "SPEC_EINVAL"), (dict(max_ctx=2 ** 30 + 1), "SPEC_EINVAL"),
    (dict(window=-1), "SPEC_EINVAL"), (dict(dtype=0), "SPEC_EDTYPE"), (dict(scale=math.nan), "SPEC_EINVAL"),
    (dict(scale=math.inf), "SPEC_EINVAL"), (dict(q=None), "SPEC_EINVAL"), (dict(q_start=None), "SPEC_EINVAL"),
    (dict(ctx_len=None), "SPEC_EINVAL"), (dict(block_table=None), "SPEC_EINVAL"), (dict(out=None), "SPEC_EINVAL"),
    (dict(out=P + 4), "SPEC_EALIGN"), (dict(max_blocks=-1), "SPEC_EINVAL"), (dict(bt_row_stride=6), "SPEC_EINVAL"),
    (dict(q_token_stride=-1), "SPEC_EINVAL"), (dict(q_head_stride=-64), "SPEC_EINVAL"),
    (dict(B=2 ** 30, max_q=2 ** 24), "SPEC_EINVAL"), (dict(B=2 ** 25, N=2 ** 25), "SPEC_EINVAL")])
def test_attention_refusals(sv, kw, status):
    assert sv.spec_attn_launch(attn_args(sv, **kw), None) == getattr(sv, status)


def test_attention_workspace(sv):
    """Few requests with long contexts are split and need a workspace."""
    a = attn_args(sv, max_ctx=100000)
    need = sv.spec_attn_workspace_bytes(a)
    assert need > 0
    for kw, status in ((dict(workspace=None), sv.SPEC_EINVAL), (dict(workspace=P + 8), sv.SPEC_EALIGN),
                       (dict(workspace_bytes=need - 1), sv.SPEC_EWORKSPACE)):
        assert sv.spec_attn_launch(attn_args(sv, max_ctx=100000, **kw), None) == status
    assert sv.spec_attn_workspace_bytes(attn_args(sv, max_q=0)) == 0
    assert sv.lib.spec_attn_workspace_bytes(None) == 0 and sv.lib.spec_attn_launch(None, None) == sv.SPEC_EINVAL


def test_attention_of_nothing(sv):
    assert sv.spec_attn_launch(attn_args(sv, B=0, q=None), None) == sv.SPEC_OK
    assert sv.spec_attn_launch(attn_args(sv, N=0, out=None), None) == sv.SPEC_OK


# ------------------------------------------------------------------- binding
def test_binding_refusals(sv):
    """Host tensors, wrong shapes and types are refused before the library."""
    x = torch.zeros(1, 2, 10)
    with pytest.raises(ValueError):
        sv.token_logprobs(x, torch.zeros(1, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        sv.make_kv_cache(2, 16, 1, 64, device="cpu")
    with pytest.raises(ValueError):
        sv.make_kv_cache(2, 16, 1, 64, scale_tokens=3, device="cpu")


# --------------------------------------------------------------- the oracle
def test_oracle_conversion_against_torch():
    x = torch.cat([torch.linspace(-448, 448, 40001), torch.randn(20000) * 0.01, torch.linspace(-2e-2, 2e-2, 3001)])
    assert np.array_equal(oo.DECODE[oo.encode(x.double().numpy())], x.to(torch.float8_e4m3fn).double().numpy())
    codes = np.arange(256, dtype=np.uint8)
    assert np.array_equal(oo.DECODE, torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy(), equal_nan=True)
    ties = torch.tensor([17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10])
    assert np.array_equal(oo.DECODE[oo.encode(ties.double().numpy())], [16.0, 20.0, 0.0, 2.0 ** -8])


def test_oracle_group_exponent():
    """The smallest power of two that holds the largest value of a group."""
    for amax, e in ((448.0, 0), (448.5, 1), (1.0, -8), (1.75, -8), (1.76, -7), (0.0, -117), (2.0 ** -130, -117)):
        codes, scales = np.zeros((1, 16, 1, 16), np.uint8), np.zeros((1, 1, 1), np.uint8)
        x = np.zeros((1, 1, 16))
        x[0, 0, 3] = -amax
        oo.kv_write(codes, scales, x, [0], 16)
        assert int(scales[0, 0, 0]) - 127 == e


def test_attention_sizes_past_64_bits(sv):
    """Sizes whose products pass what the plan counts in are refused."""
    for kw in (dict(B=2 ** 31 - 1, q_heads=128, max_q=2 ** 24, max_ctx=2 ** 30), dict(B=2 ** 31 - 1, max_q=2 ** 24)):
        a = attn_args(sv, **kw)
        a.cache.heads = 2
        assert sv.spec_attn_launch(a, None) == sv.SPEC_EINVAL and sv.spec_attn_workspace_bytes(a) == 0
    assert sv.spec_attn_launch(attn_args(sv, scale=3e38), None) == sv.SPEC_EINVAL
    assert sv.spec_attn_launch(attn_args(sv, scale=-3e38), None) == sv.SPEC_EINVAL
