"""Groups of the 8-bit paged cache with a scale byte of 0, which nothing was
written to yet: they hold values of 0 whatever their codes, NaN ones among
them, for the read, the attention and a write behind their first token."""
import numpy as np
import pytest
import torch

import ops_oracle as oo
from test_gpu_attention import FAR, Case, compare, sv  # noqa: F401  (sv: the fixture)

pytestmark = pytest.mark.gpu


def unwritten(codes, scales, st, seed):
    """Scales with a third of the bytes 0, codes with NaN ones there and as
    they were elsewhere, and codes with zeros there."""
    g = torch.Generator().manual_seed(seed)
    scales = torch.where(torch.rand(scales.shape, generator=g) < 1 / 3, 0, scales)
    none = (scales.repeat_interleave(st, 2).transpose(1, 2) == 0)[..., None]
    nan = torch.rand(codes.shape, generator=g) < 0.1
    return torch.where(none & nan, 0x7F, codes), scales, torch.where(none, 0, codes)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bs,st", [(16, 16), (32, 4), (16, 1)])
def test_read(sv, bs, st, dtype):  # noqa: F811
    k, v, ks, vs = oo.random_cache(7, bs, 3, 48, st, bs + st)
    k, ks, k0 = unwritten(k, ks, st, 1)
    v, vs, v0 = unwritten(v, vs, st, 2)
    slots = torch.arange(7 * bs)
    got = sv.kv_read(sv.KVCache(k.cuda(), v.cuda(), ks.cuda(), vs.cuda()), slots.cuda(), dtype=dtype)
    torch.cuda.synchronize()
    for x, c, s in ((got[0], k0, ks), (got[1], v0, vs)):
        assert np.array_equal(x.cpu().double().numpy(), oo.kv_values(c.numpy(), s.numpy(), slots.numpy(), st))


@pytest.mark.parametrize("st", [4, 16, 64])
def test_write_behind_the_first_token(sv, st):  # noqa: F811
    bs, heads, dim = 64, 2, 64
    k, v, _, _ = oo.random_cache(3, bs, heads, dim, st, st)
    k[:, ::3], v[:, 1::3] = 0x7F, 0xFF
    zero = torch.zeros(3, heads, bs // st, dtype=torch.uint8)
    cache = sv.KVCache(k.cuda(), v.cuda(), zero.cuda(), zero.cuda())
    g = torch.Generator().manual_seed(3)
    slots = torch.tensor([st - 2, st - 1, bs + st // 2, 2 * bs + 1])
    key, value = (torch.randn(4, heads, dim, generator=g) for _ in range(2))
    want = [t.numpy().copy() for t in (k, zero, v, zero)]
    for s in slots.tolist():
        first = s - s % st
        if s != st - 1:
            for c in (want[0], want[2]):  # the tokens in front of the written ones
                c.reshape(-1, heads, dim)[first:s] = 0
    oo.kv_write(want[0], want[1], key.double().numpy(), slots.tolist(), st)
    oo.kv_write(want[2], want[3], value.double().numpy(), slots.tolist(), st)
    sv.kv_write(cache, key.cuda(), value.cuda(), slots.cuda())
    torch.cuda.synchronize()
    got = oo.to_numpy(cache)
    assert np.array_equal(got[1], want[1]) and np.array_equal(got[3], want[3])
    assert oo.same_codes(got[0], want[0]) and oo.same_codes(got[2], want[2])


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("dim,n,G", [(64, 1, 4), (64, 9, 8), (128, 20, 2), (256, 3, 2)])
@pytest.mark.parametrize("bs,st", [(16, 16), (64, 64), (16, 4), (16, 1)])
def test_attention(sv, bs, st, dim, n, G, far):  # noqa: F811
    c = Case([n, 1], [1300, 41], G, 2, dim, bs, st, dim + st + n)
    c.k, c.ks, k0 = unwritten(c.k, c.ks, st, 4)
    c.v, c.vs, v0 = unwritten(c.v, c.vs, st, 5)
    out, lse = c.call(sv, window=1111, **(dict(max_ctx=FAR) if far else {}))
    torch.cuda.synchronize()
    c.k, c.v = k0, v0
    compare(out, lse, *c.want(window=1111))
