"""Attention over values that a cache holds and bf16 reads as infinite (a write
stores one of 1.9375 * 2^127 or more in 8 bits, of 1.75 * 2^127 or more in 4 as
2^128): the tokens that do not see them are the definition's, and of those that
do the other dims, where a scale is not multiplied into the weights (scales of
16 tokens and more, and 4 bits)."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
FAR = 1 << 22  # a bound on the contexts that takes the cut of long ones
U = 2.0 ** -24
BIG = 3.3e38


@pytest.fixture(scope="module")
def sv():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import rejection_sampling_verify_03_amd as m
    return m


def row(q, K, V, see, scale):
    """A row by the definition in 64 bits over the positions that it sees, and
    its tolerance: scores are sums of dim products in 32 bits with two more
    roundings, the weights of the second product and the output are bf16."""
    k, v = K[see], V[see]
    s = (k @ q) * scale
    m = s.max()
    w = np.exp(s - m)
    l = w.sum()
    w = w / l
    ds = 2 * len(q) * U * scale * (np.abs(k) @ np.abs(q)).max() + 8 * U * (np.abs(s).max() + abs(m)) + 64 * U
    fin = np.isfinite(v).all(0)
    v = np.where(fin, v, 0.0)
    o, mag = w @ v, w @ np.abs(v)
    z = m + math.log(l)
    return o, fin, 2.0 ** -8 * (np.abs(o) + mag) + 2 * ds * mag + 1e-30, z, ds + 2 * U * abs(z)


@pytest.mark.parametrize("form", ["8 bits, 16 tokens to a scale", "8 bits, a scale to a token", "4 bits"])
@pytest.mark.parametrize("dim,n,far", [(64, 2, False), (64, 5, True), (64, 17, False), (128, 3, False), (128, 11, True),
                                       (256, 3, False)])
def test_values_past_bf16_reach_only_who_sees_them(sv, form, dim, n, far):
    G, heads, bs, L, w = 4, 2, 16, 75, 40
    g = torch.Generator().manual_seed(dim + n)
    cache = (sv.make_kv4_cache(6, bs, heads, dim) if form == "4 bits" else
             sv.make_kv_cache(6, bs, heads, dim, scale_tokens=16 if "16" in form else 1))
    table = torch.tensor([[3, 0, 5, 1, 4]], dtype=torch.int32)
    pos = torch.arange(L)
    slots = table[0].long()[pos // bs] * bs + pos % bs
    key, val = (torch.randn(L, heads, dim, generator=g).to(torch.bfloat16) for _ in range(2))
    first = L - n - w + 1                 # under the window seen by the first new token alone
    val[first, 0, 5] = -BIG
    val[L - 1, 0, 7] = BIG                # by the last one alone
    val[L - 1, 1, dim - 1] = BIG          # of two signs: the last one sees both
    val[L - 2, 1, dim - 1] = -BIG
    sv.kv_write(cache, key.cuda(), val.cuda(), slots.cuda())
    K, V = (t.cpu().double().numpy() for t in sv.kv_read(cache, slots.cuda(), dtype=torch.float32))
    assert np.isinf(V[first, 0, 5]) and np.isinf(V[L - 1, 0, 7]) and np.isinf(V[L - 2:, 1, dim - 1]).all()
    assert np.isfinite(K).all() and np.isinf(V).sum() == 4
    q = torch.randn(n, G * heads, dim, generator=g).to(torch.bfloat16)
    out, lse = sv.kv_attention(q.cuda(), cache, table.cuda(), torch.tensor([0, n], dtype=torch.int32).cuda(),
                               torch.tensor([L], dtype=torch.int32).cuda(), max_q=n, max_ctx=FAR if far else L, window=w,
                               return_lse=True)
    torch.cuda.synchronize()
    out, lse = out.cpu().double().numpy(), lse.cpu().double().numpy()
    for i in range(n):
        p = L - n + i
        see = (np.arange(L) <= p) & (np.arange(L) > p - w)
        for h in range(G * heads):
            o, fin, otol, z, ltol = row(q[i, h].double().numpy(), K[:, h // G], V[:, h // G], see, dim ** -0.5)
            assert fin.sum() == dim - (h < G and i in (0, n - 1)) - (h >= G and i >= n - 2)
            if fin.all() or "a scale to a token" not in form:
                assert np.isfinite(out[i, h][fin]).all(), (i, h, np.nonzero(~np.isfinite(out[i, h]) & fin))
                assert np.all(np.abs(out[i, h] - o)[fin] <= otol[fin])
            if "a scale to a token" not in form:
                assert not np.isfinite(out[i, h][~fin]).any()
            assert abs(lse[i, h] - z) <= ltol
