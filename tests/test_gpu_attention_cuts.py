"""Attention over the 8-bit paged cache on the GPU where a wave goes through
more tiles than it holds pages of, and at sizes that take the cuts of the work
which small batches do not: against the definition in 64 bits, computed here by
torch (tests/test_attention_plan.py checks which cut each batch takes)."""
import math

import pytest
import torch

import ops_oracle as oo
from attention_cases import CASES

pytestmark = pytest.mark.gpu
U = oo.U


@pytest.fixture(scope="module")
def sv():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import rejection_sampling_verify_03_amd as m
    return m


def batch(c, seed):
    """Queries, cache tensors and tables of a batch, on the GPU; pages in random
    order, some of them missing behind position 1056."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    bs, st, heads, dim = c["bs"], c["st"], c["heads"], c["dim"]
    ctx = torch.tensor(c["ctx"], device="cuda")
    need = (ctx + bs - 1) // bs
    blocks = int(need.sum()) + 2
    cols = int(need.max())
    # entry j of request b is number (entries in front) + j of a random order of the blocks
    perm = torch.randperm(blocks, generator=g, device="cuda")
    at = (need.cumsum(0) - need)[:, None] + torch.arange(cols, device="cuda")
    inside = torch.arange(cols, device="cuda")[None] < need[:, None]
    table = torch.where(inside, perm[at.clamp(max=blocks - 1)], -1).int()
    if c["holes"]:
        hole = torch.rand(table.shape, generator=g, device="cuda") < 0.04
        hole[:, :1056 // bs] = False
        table[hole] = -1

    def codes():
        shape = (blocks, bs, heads, dim) if c["order"] == "tokens" else (blocks, heads, bs, dim)
        x = (torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16) * 90).clamp_(-448, 448)
        x = x.to(torch.float8_e4m3fn).view(torch.uint8)
        return x if c["order"] == "tokens" else x.transpose(1, 2)

    def scales():
        return torch.randint(118, 123, (blocks, heads, bs // st), generator=g, device="cuda").to(torch.uint8)
    k, v, ks, vs = codes(), codes(), scales(), scales()
    q = (torch.randn(sum(c["lens"]), c["G"] * heads, dim, generator=g, device="cuda") * 2).to(torch.bfloat16)
    q_start = torch.tensor([0] + c["lens"], device="cuda").cumsum(0).int()
    return q, (k, v, ks, vs), table, q_start, ctx.int()


def values(codes, scales, table, L, c):
    """Values [L, heads, dim] in 64 bits and whether each position exists."""
    pos = torch.arange(L, device="cuda")
    page = table[pos // c["bs"]].long()
    there = (page >= 0) & (page < codes.shape[0])
    page = page.clamp(min=0)
    decode = torch.from_numpy(oo.DECODE).cuda()
    e = scales[page, :, pos % c["bs"] // c["st"]].double() - 127
    return decode[codes[page, pos % c["bs"]].int()] * torch.exp2(e)[..., None], there


def check_request(c, b, q, cache, table, q_start, out, lse):
    """One request against the definition.  Scores: 2 D U scale sum|q k| and
    two roundings; weights and output half a step of bf16 each; sums kept in 32
    bits: one step U of the sum of magnitudes for each of a lane's tiles, and
    four in the matrix products."""
    L, D, G = c["ctx"][b], c["dim"], c["G"]
    r0, r1 = int(q_start[b]), int(q_start[b + 1])
    n = r1 - r0
    if n == 0:
        return 0
    K, there = values(cache[0], cache[2], table[b], L, c)
    V, _ = values(cache[1], cache[3], table[b], L, c)
    pos = torch.arange(L, device="cuda")
    p = L - n + torch.arange(n, device="cuda")
    see = there[None] & (pos[None] <= p[:, None])
    if c["window"]:
        see &= pos[None] > p[:, None] - c["window"]
    see = see.repeat_interleave(G, 0)  # rows token-major
    scale, steps = D ** -0.5, L / 32 + 64
    for h in range(c["heads"]):
        rows = q[r0:r1, h * G:(h + 1) * G].reshape(n * G, D).double()
        k, v = K[:, h].contiguous(), V[:, h].contiguous()
        s = torch.where(see, rows @ k.T.contiguous() * scale, -math.inf)
        big = torch.where(see, rows.abs() @ k.abs().T.contiguous() * scale, 0.0)
        m = s.amax(1, keepdim=True) if L else torch.full((n * G, 1), -math.inf, device="cuda", dtype=torch.float64)
        some = m > -math.inf
        m = torch.where(some, m, 0.0)
        w = torch.exp(s - m)
        l = w.sum(1, keepdim=True)
        w = torch.where(some, w / l, 0.0)
        want, z = w @ v, torch.where(some, m + torch.log(l), -math.inf)[:, 0]
        ds = 2 * D * U * (big.amax(1) if L else 0.0)
        ds = ds + 8 * U * (torch.where(see, s.abs(), 0.0).amax(1) if L else 0.0) + 8 * U * m[:, 0].abs() + steps * U
        mag = w @ v.abs()
        otol = 2.0 ** -8 * (want.abs() + mag) + (2 * ds[:, None] + 4 * steps * U) * mag + 1e-30
        got = out[r0:r1, h * G:(h + 1) * G].reshape(n * G, D).double()
        assert bool(((got - want).abs() <= otol).all()), (b, h, float(((got - want).abs() / otol).max()))
        got = lse[r0:r1, h * G:(h + 1) * G].reshape(n * G).double()
        off = torch.where(some[:, 0], (got - z).abs() - ds - 2 * U * z.abs(), torch.where(got == z, 0.0, 1.0))
        assert bool((off <= 0).all()), (b, h, float(off.max()))
    return n


@pytest.mark.parametrize("c", CASES, ids=[c["name"] for c in CASES])
def test_against_the_definition(sv, c):
    q, cache, table, q_start, ctx = batch(c, len(c["ctx"]) + c["heads"])
    kv = sv.KVCache(*cache)
    out, lse = sv.kv_attention(q, kv, table, q_start, ctx, max_q=max(c["lens"]), max_ctx=c["max_ctx"],
                               window=c["window"], return_lse=True)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(out.float()).all())
    B = len(c["ctx"])
    step = 1 if B <= 1000 else B // 400  # (of tens of thousands of small requests a part, the last among them)
    rows = sum(check_request(c, b, q, cache, table, q_start, out, lse) for b in range(B - 1, -1, -step))
    assert rows > 0
    if step > 1:
        # all of them as the cut of short contexts gives them
        o, z = sv.kv_attention(q, kv, table, q_start, ctx, max_q=max(c["lens"]), max_ctx=100, return_lse=True)
        torch.cuda.synchronize()
        assert torch.equal(o, out) and torch.equal(z, lse)
