"""Attention over the 4-bit paged cache on the GPU against the 64-bit
definition: head layouts, lengths from none to long ones, windows, sinks,
pages that are missing or end inside a tile, what a token does not see, every
cut of the work, requests that cannot be used, and a whole decode round."""
import math

import numpy as np
import pytest
import torch

import decode_oracle as do
from attention_cases import CASES

pytestmark = pytest.mark.gpu
FAR = 1 << 22  # a bound on the contexts that takes the cut of long ones


@pytest.fixture(scope="module")
def sv():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import rejection_sampling_verify_03_amd as m
    return m


class Case:
    def __init__(self, lens, ctx, G, heads, dim, bs, seed, spare=2, order="heads"):
        g = torch.Generator().manual_seed(seed)
        need = [-(-c // bs) for c in ctx]
        blocks = sum(need) + spare
        perm = torch.randperm(blocks, generator=g)
        self.table = torch.full((len(ctx), max(max(need), 1) + 1), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n].int()
            at += n
        self.k, self.v, self.ks, self.vs = do.random_cache(blocks, bs, heads, dim, seed, order)
        self.q = torch.randn(sum(lens), G * heads, dim, generator=g).to(torch.bfloat16)
        self.q_start = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
        self.ctx = torch.tensor(ctx, dtype=torch.int32)
        self.sinks = torch.randn(G * heads, generator=g)
        self.max_q, self.max_ctx = max(max(lens), 1), max(ctx)

    def cache(self, sv):
        return sv.KVCache4(do.up(self.k), do.up(self.v), self.ks.cuda(), self.vs.cuda())

    def call(self, sv, window=0, sinks=False, q=None, **kw):
        kw.setdefault("max_q", self.max_q)
        kw.setdefault("max_ctx", self.max_ctx)
        out = sv.kv_attention(self.q.cuda() if q is None else q, self.cache(sv), self.table.cuda(), self.q_start.cuda(),
                              self.ctx.cuda(), window=window, sinks=self.sinks.cuda() if sinks else None, return_lse=True, **kw)
        torch.cuda.synchronize()
        return out

    def want(self, window=0, sinks=False, scale=None):
        return do.attention(self.q, self.k.numpy(), self.ks.numpy(), self.v.numpy(), self.vs.numpy(), self.table.numpy(),
                            self.q_start.tolist(), self.ctx.tolist(), self.q.shape[2] ** -0.5 if scale is None else scale,
                            window, self.sinks if sinks else None)

    def check(self, sv, window=0, sinks=False, scale=None, **kw):
        out, lse = self.call(sv, window, sinks, scale=scale, **kw)
        compare(out, lse, *self.want(window, sinks, scale))
        return out, lse


def compare(out, lse, o, z, otol, ltol):
    got = out.cpu().double().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(o))
    fin = ~np.isnan(o)
    assert np.all(np.abs(got - o)[fin] <= otol[fin]), np.max((np.abs(got - o) / otol)[fin])
    got = lse.cpu().double().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(z)) and np.array_equal(np.isinf(got), np.isinf(z))
    fin = np.isfinite(z)
    assert np.all(np.abs(got - z)[fin] <= ltol[fin]), np.max((np.abs(got - z) / ltol)[fin])


@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("G,heads", [(1, 3), (8, 2), (5, 1)])
def test_head_layouts(sv, dim, G, heads):
    Case([1, 4, 2], [70, 33, 200], G, heads, dim, 16, dim + G).check(sv)


@pytest.mark.parametrize("bs", [16, 32, 64, 256, 1024])
@pytest.mark.parametrize("order", ["tokens", "heads"])
def test_pages(sv, bs, order):
    Case([3, 1], [bs + 5, 3 * bs if bs < 200 else bs + 40], 4, 2, 64, bs, bs, order=order).check(sv)
    Case([1, 1], [bs + 5, bs], 2, 4, 128, bs, bs, order=order).check(sv)


@pytest.mark.parametrize("ctx", [1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 1000])
def test_lengths(sv, ctx):
    c = Case([1, min(ctx, 5)], [ctx, ctx], 4, 1, 64, 16, ctx)
    c.check(sv)
    c.check(sv, sinks=True)


def test_a_request_without_context_or_tokens(sv):
    c = Case([2, 0, 3, 1], [0, 40, 2, 50], 2, 2, 64, 16, 4)
    out, lse = c.check(sv)
    assert not bool(out[:2].any()) and bool((lse[:2] == -math.inf).all())
    assert not bool(out[2].any())  # three new tokens, two of them in the cache
    c.check(sv, sinks=True)


@pytest.mark.parametrize("window", [1, 2, 16, 31, 33, 100, 129, 5000])
@pytest.mark.parametrize("n", [1, 9, 70])
def test_windows(sv, window, n):
    c = Case([n, 1], [300, 299], 4, 1, 64, 32, window + n)
    c.check(sv, window=window, sinks=window % 2 == 1)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_many_rows(sv, dim):
    """Blocks of rows of each size, ragged, and more than one of them."""
    for n, G in ((2, 8), (3, 8), (5, 8), (9, 8), (33, 8), (130, 1), (17, 16), (40, 3)):
        if dim == 64 or n <= 33:
            Case([n, n // 2 + 1], [n + 77, n + 120], G, 1, dim, 16, n * G).check(sv)


@pytest.mark.parametrize("dim,n,G", [(64, 1, 8), (128, 2, 4), (256, 1, 1), (64, 9, 8), (96, 3, 2)])
def test_long_contexts_in_runs(sv, dim, n, G):
    c = Case([n, 1], [5000, 1203], G, 1, dim, 64, dim + n)
    c.check(sv)
    c.check(sv, sinks=True, window=3000)


@pytest.mark.parametrize("order", ["tokens", "heads"])
@pytest.mark.parametrize("dim,heads,G,n", [(64, 4, 8, 1), (128, 12, 2, 1), (256, 2, 3, 1), (64, 2, 8, 9), (128, 4, 4, 6)])
def test_runs_at_small_sizes(sv, dim, heads, G, n, order):
    """The cut of long contexts (equal runs, a head to a wave, joins)."""
    c = Case([n, 1, n], [700, 33, 1100], G, heads, dim, 16, dim + heads, order=order)
    c.check(sv, max_ctx=FAR)
    c.check(sv, max_ctx=FAR, window=300, sinks=True)


def test_peaked_and_flat_scores(sv):
    c = Case([4], [600], 4, 1, 64, 16, 9)
    c.check(sv, scale=4.0)     # weights of single keys near one
    c.check(sv, scale=0.0)     # all equal
    c.check(sv, scale=-0.125)


@pytest.mark.parametrize("far", [False, True])
def test_missing_pages_are_not_seen(sv, far):
    kw = dict(max_ctx=FAR) if far else {}
    c = Case([2, 1], [160, 100], 4, 2, 64, 16, 30)
    c.table = torch.cat([c.table, torch.full((2, FAR // 16), -1, dtype=torch.int32)], 1) if far else c.table
    c.table[0, 0], c.table[0, 3], c.table[1, 2] = -1, 10 ** 6, -5
    c.check(sv, **kw)
    c.table[1, :] = -1
    out, lse = c.check(sv, **kw)
    assert not bool(out[2].any()) and bool((lse[2] == -math.inf).all())


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("far", [False, True])
def test_what_is_not_seen_never_reaches_the_output(sv, dim, far):
    """Exponent bytes of NaN behind the context, in front of the window and at
    later tokens."""
    kw = dict(max_ctx=FAR) if far else {}
    c = Case([3, 1], [37, 70], 4, 1, dim, 16, 40)
    last, first = int(c.table[0, 2]), int(c.table[1, 0])
    for t in (c.ks, c.vs):
        t[last, :, :, 5:] = 255   # positions 37.. of request 0
        t[first] = 255            # request 1: positions 0..15, behind the window
    out, lse = c.call(sv, window=40, **kw)
    compare(out, lse, *c.want(window=40))
    assert bool(torch.isfinite(out.float()).all())
    # a NaN group of the last token's value is seen by that token alone, in its dims
    c = Case([3], [37], 4, 1, dim, 16, 41)
    page = int(c.table[0, 2])
    c.vs[page, 0, 1, 4] = 255     # position 36, dims 32..63
    c.ks[page, 0, 0, 3] = 255     # position 35: tokens 1 and 2 have a NaN score
    out, lse = c.call(sv, **kw)
    assert bool(torch.isfinite(out[0].float()).all()) and bool(torch.isfinite(lse[0]).all())
    assert bool(torch.isnan(out[1:].float()).all()) and bool(torch.isnan(lse[1:]).all())
    c.ks[page, 0, 0, 3] = 127
    out, lse = c.call(sv, **kw)
    bad = torch.isnan(out.float()).cpu()
    assert bool(torch.isfinite(lse).all()) and bool(bad[2, :, 32:64].all()) and int(bad.sum()) == 4 * 32
    o, z, otol, ltol = c.want()
    assert np.array_equal(np.isnan(o), bad.numpy())
    compare(out, lse, o, z, otol, ltol)


def test_a_nan_that_every_row_sees(sv):
    c = Case([2], [300], 4, 2, 128, 16, 42)
    c.vs[int(c.table[0, 1]), 1, 2, 3] = 255
    out, lse = c.call(sv)
    compare(out, lse, *c.want())
    bad = torch.isnan(out.float()).cpu()
    assert bool(bad[:, 4:, 64:96].all()) and int(bad.sum()) == 2 * 4 * 32


def test_unusable_requests_and_rows_outside(sv):
    c = Case([2, 3, 1, 2], [50, 60, 70, 80], 2, 2, 64, 16, 50)
    q = torch.cat([c.q, c.q[:3]]).cuda()     # three rows behind the last request
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    c.ctx[1], c.ctx[2] = -1, 10 ** 6
    got, lse = c.call(sv, q=q, out=out, max_q=2)
    assert got is out and bool((out[8:] == 7.0).all())
    assert bool(torch.isnan(out[2:6].float()).all()) and bool(torch.isnan(lse[2:6]).all())
    assert bool(torch.isfinite(out[:2].float()).all()) and bool(torch.isfinite(out[6:8].float()).all())


def test_strided_queries_and_other_types(sv):
    c = Case([3, 2], [90, 41], 4, 2, 96, 16, 60)
    wide = torch.zeros(5, 8, 200, dtype=torch.bfloat16)
    wide[..., 7:103] = c.q
    d = wide.cuda()
    out, lse = c.call(sv, q=d[..., 7:103])
    compare(out, lse, *c.want())
    cache = c.cache(sv)
    typed = sv.KVCache4(cache.k.view(torch.float4_e2m1fn_x2), cache.v.view(torch.float4_e2m1fn_x2),
                        cache.k_scale.view(torch.float8_e8m0fnu), cache.v_scale.view(torch.float8_e8m0fnu))
    o, none = sv.kv_attention(c.q.cuda(), typed, c.table.cuda(), c.q_start.cuda(), c.ctx.cuda(), max_q=c.max_q,
                              max_ctx=c.max_ctx)
    torch.cuda.synchronize()
    assert none is None and torch.equal(o, out)
    with pytest.raises(TypeError):
        sv.kv_attention(c.q.float().cuda(), typed, c.table.cuda(), c.q_start.cuda(), c.ctx.cuda(), max_q=3)
    with pytest.raises(ValueError):
        sv.kv_attention(c.q[..., :64].contiguous().cuda(), typed, c.table.cuda(), c.q_start.cuda(), c.ctx.cuda(), max_q=3)


def test_offsets_past_32_bits(sv):
    """Pages that begin past 2^32 bytes."""
    c = Case([2], [100], 4, 1, 256, 16, 61)
    blocks = 2 ** 32 // (16 * 128) + 40
    k, v = (torch.empty(blocks, 1, 16, 128, dtype=torch.uint8, device="cuda").transpose(1, 2) for _ in range(2))
    scales = [torch.empty(blocks, 1, 8, 16, dtype=torch.uint8, device="cuda") for _ in range(2)]
    far = c.table.clone()
    for j in range(7):
        p, f = int(c.table[0, j]), blocks - 1 - 3 * j
        far[0, j] = f
        k[f], v[f], scales[0][f], scales[1][f] = c.k[p].cuda(), c.v[p].cuda(), c.ks[p].cuda(), c.vs[p].cuda()
    for bound in (100, FAR):
        out, lse = sv.kv_attention(c.q.cuda(), sv.KVCache4(k, v, *scales), far.cuda(), c.q_start.cuda(), c.ctx.cuda(), max_q=2,
                                   max_ctx=bound, return_lse=True)
        torch.cuda.synchronize()
        compare(out, lse, *c.want())


def test_replays_with_a_shared_workspace(sv):
    cs = [Case([1, 1], [900, 1300], 8, 2, 64, 16, 86), Case([3, 1], [1100, 200], 4, 4, 128, 16, 87)]
    args = [(c.q.cuda(), c.cache(sv), c.table.cuda(), c.q_start.cuda(), c.ctx.cuda()) for c in cs]
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")

    def go(i, **kw):
        return sv.kv_attention(*args[i], max_q=cs[i].max_q, max_ctx=FAR, return_lse=True, **kw)
    for i in range(2):
        go(i, workspace=ws)
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph() for _ in cs], []
    for i, graph in enumerate(graphs):
        with torch.cuda.graph(graph):
            outs.append(go(i, workspace=ws))
    for lens in (([900, 1300], [1100, 200]), ([17, 1001], [5, 0]), ([1, 0], [1100, 199])):
        for i in range(2):
            args[i][4].copy_(torch.tensor(lens[i], dtype=torch.int32))
            graphs[i].replay()
            o, z = go(i)
            torch.cuda.synchronize()
            assert torch.equal(outs[i][0], o) and torch.equal(outs[i][1], z)
    streams = [torch.cuda.Stream() for _ in cs]
    want = [go(i) for i in range(2)]
    torch.cuda.synchronize()
    got = [go(i, stream=s) for i, s in enumerate(streams)]
    for s in streams:
        s.synchronize()
    for (a, b), (x, y) in zip(got, want):
        assert torch.equal(a, x) and torch.equal(b, y)


# ------------------------------------------------- every cut, on the GPU
def values(codes, scales, table, L, bs):
    """Values [L, heads, dim] in 64 bits and whether each position exists."""
    pos = torch.arange(L, device="cuda")
    page = table[pos // bs].long()
    there = (page >= 0) & (page < codes.shape[0])
    page = page.clamp(min=0)
    c = codes[page, pos % bs].int()
    c = torch.stack([c & 15, c >> 4], -1).flatten(-2)
    grid = torch.from_numpy(do.GRID).cuda()
    x = torch.where(c >= 8, -1.0, 1.0).double() * grid[c & 7]
    e = scales[page, :, :, pos % bs].double() - 127
    return (x.unflatten(-1, (-1, 32)) * torch.exp2(e)[..., None]).flatten(-2), there


def check_request(c, b, dim, q, cache, table, q_start, out, lse):
    """One request against the definition, with the tolerances of
    decode_oracle.attention, and a step of fp32 of the sum of magnitudes for
    each tile and four in the matrix products."""
    L, G, U = c["ctx"][b], c["G"], do.U
    r0, r1 = int(q_start[b]), int(q_start[b + 1])
    n = r1 - r0
    if n == 0:
        return 0
    K, there = values(cache[0], cache[2], table[b], L, c["bs"])
    V, _ = values(cache[1], cache[3], table[b], L, c["bs"])
    pos = torch.arange(L, device="cuda")
    p = L - n + torch.arange(n, device="cuda")
    see = there[None] & (pos[None] <= p[:, None])
    if c["window"]:
        see &= pos[None] > p[:, None] - c["window"]
    see = see.repeat_interleave(G, 0)  # rows token-major
    scale, steps = dim ** -0.5, L / 32 + 64
    for h in range(c["heads"]):
        rows = q[r0:r1, h * G:(h + 1) * G].reshape(n * G, dim).double()
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
        ds = 2 * dim * U * (big.amax(1) if L else 0.0)
        ds = ds + 8 * U * (torch.where(see, s.abs(), 0.0).amax(1) if L else 0.0) + 8 * U * m[:, 0].abs() + steps * U
        mag = w @ v.abs()
        otol = 2.0 ** -8 * (want.abs() + mag) + (2 * ds[:, None] + 4 * steps * U) * mag + 1e-30
        got = out[r0:r1, h * G:(h + 1) * G].reshape(n * G, dim).double()
        assert bool(((got - want).abs() <= otol).all()), (b, h, float(((got - want).abs() / otol).max()))
        got = lse[r0:r1, h * G:(h + 1) * G].reshape(n * G).double()
        off = torch.where(some[:, 0], (got - z).abs() - ds - 2 * U * z.abs(), torch.where(got == z, 0.0, 1.0))
        assert bool((off <= 0).all()), (b, h, float(off.max()))
    return n


@pytest.mark.parametrize("c", CASES, ids=[c["name"] for c in CASES])
def test_every_cut(sv, c):
    """The 8-bit cache's batches over the 4-bit one, head sizes rounded up to
    whole scales."""
    dim, bs, heads = (c["dim"] + 31) // 32 * 32, c["bs"], c["heads"]
    g = torch.Generator(device="cuda").manual_seed(len(c["ctx"]) + heads)
    ctx = torch.tensor(c["ctx"], device="cuda")
    need = (ctx + bs - 1) // bs
    blocks, cols = int(need.sum()) + 2, int(need.max())
    perm = torch.randperm(blocks, generator=g, device="cuda")
    at = (need.cumsum(0) - need)[:, None] + torch.arange(cols, device="cuda")
    inside = torch.arange(cols, device="cuda")[None] < need[:, None]
    table = torch.where(inside, perm[at.clamp(max=blocks - 1)], -1).int()
    if c["holes"]:
        hole = torch.rand(table.shape, generator=g, device="cuda") < 0.04
        hole[:, :1056 // bs] = False
        table[hole] = -1

    def codes():
        shape = (blocks, bs, heads, dim // 2) if c["order"] == "tokens" else (blocks, heads, bs, dim // 2)
        x = torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)
        return x if c["order"] == "tokens" else x.transpose(1, 2)

    def scales():
        return torch.randint(124, 128, (blocks, heads, dim // 32, bs), generator=g, device="cuda", dtype=torch.uint8)
    cache = codes(), codes(), scales(), scales()
    q = torch.randn(sum(c["lens"]), c["G"] * heads, dim, generator=g, device="cuda").to(torch.bfloat16)
    q_start = torch.tensor([0] + c["lens"], device="cuda").cumsum(0).int()
    kv = sv.KVCache4(*cache)
    out, lse = sv.kv_attention(q, kv, table, q_start, ctx.int(), max_q=max(c["lens"]), max_ctx=c["max_ctx"],
                               window=c["window"], return_lse=True)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(out.float()).all())
    B = len(c["ctx"])
    step = 1 if B <= 1000 else B // 400  # (of tens of thousands of small requests a part, the last among them)
    rows = sum(check_request(c, b, dim, q, cache, table, q_start, out, lse) for b in range(B - 1, -1, -step))
    assert rows > 0


def test_a_full_card(sv):
    """A unit to a wave's head, four heads to a workgroup: more requests than
    the 8-bit cache's batch of that cut has, as more workgroups are resident."""
    test_every_cut(sv, do.MANY_SHORT)


# ----------------------------------------------------------- a decode round
def test_a_decode_round(sv):
    """Expansion, rotation and cache write at its positions and slots, attention
    over the cache, drafts sampled from cut rows, and their verification: each
    from the outputs of the one before, each against its definition."""
    import workloads
    Hk, G, D, bs = 2, 4, 64, 16
    inp = workloads.verify_tiny(seed=5, device=torch.device("cuda"))
    B, K, V = inp.B, inp.K, inp.target.shape[-1]
    e = workloads.expand_inputs(B=B, K=K, H=64, seed=2, device=torch.device("cuda"), max_offset=200)
    nblk = -(-(int(e.in_positions.max()) + K + 3) // bs)
    table = torch.randperm(B * nblk, generator=torch.Generator().manual_seed(3)).view(B, nblk).int().cuda()
    out = sv.expand(e.in_token_ids, e.in_positions, e.in_start, e.accepted, e.bonus, K, e.mask_id, e.target_hidden,
                    e.mask_hidden, block_table=table, block_size=bs)
    N = out.slot_mapping.numel()
    k, v, ks, vs = do.random_cache(B * nblk, bs, Hk, D, 4)
    cache = sv.KVCache4(*(do.up(t) for t in (k, v, ks, vs)))
    g = torch.Generator().manual_seed(6)
    q, key, val = (torch.randn(N, h, D, generator=g).to(torch.bfloat16) for h in (Hk * G, Hk, Hk))
    rope = sv.make_rope(D, scaling="yarn", factor=4.0, trained=128, interleaved=True)
    f = rope.inv_freq.cpu().numpy()
    turned = sv.rope_kv_write(cache, q.cuda(), key.cuda(), val.cuda(), out.out_positions, out.slot_mapping, rope)
    torch.cuda.synchronize()
    pos, slots = out.out_positions.cpu(), out.slot_mapping.cpu()
    assert (slots == -1).any() and (slots >= 0).any()
    host = [t.numpy().copy() for t in (k, ks, v, vs)]
    do.kv_write(host[0], host[1], do.rotate(key.double().numpy(), pos.numpy(), f, rope.scale, True), slots.tolist())
    do.kv_write(host[2], host[3], val.double().numpy(), slots.tolist())
    for t, h in zip((cache.k, cache.k_scale, cache.v, cache.v_scale), host):
        assert np.array_equal(t.cpu().numpy(), h)
    want = do.rotate(q.double().numpy(), pos.numpy(), f, rope.scale, True)
    size = 2.0 ** -22 * rope.scale * 2 * float(q.abs().max())  # (fp32 products before the rounding to bf16)
    assert np.all(np.abs(turned.cpu().double().numpy() - want) <= 2.0 ** -8 * (np.abs(want) + size) + size)
    # the new tokens of the round: the bonus token and the MASK positions
    new = out.new_token_indices
    last = (pos[new[:, -1].long().cpu()] + 1).int()
    qs = torch.arange(B + 1, dtype=torch.int32) * K
    mine = turned[new.long().flatten()]
    o, z = sv.kv_attention(mine, cache, table, qs.cuda(), last.cuda(), max_q=K, return_lse=True)
    torch.cuda.synchronize()
    compare(o, z, *do.attention(mine.cpu(), host[0], host[1], host[2], host[3], table.cpu().numpy(), qs.tolist(),
                                last.tolist(), D ** -0.5))
    # drafts from the drafter's rows at the new tokens, cut, and their verification over cut rows
    T = torch.tensor([0.7, 1.0, 0.0, 1.2])[:B]
    cut = dict(top_k=torch.tensor([30, 0, 5, 200], dtype=torch.int32)[:B], top_p=torch.tensor([0.9, 0.95, 1.0, 1.0])[:B],
               min_p=torch.tensor([0.0, 0.0, 0.0, 0.01])[:B])
    dcut = {n: t.cuda() for n, t in cut.items()}
    logits = (torch.randn(N, V, generator=g) * 2).to(torch.float32)
    rows = logits[new.long().cpu()]
    target = torch.cat([rows, rows[:, :1]], 1) + 0.4 * torch.randn(B, K + 1, V, generator=g)
    u = torch.rand(B, K, generator=g)
    drafts = sv.sample(logits.cuda(), u.cuda(), T.cuda(), row_index=new, **dcut)
    assert np.array_equal(drafts.cpu().numpy(), do.sample(rows, u.tolist(), T, *cut.values()))
    p = sv.truncate_logits(target.cuda(), T.cuda(), **dcut)
    d = sv.truncate_logits(rows.cuda(), T.cuda(), **dcut)
    assert np.array_equal(p.cpu().double().numpy(), do.truncate(target, T, *cut.values()))
    acc, tok, _ = sv.verify(p, d, drafts, T.cuda(), seed=0, step=1)
    r = sv.token_logprobs(p, tok, T.cuda())
    torch.cuda.synchronize()
    assert bool((acc >= 0).all()) and bool(torch.isfinite(r.logprobs).all())
    kept = torch.isfinite(p.cpu())
    for b in range(B):
        for i in range(int(acc[b]) + 1):
            assert bool(kept[b, i, int(tok[b, i])])
