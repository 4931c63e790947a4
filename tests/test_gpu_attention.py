"""Attention over the 8-bit paged cache on the GPU against the 64-bit
definition: head layouts, lengths from none to long ones, windows, sinks,
pages that are missing or end inside a tile, what a token does not see, and
requests that cannot be used."""
import math

import numpy as np
import pytest
import torch

import ops_oracle as oo

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import rejection_sampling_verify_03_amd as m
    return m


class Case:
    def __init__(self, lens, ctx, G, heads, dim, bs, st, seed, spare=2, order="tokens"):
        g = torch.Generator().manual_seed(seed)
        need = [-(-c // bs) for c in ctx]
        blocks = sum(need) + spare
        perm = torch.randperm(blocks, generator=g)
        self.table = torch.full((len(ctx), max(max(need), 1) + 1), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n].int()
            at += n
        k, v, ks, vs = oo.random_cache(blocks, bs, heads, dim, st, seed)
        if order == "heads":
            k, v = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k, v))
        self.k, self.v, self.ks, self.vs = k, v, ks, vs
        self.q = (torch.randn(sum(lens), G * heads, dim, generator=g) * 2).to(torch.bfloat16)
        self.q_start = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
        self.ctx = torch.tensor(ctx, dtype=torch.int32)
        self.sinks = torch.randn(G * heads, generator=g)
        self.max_q, self.max_ctx, self.st = max(max(lens), 1), max(ctx), st

    def cache(self, sv):
        def up(t):
            d = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda")
            return d.copy_(t)
        return sv.KVCache(up(self.k), up(self.v), self.ks.cuda(), self.vs.cuda())

    def call(self, sv, window=0, sinks=False, q=None, **kw):
        kw.setdefault("max_q", self.max_q)
        kw.setdefault("max_ctx", self.max_ctx)
        return sv.kv_attention(self.q.cuda() if q is None else q, self.cache(sv), self.table.cuda(),
                               self.q_start.cuda(), self.ctx.cuda(), window=window,
                               sinks=self.sinks.cuda() if sinks else None, return_lse=True, **kw)

    def want(self, window=0, sinks=False, scale=None):
        return oo.attention(self.q, self.k.numpy(), self.ks.numpy(), self.v.numpy(), self.vs.numpy(), self.st,
                            self.table.numpy(), self.q_start.tolist(), self.ctx.tolist(),
                            self.q.shape[2] ** -0.5 if scale is None else scale, window,
                            self.sinks if sinks else None)

    def check(self, sv, window=0, sinks=False, scale=None, **kw):
        out, lse = self.call(sv, window, sinks, scale=scale, **kw)
        torch.cuda.synchronize()
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


@pytest.mark.parametrize("dim", [16, 32, 64, 80, 96, 128, 192, 256])
@pytest.mark.parametrize("G,heads", [(1, 3), (8, 2), (5, 1)])
def test_head_layouts(sv, dim, G, heads):
    Case([1, 4, 2], [70, 33, 200], G, heads, dim, 16, 16, dim + G).check(sv)


@pytest.mark.parametrize("bs,st", [(16, 1), (16, 2), (16, 4), (16, 16), (32, 8), (64, 64), (256, 32), (1024, 64)])
@pytest.mark.parametrize("order", ["tokens", "heads"])
def test_pages_and_groups(sv, bs, st, order):
    Case([3, 1], [bs + 5, 3 * bs if bs < 200 else bs + 40], 4, 2, 64, bs, st, bs + st, order=order).check(sv)


@pytest.mark.parametrize("ctx", [1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 1000])
def test_lengths(sv, ctx):
    c = Case([1, min(ctx, 5)], [ctx, ctx], 4, 1, 64, 16, 16, ctx)
    c.check(sv)
    c.check(sv, sinks=True)


def test_a_request_without_context_or_tokens(sv):
    c = Case([2, 0, 3, 1], [0, 40, 2, 50], 2, 2, 64, 16, 8, 4)
    out, lse = c.check(sv)
    assert not bool(out[:2].any()) and bool((lse[:2] == -math.inf).all())
    assert not bool(out[2].any())  # three new tokens, two of them in the cache
    out, lse = c.check(sv, sinks=True)
    assert torch.equal(lse[0].cpu(), c.sinks) or bool(((lse[0].cpu() - c.sinks).abs() <= 4 * oo.U * c.sinks.abs()).all())


@pytest.mark.parametrize("window", [1, 2, 16, 31, 33, 100, 129, 5000])
@pytest.mark.parametrize("n", [1, 9, 70])
def test_windows(sv, window, n):
    c = Case([n, 1], [300, 299], 4, 1, 64, 32, 32, window + n)
    c.check(sv, window=window, sinks=window % 2 == 1)


def test_many_rows(sv):
    """Blocks of rows of each size, ragged, and more than one of them."""
    for n, G in ((2, 8), (3, 8), (5, 8), (9, 8), (33, 8), (130, 1), (17, 16), (40, 3)):
        Case([n, n // 2 + 1], [n + 77, n + 200], G, 1, 64, 16, 16, n * G).check(sv)
    Case([9, 30], [400, 90], 8, 1, 256, 16, 16, 5).check(sv)


@pytest.mark.parametrize("dim,n,G", [(64, 1, 8), (128, 2, 4), (256, 1, 1), (64, 9, 8)])
def test_long_contexts_in_splits(sv, dim, n, G):
    c = Case([n, 1], [5000, 1203], G, 1, dim, 64, 64, dim + n)
    c.check(sv)
    c.check(sv, sinks=True, window=3000)


def test_peaked_and_flat_scores(sv):
    c = Case([4], [600], 4, 1, 64, 16, 16, 9)
    c.check(sv, scale=4.0)     # weights of single keys near one
    c.check(sv, scale=0.0)     # all equal
    c.check(sv, scale=-0.125)


def test_missing_pages_are_not_seen(sv):
    c = Case([2, 1], [160, 100], 4, 2, 64, 16, 16, 30)
    c.table[0, 0], c.table[0, 3], c.table[1, 2] = -1, 10 ** 6, -5
    c.check(sv)
    c.table[1, :] = -1
    out, lse = c.check(sv)
    assert not bool(out[2].any()) and bool((lse[2] == -math.inf).all())


@pytest.mark.parametrize("st", [1, 2, 16])
def test_what_is_not_seen_never_reaches_the_output(sv, st):
    """NaN codes and scale bytes of 255 behind the context, in front of the
    window, in pages the table does not name, and at later tokens."""
    c = Case([3, 1], [37, 70], 4, 1, 64, 16, st, 40)
    last = int(c.table[0, 2])
    for t in (c.k, c.v):
        t[last, 5:] = 0x7F      # positions 37.. of request 0
    first = int(c.table[1, 0])
    for t in (c.k, c.v):
        t[first] = 0xFF         # request 1: positions 0..15, behind the window
    for t in (c.ks, c.vs):
        t[first] = 255
        if st == 1:
            t[last, :, 5:] = 255
    out, lse = c.call(sv, window=40)
    torch.cuda.synchronize()
    compare(out, lse, *c.want(window=40))
    assert bool(torch.isfinite(out.float()).all())
    # a NaN value of the last token is seen by that token alone, in its dims
    c = Case([3], [37], 4, 1, 64, 16, st, 41)
    c.v[int(c.table[0, 2]), 4, 0, 10] = 0x7F   # position 36
    c.k[int(c.table[0, 2]), 3, 0, 0] = 0xFF    # position 35: tokens 1 and 2 have a NaN score
    out, lse = c.call(sv)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(out[0].float()).all()) and bool(torch.isfinite(lse[0]).all())
    assert bool(torch.isnan(out[1:].float()).all()) and bool(torch.isnan(lse[1:]).all())
    c.k[int(c.table[0, 2]), 3, 0, 0] = 0
    out, lse = c.call(sv)
    torch.cuda.synchronize()
    bad = torch.isnan(out.float()).cpu()
    assert bool(torch.isfinite(lse).all()) and bool(bad[2, :, 10].all()) and int(bad.sum()) == 4


def test_unusable_requests_and_rows_outside(sv):
    c = Case([2, 3, 1, 2], [50, 60, 70, 80], 2, 2, 64, 16, 16, 50)
    q = torch.cat([c.q, c.q[:3]]).cuda()     # three rows behind the last request
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    c.ctx[1], c.ctx[2] = -1, 10 ** 6
    got, lse = c.call(sv, q=q, out=out, max_q=2)
    torch.cuda.synchronize()
    assert got is out and bool((out[8:] == 7.0).all())
    assert bool(torch.isnan(out[2:6].float()).all()) and bool(torch.isnan(lse[2:6]).all())
    assert bool(torch.isfinite(out[:2].float()).all()) and bool(torch.isfinite(out[6:8].float()).all())
    # more new tokens than max_q
    c = Case([2, 5, 1], [50, 60, 2000], 2, 2, 64, 16, 16, 51)
    out, lse = c.call(sv, max_q=3)
    torch.cuda.synchronize()
    o, z, otol, ltol = c.want()
    o[2:7], z[2:7] = np.nan, np.nan
    compare(out, lse, o, z, otol, ltol)


def test_strided_queries_and_no_lse(sv):
    c = Case([3, 2], [90, 41], 4, 2, 80, 16, 16, 60)
    o, z, otol, ltol = c.want()
    for lead in (0, 8, 3):
        wide = torch.zeros(5, 8 + 3, 80 + lead, dtype=torch.bfloat16, device="cuda")
        view = wide[:, 2:10, lead:lead + 80]
        view.copy_(c.q)
        out, lse = c.call(sv, q=view)
        torch.cuda.synchronize()
        compare(out, lse, o, z, otol, ltol)
    again, none = sv.kv_attention(c.q.cuda(), c.cache(sv), c.table.cuda(), c.q_start.cuda(), c.ctx.cuda(), max_q=3)
    torch.cuda.synchronize()
    assert none is None and torch.equal(again, out)


def test_offsets_past_32_bits(sv):
    heads, dim, bs = 4, 256, 1024
    blocks = 2 ** 32 // (heads * dim * bs) + 2
    k = torch.zeros(blocks, bs, heads, dim, dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    sc = torch.full((2, blocks, heads, bs // 64), 120, dtype=torch.uint8, device="cuda")
    rk, rv, _, _ = oo.random_cache(1, bs, heads, dim, 64, 3)
    k[-1], v[-1] = rk[0].cuda(), rv[0].cuda()
    cache = sv.KVCache(k, v, sc[0], sc[1])
    q = (torch.randn(2, heads, dim, generator=torch.Generator().manual_seed(1)) * 2).to(torch.bfloat16)
    table = torch.tensor([[blocks - 1]], dtype=torch.int32)
    out, lse = sv.kv_attention(q.cuda(), cache, table.cuda(), torch.tensor([0, 2], dtype=torch.int32).cuda(),
                               torch.tensor([500], dtype=torch.int32).cuda(), max_q=2, return_lse=True)
    torch.cuda.synchronize()
    s = np.full((1, heads, bs // 64), 120, np.uint8)
    compare(out, lse, *oo.attention(q, rk.numpy(), s, rv.numpy(), s, 64, np.zeros((1, 1), np.int64), [0, 2], [500],
                                    dim ** -0.5))


def test_graph_replays_and_other_streams(sv):
    c = Case([2, 1], [900, 1500], 4, 1, 64, 16, 16, 70)
    cache, table, qs = c.cache(sv), c.table.cuda(), c.q_start.cuda()
    q, ctx = c.q.cuda(), c.ctx.cuda()

    def go(**kw):
        return sv.kv_attention(q, cache, table, qs, ctx, max_q=2, max_ctx=1500, return_lse=True, **kw)
    go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = go()
    for lens in ([900, 1500], [17, 1001], [2, 1]):
        ctx.copy_(torch.tensor(lens, dtype=torch.int32))
        q.copy_(q.flip(0))
        graph.replay()
        e, el = go()
        torch.cuda.synchronize()
        assert torch.equal(out, e) and torch.equal(lse, el)
    side = torch.cuda.Stream()
    s, sl = go(stream=side)
    side.synchronize()
    assert torch.equal(s, e) and torch.equal(sl, el)


def test_a_round_of_speculative_decoding(sv):
    """Expansion, cache write at its slot mapping, attention over the cache,
    verification and log probabilities, all from one call's outputs to the
    next, each against its definition."""
    import workloads
    Hk, G, D, bs, st = 2, 4, 64, 16, 16
    inp = workloads.verify_tiny(seed=5, device=torch.device("cuda"))
    B, K = inp.B, inp.K
    e = workloads.expand_inputs(B=B, K=K, H=64, seed=2, device=torch.device("cuda"), max_offset=200)
    most = int(e.in_positions.max()) + K + 3
    nblk = -(-most // bs)
    table = torch.randperm(B * nblk, generator=torch.Generator().manual_seed(3)).view(B, nblk).int().cuda()
    out = sv.expand(e.in_token_ids, e.in_positions, e.in_start, e.accepted, e.bonus, K, e.mask_id, e.target_hidden,
                    e.mask_hidden, block_table=table, block_size=bs)
    N = out.slot_mapping.numel()
    k, v, ks, vs = oo.random_cache(B * nblk, bs, Hk, D, st, 4)
    cache = sv.KVCache(k.cuda(), v.cuda(), ks.cuda(), vs.cuda())
    g = torch.Generator().manual_seed(6)
    key, val = ((torch.randn(N, Hk, D, generator=g) * 2).to(torch.bfloat16) for _ in range(2))
    before = oo.to_numpy(cache)
    sv.kv_write(cache, key.cuda(), val.cuda(), out.slot_mapping)
    torch.cuda.synchronize()
    slots = out.slot_mapping.cpu()
    assert (slots == -1).any() and (slots >= 0).any()
    oo.kv_write(before[0], before[1], key.double().numpy(), slots.tolist(), st)
    oo.kv_write(before[2], before[3], val.double().numpy(), slots.tolist(), st)
    after = oo.to_numpy(cache)
    assert np.array_equal(after[1], before[1]) and np.array_equal(after[3], before[3])
    assert oo.same_codes(after[0], before[0]) and oo.same_codes(after[2], before[2])
    # the new tokens of the round: the bonus token and the MASK positions
    pos = out.out_positions.cpu()
    new = out.new_token_indices.cpu()
    last = pos[new[:, -1].long()] + 1
    q = (torch.randn(B * K, Hk * G, D, generator=g) * 2).to(torch.bfloat16)
    qs = torch.arange(B + 1, dtype=torch.int32) * K
    o, z = sv.kv_attention(q.cuda(), cache, table, qs.cuda(), last.int().cuda(), max_q=K, return_lse=True)
    torch.cuda.synchronize()
    compare(o, z, *oo.attention(q, after[0], after[1], after[2], after[3], st, table.cpu().numpy(), qs.tolist(),
                                last.tolist(), D ** -0.5))
    acc, tok, _ = sv.verify(inp.target, inp.draft, inp.draft_tokens, inp.temperature, seed=0, step=1)
    r = sv.token_logprobs(inp.target, tok, inp.temperature, top=3)
    torch.cuda.synchronize()
    (lp, ent, ids, _), (tol, etol) = oo.logprobs(inp.target.cpu(), tok.cpu(), inp.temperature.cpu(), 3)
    assert np.all(np.abs(r.logprobs.cpu().double().numpy() - lp) <= tol)
    assert np.array_equal(r.top_ids.cpu().numpy(), ids)
    assert np.array_equal((tok >= 0).sum(1).cpu().numpy(), acc.cpu().numpy() + 1)


# The cut of the work follows the bounds that the caller gives (max_ctx,
# max_q), not the lengths on the device: a bound far above them takes the cut
# of long contexts (equal runs, a head to a wave, large joins) at small sizes.
FAR = 1 << 22


@pytest.mark.parametrize("dim", [64, 80, 128, 256])
@pytest.mark.parametrize("heads,G", [(1, 16), (2, 3), (4, 8), (8, 1), (12, 2)])
def test_runs_of_tiles_and_heads_to_waves(sv, dim, heads, G):
    for st, order in ((16, "tokens"), (1, "tokens"), (16, "heads")):
        c = Case([1, 1, 0, 1], [700, 33, 0, 1100], G, heads, dim, 16, st, dim + heads + st, order=order)
        c.check(sv, max_ctx=FAR, sinks=st == 1)
    c.check(sv, max_ctx=FAR, window=1030)


@pytest.mark.parametrize("dim,n,G", [(64, 9, 8), (64, 40, 4), (128, 30, 4), (256, 20, 3)])
def test_runs_with_several_blocks_of_rows(sv, dim, n, G):
    c = Case([n, n // 3, 1, n], [n + 1500, n, 500, n - 5], G, 2, dim, 32, 32, dim + n)
    c.check(sv, max_ctx=FAR)
    c.check(sv, max_ctx=FAR, sinks=True, window=1030)


@pytest.mark.parametrize("order", ["tokens", "heads"])
def test_long_runs_of_many_heads(sv, order):
    """Fewer runs than the shortest ones would make: with many heads a run
    has more tiles, and a wave's look-up window ends inside it."""
    Case([1, 2, 1], [4100, 37, 3333], 1, 64, 16, 16, 16, 85, order=order).check(sv, max_ctx=FAR)


def test_runs_captured_and_replayed(sv):
    """Two graphs whose calls share one workspace, replayed in turn with the
    program's own calls between them; lengths on the device change."""
    cs = [Case([1, 1], [900, 1300], 8, 2, 64, 16, 16, 86), Case([3, 1], [1100, 200], 4, 4, 128, 16, 1, 87)]
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
            args[i][0].copy_(args[i][0].flip(0))
            graphs[i].replay()
        eager = [go(i) for i in range(2)]
        torch.cuda.synchronize()
        for (o, z), (eo, ez) in zip(outs, eager):
            assert torch.equal(o, eo) and torch.equal(z, ez)


def test_runs_keep_what_is_not_seen_out(sv):
    c = Case([3, 1], [1037, 970], 4, 4, 64, 16, 16, 80)
    last = int(c.table[0, 64])
    for t in (c.k, c.v):
        t[last, 13:] = 0x7F
    c.table[1, 3] = -1
    out, lse = c.check(sv, max_ctx=FAR)
    assert bool(torch.isfinite(out.float()).all()) and bool(torch.isfinite(lse).all())
    c.v[last, 12, 2, 7] = 0x7F   # the last token's value: position 1036
    out, _ = c.call(sv, max_ctx=FAR)
    torch.cuda.synchronize()
    bad = torch.isnan(out.float()).cpu()
    assert bool(bad[2, 8:12, 7].all()) and int(bad.sum()) == 4


def test_runs_with_unusable_and_empty_requests(sv):
    c = Case([1, 2, 0, 1, 1], [400, 300, 10, 0, 900], 4, 4, 64, 16, 16, 81)
    c.ctx[1] = -3
    out, lse = c.call(sv, max_ctx=FAR)
    torch.cuda.synchronize()
    c.ctx[1] = 300
    o, z, otol, ltol = c.want()
    o[1:3], z[1:3] = np.nan, np.nan
    compare(out, lse, o, z, otol, ltol)
    c.ctx[:] = 0
    out, lse = c.check(sv, max_ctx=FAR)
    assert not bool(out.any())


def test_many_requests(sv):
    """Ragged batches of hundreds (in runs) and thousands (a workgroup each)."""
    g = torch.Generator().manual_seed(82)
    for B, most in ((300, 200), (4200, 20)):
        ctx = torch.randint(0, most, (B,), generator=g).tolist()
        lens = [min(int(v), 3) for v in torch.randint(0, 4, (B,), generator=g)]
        Case(lens, ctx, 2, 1, 32, 16, 16, B).check(sv, max_ctx=FAR)


def test_two_streams_at_once(sv):
    a, b = Case([1, 1], [3000, 1700], 8, 2, 64, 16, 16, 83), Case([2, 1], [2500, 4100], 4, 4, 128, 16, 1, 84)
    args = [(c.q.cuda(), c.cache(sv), c.table.cuda(), c.q_start.cuda(), c.ctx.cuda(), c.max_q) for c in (a, b)]
    plain = [sv.kv_attention(*x, max_ctx=FAR, return_lse=True) for x in args]
    torch.cuda.synchronize()  # (the streams below wait for nothing: all inputs are there)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = [sv.kv_attention(*x, max_ctx=FAR, return_lse=True, stream=s) for x, s in zip(args, streams)]
        torch.cuda.synchronize()
        for (o, z), (po, pz) in zip(got, plain):
            assert torch.equal(o, po) and torch.equal(z, pz)


@pytest.mark.parametrize("far", [False, True])
def test_scores_past_the_range_of_fp32(sv, far):
    """Above it: the row is NaN; below it: the key has no weight."""
    c = Case([1, 1], [40, 70], 2, 1, 64, 16, 16, 88)
    c.k[:], c.ks[:] = 0, 127
    one = 0x38  # 1.0
    at = int(c.table[1, 1])  # positions 16..31 of request 1, of which 20 is aligned with q
    c.k[at, 4, 0, :] = one
    c.ks[at] = 247  # 2^120
    c.q[:] = 1.0
    c.q[1, 0, :], c.q[1, 1, :] = 2.0 ** 20, -2.0 ** 20
    out, lse = c.call(sv, max_ctx=FAR if far else c.max_ctx)
    torch.cuda.synchronize()
    assert bool(torch.isnan(out[1, 0]).all()) and bool(torch.isnan(lse[1, 0]))
    assert not bool(torch.isnan(out[0]).any())
    # 69 keys of score 0 and one of no weight
    j = np.array([t for t in range(70) if t != 20])
    v = oo.kv_values(c.v.numpy(), c.vs.numpy(), c.table[1].numpy()[j // 16] * 16 + j % 16, 16)[:, 0]
    want, tol = v.mean(0), np.abs(v.mean(0)) * 2.0 ** -8 + np.abs(v).mean(0) * 80 * oo.U
    assert np.all(np.abs(out[1, 1].cpu().double().numpy() - want) <= tol)
    assert abs(float(lse[1, 1]) - math.log(69)) <= 8 * oo.U * math.log(69)


def test_tables_without_columns_and_batches_of_nothing(sv):
    c = Case([2, 1], [0, 0], 2, 2, 64, 16, 16, 89)
    c.table = torch.empty(2, 0, dtype=torch.int32)
    out, lse = c.call(sv)
    torch.cuda.synchronize()
    assert not bool(out.any()) and bool((lse == -math.inf).all())
    c.ctx[1] = 1  # more than the table holds
    out, _ = c.call(sv, max_ctx=FAR)
    torch.cuda.synchronize()
    assert not bool(out[:2].any()) and bool(torch.isnan(out[2].float()).all())
    cache = c.cache(sv)
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    out, _ = sv.kv_attention(q, cache, torch.empty(0, 3, **i32), torch.zeros(1, **i32), torch.empty(0, **i32), max_q=1)
    assert out.shape == q.shape
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.empty(0, dtype=torch.int64, device="cuda")
    sv.kv_write(cache, none, none, slots)
    assert sv.kv_read(cache, slots)[0].shape == none.shape
    r = sv.token_logprobs(torch.empty(0, 3, 100, device="cuda"), torch.empty(0, 3, **i32), top=2)
    assert r.top_ids.shape == (0, 3, 2)


@pytest.mark.parametrize("far", [False, True])
def test_output_in_place_of_the_queries(sv, far):
    c = Case([3, 40, 1], [900, 70, 1300], 4, 2, 64, 16, 16, 90)
    kw = dict(max_ctx=FAR) if far else {}
    out, _ = c.call(sv, **kw)
    q = c.q.cuda()
    got, _ = c.call(sv, q=q, out=q, **kw)
    torch.cuda.synchronize()
    assert got is q and torch.equal(got, out)


@pytest.mark.parametrize("far", [False, True])
def test_requests_that_share_pages(sv, far):
    """A common prefix: two tables name the same blocks; and one block named
    by several entries of a table."""
    c = Case([1, 2, 1], [800, 640, 330], 4, 2, 128, 16, 16, 91)
    c.table[1, :40] = c.table[0, :40]
    c.table[2, 3:9] = c.table[2, 2]
    c.check(sv, **(dict(max_ctx=FAR) if far else {}))


@pytest.mark.parametrize("dim,st,order", [(64, 16, "tokens"), (64, 1, "tokens"), (80, 4, "tokens"), (128, 16, "tokens"),
                                          (256, 2, "tokens"), (64, 16, "heads")])
@pytest.mark.parametrize("B,heads,G", [(800, 4, 1), (420, 2, 3), (800, 2, 16), (200, 12, 1)])
def test_many_requests_with_heads_to_waves(sv, B, heads, G, dim, st, order):
    """Batches that fill the card: a workgroup takes several heads of a
    request, a wave each; with empty and unusable requests among them."""
    g = torch.Generator().manual_seed(B + dim)
    ctx = torch.randint(0, 90, (B,), generator=g).tolist()
    lens = torch.randint(0, 2, (B,), generator=g).tolist()
    lens[5], ctx[5] = 1, 40
    c = Case(lens, ctx, G, heads, dim, 16, st, B + dim + st, order=order)
    o, z, otol, ltol = c.want(window=50)
    row = int(c.q_start[5])
    c.ctx[5] = -1
    o[row], z[row] = np.nan, np.nan
    out, lse = c.call(sv, window=50, max_ctx=1000)
    torch.cuda.synchronize()
    on = np.arange(int(c.q_start[-1]))
    assert len(on) == out.shape[0]
    compare(out, lse, o, z, otol, ltol)
