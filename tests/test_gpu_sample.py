"""Sampling from cut distributions and the same cut applied to logits, on the
GPU against the 64-bit definition: types, sizes, settings alone and together,
ties, rows at the ends of the range, masked and unusable rows, row tables,
strides, captured and concurrent calls, and a verification of cut rows.

Tokens and kept sets have to be equal: the definition's borders are a double's
step apart from the kernel's (weights are multiples of 2^-45 or finer of the
largest), so that one of the random borders here would have to lie within about
1e-11 of a sum of weights to tell them apart."""
import math

import numpy as np
import pytest
import torch

import decode_oracle as do

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16

SETTINGS = [  # T, k, p, min_p
    (0.7, 50, 0.95, 0.0), (1.0, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.05), (0.6, 20, 1.0, 0.0), (0.0, 0, 1.0, 0.0),
    (0.9, 1000, 0.98, 0.02), (1.0, 0, 1.0, 0.0), (1.5, 3000, 1.0, 0.0), (1.5, 2500, 0.97, 0.001), (0.8, 0, 0.5, 0.3),
    (1.0, 1, 1.0, 0.0), (2.0, 0, 0.999, 0.0)]


@pytest.fixture(scope="module")
def sv():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import rejection_sampling_verify_03_amd as m
    return m


def columns(rows):
    T, k, p, mn = zip(*rows)
    return torch.tensor(T), torch.tensor(k, dtype=torch.int32), torch.tensor(p), torch.tensor(mn)


def cuda(ts):
    return [None if t is None else t.cuda() for t in ts]


def check(sv, x, sets, u=None, seed=0, dev=None):
    """Tokens and cut logits of x [B, R, V] against the definition."""
    B, R, V = x.shape
    if u is None:
        u = torch.rand(B, R, generator=torch.Generator().manual_seed(seed))
    d = x.cuda() if dev is None else dev
    tokens = sv.sample(d, u.cuda(), *cuda(sets))
    out = sv.truncate_logits(d, *cuda(sets))
    torch.cuda.synchronize()
    assert np.array_equal(tokens.cpu().numpy(), do.sample(x, u.tolist(), *sets))
    got, want = out.cpu().double().numpy(), do.truncate(x, *sets)
    assert np.array_equal(got, want, equal_nan=True)
    return tokens, out


def zipf(B, R, V, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    rank = torch.stack([torch.randperm(V, generator=g) for _ in range(B * R)]).view(B, R, V)
    return (-1.1 * torch.log(rank.float() + 1) + 0.3 * torch.randn(B, R, V, generator=g)).to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 63, 64, 65, 500, 1023, 2047, 2048, 2049, 2055, 4096, 8191, 8192, 8193, 16385,
                               32001])
def test_sizes(sv, V, dtype):
    g = torch.Generator().manual_seed(V)
    x = (torch.randn(len(SETTINGS), 2, V, generator=g) * 3).to(dtype)
    check(sv, x, columns(SETTINGS), seed=V + 1)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [40000, 151936, 201088])
def test_vocabularies(sv, V, dtype):
    """Distributions that keep few tokens and tens of thousands."""
    check(sv, zipf(len(SETTINGS), 1, V, dtype, V), columns(SETTINGS), seed=V)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_rows(sv, dtype):
    """More rows than the card has compute units: half of the threads to each."""
    x = zipf(24, 12, 3000, dtype, 3)
    check(sv, x, columns([SETTINGS[b % len(SETTINGS)] for b in range(24)]), seed=4)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [300, 5000, 40000])
def test_ties(sv, V, dtype):
    """Few different values, so that every border falls among equal logits,
    and rows of one value: the lower indices stay."""
    g = torch.Generator().manual_seed(V)
    x = torch.randint(-2, 3, (len(SETTINGS), 1, V), generator=g).to(dtype)
    check(sv, x, columns(SETTINGS), seed=1)
    for value in (0.0, -0.0, 1.5, -3.0, 1e-30, 200.0, -500.0):
        y = torch.full((len(SETTINGS), 1, V), value).to(dtype)
        _, out = check(sv, y, columns(SETTINGS), seed=2)
        k = min(50, V)
        kept = torch.isfinite(out[0, 0].float()).nonzero()[:, 0]
        assert int(kept[-1]) == len(kept) - 1 <= k
    signs = torch.where(torch.rand(len(SETTINGS), 1, V, generator=g) < 0.5, 0.0, -0.0).to(dtype)
    check(sv, signs, columns(SETTINGS), seed=3)  # (both zeros are one value)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_values_at_the_ends_of_the_range(sv, dtype):
    """Logits so small, or so large, that the counted bins hold several of
    them, alone and among ordinary ones; the largest numbers there are."""
    g = torch.Generator().manual_seed(5)
    S = len(SETTINGS)
    small = torch.randn(S, 1, 6000, generator=g) * 2.0 ** -21
    mixed = torch.where(torch.rand(S, 1, 6000, generator=g) < 0.5, small, torch.randn(S, 1, 6000, generator=g))
    large = torch.randn(S, 1, 6000, generator=g) * 300
    deep = -300 - torch.rand(S, 1, 6000, generator=g) * 20
    near = -128 + torch.randn(S, 1, 6000, generator=g)
    subnormal = torch.randn(S, 1, 6000, generator=g) * 1e-39
    for x in (small, mixed, large, deep, near, 128 + small * 2 ** 20, subnormal):
        check(sv, x.to(dtype), columns(SETTINGS), seed=6)
    huge = torch.randn(S, 1, 6000, generator=g).sign() * torch.finfo(dtype).max
    check(sv, huge.to(dtype), columns(SETTINGS), seed=7)
    # temperatures that bring them into range, and the ends of temperatures
    ends = [(T, k, p, mn) for T in (100.0, 1e5, 1e30, 3e38, 1e-3, 2.0 ** -126) for k, p, mn in
            ((0, 1.0, 0.0), (40, 0.9, 0.0), (0, 0.9, 0.01), (3000, 1.0, 0.0))]
    y = (torch.randn(len(ends), 1, 6000, generator=g) * 200).to(dtype)
    check(sv, y, columns(ends), seed=8)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [1500, 30000])
def test_masked_rows(sv, V, dtype):
    """Logits of -inf, and of the type's lowest value, in most places; few, one
    and no finite ones; NaN and +inf."""
    g = torch.Generator().manual_seed(V)
    x = (torch.randn(len(SETTINGS), 8, V, generator=g) * 3).to(dtype)
    x[:, 0, ::2] = -math.inf
    x[:, 1, 5:] = -math.inf
    x[:, 2, :] = -math.inf
    x[:, 2, V - 3] = 2.0
    x[:, 3, :] = -math.inf
    x[:, 4, 7] = math.nan
    x[:, 5, V - 1] = math.inf
    x[:, 6, 10:] = torch.finfo(dtype).min
    x[:, 7, 1] = -math.nan
    check(sv, x, columns(SETTINGS), seed=9)


def test_settings_that_cannot_be_used(sv):
    bad = [(-1.0, 0, 1.0, 0.0), (math.nan, 0, 1.0, 0.0), (math.inf, 0, 1.0, 0.0), (1e-39, 0, 1.0, 0.0), (1.0, -1, 1.0, 0.0),
           (1.0, 0, 0.0, 0.0), (1.0, 0, -0.5, 0.0), (1.0, 0, math.nan, 0.0), (1.0, 0, 1.0, -0.1), (1.0, 0, 1.0, 1.1),
           (1.0, 0, 1.0, math.nan), (0.0, -1, 1.0, 0.0), (1.0, 5, 1.0, 0.0)]
    x = torch.randn(len(bad), 2, 3000, generator=torch.Generator().manual_seed(1))
    tokens, out = check(sv, x, columns(bad))
    assert bool((tokens[:-1] == -1).all()) and bool((tokens[-1] >= 0).all())
    assert bool(torch.isnan(out[:-1]).all())
    u = torch.tensor([[1.0, -0.1, math.nan, 0.5, 2.0, -math.inf, 0.0]])
    t = sv.sample(x[:1, :1].expand(1, 7, 3000).contiguous().cuda(), u.cuda(), torch.ones(1).cuda())
    assert (t.cpu() >= 0).tolist() == [[False, False, False, True, False, False, True]]


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_borders(sv, dtype):
    """The ends of every setting, and uniforms at the ends of [0, 1)."""
    V = 5000
    rows = [(1.0, k, 1.0, 0.0) for k in (1, 2, V - 1, V, V + 1, 2 ** 31 - 1, 2048, 2049)]
    rows += [(1.0, 0, p, 0.0) for p in (1e-38, 1e-30, 0.5, 1 - 2.0 ** -24, 1.0, 2.0, math.inf)]
    rows += [(1.0, 0, 1.0, mn) for mn in (1.0, 1e-38, 0.999, 0.5)] + [(1.0, 300, 1 - 2.0 ** -24, 1e-5)]
    x = (torch.randn(len(rows), 3, V, generator=torch.Generator().manual_seed(2)) * 2).to(dtype)
    u = torch.tensor([[0.0, 1 - 2.0 ** -24, 2.0 ** -40]]).expand(len(rows), 3).contiguous()
    check(sv, x, columns(rows), u=u)


def test_every_uniform_of_a_row(sv):
    """65536 uniforms through one row: the tokens' shares are the kept weights'."""
    n, V = 65536, 300
    x = (torch.randn(1, 1, V, generator=torch.Generator().manual_seed(3)) * 2)
    u = ((torch.arange(n) + 0.5) / n).view(n, 1)
    for s in ((1.0, 0, 1.0, 0.0), (0.8, 30, 0.9, 0.0)):
        sets = columns([s] * n)
        t = sv.sample(x.cuda().expand(n, 1, V), u.cuda(), *cuda(sets))[:, 0].cpu()
        assert bool((t[1:] >= t[:-1]).all())  # (ascending index)
        kept, w = do.cut(x[0, 0].double().numpy(), *s)
        share = np.where(kept, w, 0) / w[kept].sum()
        got = np.bincount(t.numpy(), minlength=V) / n
        assert np.abs(got - share).max() <= 1.001 / n


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [1000, 9001])
def test_rows_by_a_table(sv, V, dtype):
    g = torch.Generator().manual_seed(V)
    x = (torch.randn(40, V, generator=g) * 3).to(dtype)
    B, R = len(SETTINGS), 3
    index = torch.randint(0, 40, (B, R), generator=g).to(torch.int32)
    index[0], index[1, 0], index[2, 1] = 7, -1, 40   # (one row several times, and rows that do not exist)
    u = torch.rand(B, R, generator=g)
    sets = columns(SETTINGS)
    t = sv.sample(x.cuda(), u.cuda(), *cuda(sets), row_index=index.cuda()).cpu().numpy()
    want = do.sample(x[index.clamp(0, 39).long()], u.tolist(), *sets)
    want[1, 0] = want[2, 1] = -1
    assert np.array_equal(t, want)
    none = sv.sample(torch.empty(0, V, dtype=dtype, device="cuda"), u.cuda(), *cuda(sets), row_index=index.cuda())
    assert bool((none == -1).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [1001, 5003])
def test_strides_and_shared_rows(sv, V, dtype):
    """Rows at odd strides and offsets, requests that share rows, in and out."""
    g = torch.Generator().manual_seed(V)
    S = len(SETTINGS)
    wide = (torch.randn(S, 3, V + 13, generator=g) * 3).to(dtype).cuda()
    view = wide[:, :2, 5:5 + V]
    sets = columns(SETTINGS)
    check(sv, view.cpu(), sets, dev=view)
    shared = wide[:1, :2, 1:1 + V].expand(S, 2, V)
    check(sv, shared.cpu(), sets, dev=shared)
    # into a strided output, whose other places stay
    out = torch.full((S, 4, V + 9), 7.0, dtype=dtype, device="cuda")
    got = sv.truncate_logits(view, *cuda(sets), out=out[:, 1:3, 3:3 + V])
    assert np.array_equal(got.cpu().double().numpy(), do.truncate(view.cpu(), *sets), equal_nan=True)
    out[:, 1:3, 3:3 + V] = 7.0
    assert bool((out == 7.0).all())
    # in place
    before = wide.clone()
    sv.truncate_logits(view, *cuda(sets), out=view)
    assert np.array_equal(view.cpu().double().numpy(), do.truncate(before.cpu()[:, :2, 5:5 + V], *sets), equal_nan=True)
    wide[:, :2, 5:5 + V] = before[:, :2, 5:5 + V]
    assert torch.equal(wide, before)


def test_truncating_what_may_not_be(sv):
    x = torch.zeros(2, 3, 100, device="cuda")
    T = torch.ones(2, device="cuda")
    with pytest.raises(ValueError):
        sv.truncate_logits(x, T, out=torch.zeros(2, 3, 99, device="cuda"))
    with pytest.raises(ValueError):
        sv.truncate_logits(x, T, out=torch.zeros(2, 3, 100, device="cuda", dtype=BF16))
    with pytest.raises(sv.SpecError):
        sv.truncate_logits(x, T, out=torch.zeros(1, 3, 100, device="cuda").expand(2, 3, 100))
    shared = torch.zeros(1, 3, 100, device="cuda").expand(2, 3, 100)
    with pytest.raises(sv.SpecError):
        sv.truncate_logits(shared, T, out=shared)
    with pytest.raises(ValueError):
        sv.sample(x, torch.zeros(2, 2, device="cuda"), T)
    with pytest.raises(ValueError):
        sv.sample(x, torch.zeros(2, 3, device="cuda"), T, top_k=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        sv.sample(x, torch.zeros(2, 3, device="cuda"), torch.ones(3, device="cuda"))
    with pytest.raises(sv.SpecError):
        sv.sample(x, torch.zeros(2, 3, device="cuda"), T, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert sv.sample(x[:0], torch.zeros(0, 3, device="cuda"), T[:0]).shape == (0, 3)


def test_without_settings(sv):
    """A temperature alone draws by the inverse distribution function of the
    whole row; a cut that leaves everything is none."""
    x = zipf(3, 2, 20000, BF16, 12)
    T = torch.tensor([1.0, 0.0, 0.5])
    u = torch.rand(3, 2, generator=torch.Generator().manual_seed(1))
    t = sv.sample(x.cuda(), u.cuda(), T.cuda())
    assert np.array_equal(t.cpu().numpy(), do.sample(x, u.tolist(), T))
    d = x.cuda()
    out = sv.truncate_logits(d, T.cuda())
    assert torch.equal(out, d)


def test_replays_of_captured_calls(sv):
    """Two graphs that share a workspace, replayed in turn with the program's
    own calls between them; logits and settings on the device change."""
    sets = cuda(columns(SETTINGS))
    B = len(SETTINGS)
    g = torch.Generator(device="cuda").manual_seed(4)
    xs = [torch.randn(B, 2, V, generator=g, device="cuda").mul_(3).to(BF16) for V in (9000, 1200)]
    u = torch.rand(B, 2, generator=g, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")

    def go(i, **kw):
        return sv.sample(xs[i], u, *sets, **kw), sv.truncate_logits(xs[i], *sets, **kw)
    for i in range(2):
        go(i, workspace=ws)
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph() for _ in xs], []
    for i, graph in enumerate(graphs):
        with torch.cuda.graph(graph):
            outs.append(go(i, workspace=ws))
    for _ in range(4):
        for i in range(2):
            xs[i].copy_(torch.randn(xs[i].shape, generator=g, device="cuda") * 3)
            u.copy_(torch.rand(u.shape, generator=g, device="cuda"))
            sets[0].copy_(sets[0].roll(1))
            sets[1].copy_(sets[1].roll(1))
            graphs[i].replay()
            want = go(i)
            torch.cuda.synchronize()
            assert torch.equal(outs[i][0], want[0]) and torch.equal(outs[i][1], want[1])


def test_two_streams_at_once(sv):
    sets = cuda(columns(SETTINGS))
    B = len(SETTINGS)
    xs = [zipf(B, 2, V, BF16, V).cuda() for V in (30000, 20001)]
    u = torch.rand(B, 2, device="cuda")
    want = [(sv.sample(x, u, *sets), sv.truncate_logits(x, *sets)) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        got = [(sv.sample(x, u, *sets, stream=s), sv.truncate_logits(x, *sets, stream=s)) for x, s in zip(xs, streams)]
        for s in streams:
            s.synchronize()
        for (a, b), (c, d) in zip(got, want):
            assert torch.equal(a, c) and torch.equal(b, d)


def test_offsets_past_32_bits(sv):
    """A row that begins more than 2^32 bytes behind the first."""
    V, stride = 3000, 1 << 30
    buf = torch.zeros(3 * stride + V, dtype=BF16, device="cuda")
    x = zipf(1, 4, V, BF16, 9)
    view = buf.as_strided((1, 4, V), (4 * stride, stride, 1))
    view.copy_(x)
    check(sv, x, columns([(0.8, 40, 0.9, 0.0)]), dev=view)
    sv.truncate_logits(view, torch.tensor([0.8]).cuda(), torch.tensor([40], dtype=torch.int32).cuda(), out=view)
    assert np.array_equal(view.cpu().double().numpy(), do.truncate(x, torch.tensor([0.8]), torch.tensor([40])))


def test_a_long_vocabulary(sv):
    """Ranges of indices wider than a range of the search, and rows whose
    equal logits are more than any list."""
    V = 2 ** 22 + 12345
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(1, 2, V, generator=g, device="cuda").to(BF16)
    x[0, 1] = x[0, 1].round()
    for s in ((1.0, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.0), (1.0, 100000, 1.0, 0.0), (1.0, 100, 0.5, 0.0)):
        check(sv, x.cpu(), columns([s]), dev=x, seed=V)
    y = x[:, :1].float()
    for s in ((1.0, 0, 0.9, 0.0), (1.0, 100000, 0.9, 0.0)):
        check(sv, y.cpu(), columns([s]), dev=y, seed=V)


def shared_rows_of(dtype):
    """The shortest odd vocabulary of which few rows are shared out to several workgroups each."""
    return 262144 // dtype.itemsize + 5


@pytest.mark.parametrize("kind", ["ties", "equal", "signs", "small", "mixed", "large", "deep", "masked", "lowest", "few"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_shared_by_workgroups(sv, dtype, kind):
    """What the counted bins hold several values of, borders among equal logits
    of many parts, masked parts: rows that several workgroups share."""
    V, S = shared_rows_of(dtype), len(SETTINGS)
    g = torch.Generator().manual_seed(V)
    x = torch.randn(S, 1, V, generator=g)
    if kind == "ties":
        x = torch.randint(-2, 3, (S, 1, V), generator=g).float()
    elif kind == "equal":
        x[:] = torch.tensor([0.0, 1.5, -3.0, 1e-30, 200.0, -500.0]).repeat(S // 6).view(S, 1, 1)
    elif kind == "signs":
        x = torch.where(x < 0, 0.0, -0.0)
    elif kind == "small":
        x = x * 2.0 ** -21
    elif kind == "mixed":
        x = torch.where(torch.rand(S, 1, V, generator=g) < 0.5, x, x * 2.0 ** -21)
    elif kind == "large":
        x = x * 300
    elif kind == "deep":
        x = -300 - x.abs() * 20
    elif kind == "masked":
        x[:, :, : V - 3000] = -math.inf
        x[1::3, :, 17] = math.nan
        x[2::3, :, V - 1] = math.inf
    elif kind == "lowest":
        x[:, :, 10:] = torch.finfo(dtype).min
    elif kind == "few":
        x[:, :, 1:] = -math.inf
    check(sv, x.to(dtype), columns(SETTINGS), seed=11)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows", [1, 63, 64, 65])
def test_as_many_rows_as_are_shared(sv, rows, dtype):
    """The same rows of the same settings, in a call of as many as are shared
    out and of one more, at the ends of the parts and of the uniforms."""
    V = shared_rows_of(dtype)
    x = zipf(1, 1, V, dtype, 3).cuda()
    sets = [t[torch.arange(rows) % len(SETTINGS)] for t in columns(SETTINGS)]
    u = torch.linspace(0, 1, rows + 1)[:-1].view(rows, 1)
    want = do.sample(x.cpu().expand(rows, 1, V), u.tolist(), *sets)
    ws = torch.full((sv.spec_sample_workspace_bytes(rows, 1, V),), 255, dtype=torch.uint8, device="cuda")
    got = sv.sample(x.expand(rows, 1, V), u.cuda(), *cuda(sets), workspace=ws)
    assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_shared_rows_by_a_table_and_in_place(sv, dtype):
    """Rows at odd strides and offsets through a table, one several times and
    some that do not exist; cut where they stand, on two streams at once."""
    V, S = shared_rows_of(dtype), len(SETTINGS)
    buf = zipf(1, 7, V + 3, dtype, 5)[0].cuda()
    x = buf[:, 1:V + 1]
    index = (torch.arange(S * 2).view(S, 2) % 7).to(torch.int32)
    index[3, 0], index[4, 1], index[5] = -1, 7, 2
    u = torch.rand(S, 2, generator=torch.Generator().manual_seed(6))
    sets = columns(SETTINGS)
    got = sv.sample(x, u.cuda(), *cuda(sets), row_index=index.cuda()).cpu().numpy()
    want = do.sample(x.cpu()[index.clamp(0, 6).long()], u.tolist(), *sets)
    want[3, 0] = want[4, 1] = -1
    assert np.array_equal(got, want)
    rows = [x[:1].expand(S, V).unsqueeze(1).clone(), x[1:2].expand(S, V).unsqueeze(1).clone()]
    cut = [do.truncate(r.cpu(), *sets) for r in rows]
    dev, streams = cuda(sets), [torch.cuda.Stream() for _ in rows]
    torch.cuda.synchronize()
    for r, st in zip(rows, streams):
        assert sv.truncate_logits(r, *dev, out=r, stream=st) is r
    torch.cuda.synchronize()
    for r, w in zip(rows, cut):
        assert np.array_equal(r.cpu().double().numpy(), w, equal_nan=True)


@pytest.mark.parametrize("rows", [1, 65])
def test_the_longest_vocabulary(sv, rows):
    """A row of the largest size, alone (shared by workgroups) and read by 65
    requests (a workgroup each): equal logits, of which the n-th token is the
    one at u n, and few finite ones at its ends."""
    V = sv.SPEC_MAX_V
    x = torch.zeros(1, V, dtype=BF16, device="cuda")
    index = torch.zeros(rows, 1, dtype=torch.int32, device="cuda")
    k = torch.full((rows,), V // 4 + 1, dtype=torch.int32, device="cuda")
    T, p = torch.ones(rows, device="cuda"), torch.full((rows,), 0.5, device="cuda")
    u = torch.tensor([1023 / 1024, 0.0, 0.25, 0.5]).repeat(17)[:rows].view(rows, 1)
    for kw, n in (({}, V), ({"top_k": k}, V // 4 + 1), ({"top_p": p}, V // 2)):
        t = sv.sample(x, u.cuda(), T, row_index=index, **kw)[:, 0].cpu()
        assert t.tolist() == [int(float(v) * n) for v in u[:, 0]]
    x.fill_(-math.inf)
    at = torch.tensor([0, 5, 1 << 30, V - 9, V - 2, V - 1])
    few = torch.tensor([[[0.5, 1.0, 2.0, 1.0, 1.5, 1.0]]]).to(BF16)
    x[0, at.cuda()] = few[0, 0].cuda()
    for s in ((1.0, 0, 1.0, 0.0), (1.0, 3, 1.0, 0.0), (0.7, 0, 0.95, 0.0), (1.0, 0, 1.0, 0.3), (0.0, 0, 1.0, 0.0)):
        sets = columns([s] * rows)
        t = sv.sample(x, u.cuda(), *cuda(sets), row_index=index)[:, 0].cpu().numpy()
        assert np.array_equal(t, at.numpy()[do.sample(few.expand(rows, 1, 6), u.tolist(), *sets)[:, 0]])


def test_replays_of_rows_shared_by_workgroups(sv):
    """Two graphs on one workspace, replayed in turn."""
    sets = cuda(columns(SETTINGS))
    B = len(SETTINGS)
    g = torch.Generator(device="cuda").manual_seed(4)
    xs = [torch.randn(B, 1, shared_rows_of(t), generator=g, device="cuda").to(t) for t in (BF16, F32)]
    u = torch.rand(B, 1, generator=g, device="cuda")
    ws = torch.empty(max(sv.spec_sample_workspace_bytes(*x.shape) for x in xs), dtype=torch.uint8, device="cuda")

    def go(i, **kw):
        return sv.sample(xs[i], u, *sets, **kw), sv.truncate_logits(xs[i], *sets, **kw)
    for i in range(2):
        go(i, workspace=ws)
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph() for _ in xs], []
    for i, graph in enumerate(graphs):
        with torch.cuda.graph(graph):
            outs.append(go(i, workspace=ws))
    for _ in range(4):
        for i in range(2):
            xs[i].copy_(torch.randn(xs[i].shape, generator=g, device="cuda") * 2)
            u.copy_(torch.rand(u.shape, generator=g, device="cuda"))
            sets[0].copy_(sets[0].roll(1))
            graphs[i].replay()
            want = go(i)
            torch.cuda.synchronize()
            assert torch.equal(outs[i][0], want[0]) and torch.equal(outs[i][1], want[1])


def test_drafts_and_targets_cut_alike(sv):
    """A round of speculative decoding with cut distributions: the drafter's
    rows cut, drafts sampled from them, and the verification of those drafts
    over cut target and draft rows, equal to the reference implementation's on
    the same rows; every emitted token is a kept one."""
    import oracle
    B, K, V = 6, 4, 2000
    sets = columns([(0.7, 50, 0.95, 0.0), (1.0, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.05), (0.6, 20, 1.0, 0.0), (0.0, 0, 1.0, 0.0),
                    (0.9, 100, 0.98, 0.02)])
    g = torch.Generator().manual_seed(8)
    target = (torch.randn(B, K + 1, V, generator=g) * 3).to(BF16)
    draft = (target[:, :K].float() + 0.5 * torch.randn(B, K, V, generator=g)).to(BF16)
    d = cuda(sets)
    u = torch.rand(B, K, generator=g)
    tokens = sv.sample(draft.cuda(), u.cuda(), *d)
    assert np.array_equal(tokens.cpu().numpy(), do.sample(draft, u.tolist(), *sets))
    q, p = sv.truncate_logits(draft.cuda(), *d), sv.truncate_logits(target.cuda(), *d)
    acc, tok, _ = sv.verify(p, q, tokens, d[0], seed=3, step=1)
    torch.cuda.synchronize()
    ref = oracle.verify(p.cpu().view(torch.int16).numpy().view(np.uint16), q.cpu().view(torch.int16).numpy().view(np.uint16),
                        tokens.cpu().numpy(), sets[0].numpy(), seed=3, step=1)
    assert np.array_equal(acc.cpu().numpy(), ref.accepted) and np.array_equal(tok.cpu().numpy(), ref.tokens)
    assert bool((acc >= 0).all())
    kept = torch.isfinite(p.float())
    for b in range(B):
        for r in range(int(acc[b]) + 1):
            assert bool(kept[b, r, int(tok[b, r])]) or float(sets[0][b]) == 0
    # a request whose settings cannot be used is reported
    d[2][1] = math.nan
    acc, tok, _ = sv.verify(sv.truncate_logits(target.cuda(), *d), q, tokens, d[0], seed=3, step=1)
    assert int(acc[1]) == -1 and int((acc >= 0).sum()) == B - 1
