"""Token log probabilities on the GPU against the 64-bit definition: types,
sizes around the segment and cell boundaries, alignments, masks, ties, rows
without a token and rows that cannot be used."""
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


def check(sv, logits, tokens, temperature, top, dev_logits=None):
    """One call against the definition; returns it."""
    (lp, ent, ids, tlp), (tol, etol) = oo.logprobs(logits, tokens, temperature, top)
    r = sv.token_logprobs(logits.cuda() if dev_logits is None else dev_logits, tokens.cuda(),
                          None if temperature is None else temperature.cuda(), top=top)
    torch.cuda.synchronize()
    got = r.logprobs.cpu().double().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(lp)) and np.array_equal(np.isinf(got), np.isinf(lp))
    fin = np.isfinite(lp)
    assert np.all(np.abs(got - lp)[fin] <= tol[fin]), np.max((np.abs(got - lp) - tol)[fin])
    got = r.entropy.cpu().double().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ent))
    fin = np.isfinite(ent)
    assert np.all(np.abs(got - ent)[fin] <= etol[fin]), np.max((np.abs(got - ent) - etol)[fin])
    assert np.array_equal(r.top_ids.cpu().numpy(), ids)
    got = r.top_logprobs.cpu().double().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(tlp)) and np.array_equal(np.isinf(got), np.isinf(tlp))
    fin = np.isfinite(tlp)
    wide = np.broadcast_to(tol[..., None], tlp.shape)
    assert np.all(np.abs(got - tlp)[fin] <= (wide + 2 * np.abs(np.where(fin, tlp, 0)) * oo.U)[fin])
    return r


def make(B, R, V, dtype, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    logits = (torch.randn(B, R, V, generator=g) * spread).to(dtype)
    tokens = torch.randint(0, V, (B, R), generator=g).to(torch.int32)
    temperature = torch.rand(B, generator=g) + 0.5
    temperature[::3] = 0.0
    return logits, tokens, temperature


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,R,V,top", [
    (1, 1, 1, 1), (1, 1, 7, 32), (2, 3, 63, 5), (1, 2, 64, 32), (3, 1, 65, 3), (2, 2, 1000, 20), (1, 5, 4095, 1),
    (2, 1, 4096, 32), (1, 2, 4097, 7), (3, 2, 32001, 20), (1, 1, 40000, 0), (2, 9, 151936, 5), (1, 2, 201088, 32)])
def test_shapes(sv, B, R, V, top, dtype):
    check(sv, *make(B, R, V, dtype, B * 7 + R * 11 + V), top)


@pytest.mark.parametrize("V,top", [(262144, 5), (262145, 20), (300001, 32), (1 << 20, 20)])
def test_vocabularies_past_one_window_of_cells(sv, V, top):
    check(sv, *make(1, 2, V, torch.bfloat16, V % 1000), top)
    x = torch.full((1, 1, V), -4.0)
    x[0, 0, ::64] = 3.0  # more cells of equal maxima than a list holds
    x[0, 0, V - 1] = 5.0
    check(sv, x, torch.tensor([[V - 1]], dtype=torch.int32), None, top)


def test_many_rows(sv):
    check(sv, *make(700, 5, 130, torch.float32, 6), 3)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_without_tokens_and_unusable_rows(sv, dtype):
    logits, tokens, temperature = make(12, 3, 5000, dtype, 5)
    tokens[0] = -1
    tokens[1, 1:] = -1
    tokens[2, 0], tokens[2, 1] = 5000, -2
    temperature[3], temperature[4], temperature[5], temperature[6] = -1.0, math.nan, math.inf, 1e-40
    logits[7, 0, 4999] = math.nan
    logits[7, 1, 17] = math.inf
    logits[7, 2] = -math.inf
    logits[8, 0] = -math.inf
    logits[8, 0, 4321] = math.nan  # in a segment with nothing else
    logits[9, 0, int(tokens[9, 0])] = -math.inf
    logits[10, 1] = -math.inf
    logits[10, 1, 77] = 3.0
    logits[11, 2] = torch.finfo(dtype).min
    logits[11, 2, 100:103] = 1.0
    check(sv, logits, tokens, temperature, 20)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["equal", "ascending", "descending", "stripe", "plateau", "zeros", "allowed"])
def test_alternatives_of_ties_and_orders(sv, dtype, kind):
    V = 9000
    g = torch.Generator().manual_seed(3)
    if kind == "equal":
        x = torch.full((V,), 2.5)
    elif kind == "ascending":
        x = torch.linspace(-5, 5, V)
    elif kind == "descending":
        x = torch.linspace(5, -5, V)
    elif kind == "stripe":  # the large ones all in cells of one residue
        x = torch.randn(V, generator=g)
        x[(torch.arange(V) // 64) % 64 == 3] += 50
    elif kind == "plateau":
        x = torch.randn(V, generator=g).clamp(max=0.5)
    elif kind == "zeros":  # +0 and -0 are equal
        x = torch.where(torch.rand(V, generator=g) < 0.5, 0.0, -0.0)
    else:  # few allowed tokens, the rest masked
        x = torch.full((V,), -math.inf)
        x[5000:5011] = torch.randn(11, generator=g)
    logits = x.to(dtype).view(1, 1, V)
    tokens = torch.tensor([[5003]], dtype=torch.int32)
    for top in (1, 20, 32):
        check(sv, logits, tokens, None, top)


def test_many_large_logits_in_few_cells(sv):
    """More candidates than a wave's list holds, so that the threshold moves."""
    V = 64 * 64 * 8
    g = torch.Generator().manual_seed(9)
    x = torch.randn(V, generator=g)
    cell = torch.arange(V) // 64
    x[cell % 64 < 10] += 30 + torch.rand(int((cell % 64 < 10).sum()), generator=g) * 5
    check(sv, x.view(1, 1, V), torch.tensor([[1]], dtype=torch.int32), None, 32)


@pytest.mark.parametrize("T", [1.1754944e-38, 1e-20, 1e-3, 1e3, 3e38])
def test_extreme_temperatures(sv, T):
    logits, tokens, _ = make(1, 4, 3001, torch.float32, 21)
    tokens[0, 0] = int(logits[0, 0].argmax())
    tokens[0, 1] = int(logits[0, 1].argmax())
    check(sv, logits, tokens, torch.tensor([T]), 3)


def test_a_nearly_certain_token(sv):
    x = torch.full((1, 3, 20000), -20.0)
    for r, gap in enumerate((5.0, 20.0, 40.0)):
        x[0, r, 123] = -20.0 + gap
    check(sv, x, torch.full((1, 3), 123, dtype=torch.int32), None, 2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strided_and_shared_rows(sv, dtype):
    logits, tokens, temperature = make(3, 4, 1501, dtype, 8)
    wide = torch.full((3, 6, 1600), math.nan, dtype=dtype, device="cuda")
    wide[:, 1:5, 3:1504] = logits.cuda()
    check(sv, logits, tokens, temperature, 5, wide[:, 1:5, 3:1504])
    shared = logits[:1].cuda().expand(3, 4, 1501)
    check(sv, logits[:1].expand(3, 4, 1501).contiguous(), tokens, temperature, 5, shared)


def test_outputs_of_a_verification(sv):
    """The tokens a verification emitted, with the rows it read."""
    import workloads
    inp = workloads.verify_tiny(seed=3, device=torch.device("cuda"))
    _, tok, _ = sv.verify(inp.target, inp.draft, inp.draft_tokens, inp.temperature, seed=1, step=2)
    torch.cuda.synchronize()
    assert (tok == -1).any()
    check(sv, inp.target.cpu(), tok.cpu(), inp.temperature.cpu(), 4, inp.target)


def test_without_entropy_and_with_given_outputs(sv):
    logits, tokens, temperature = make(2, 3, 700, torch.float32, 2)
    full = check(sv, logits, tokens, temperature, 3)
    out = sv.token_logprobs_outputs(2, 3, 0, "cuda", entropy=False)
    r = sv.token_logprobs(logits.cuda(), tokens.cuda(), temperature.cuda(), top=0, out=out)
    torch.cuda.synchronize()
    assert r is out and r.entropy is None and torch.equal(r.logprobs, full.logprobs)


def test_graph_replays_and_other_streams(sv):
    logits, tokens, temperature = make(2, 3, 30000, torch.bfloat16, 13)
    lg, tk, tp = logits.cuda(), tokens.cuda(), temperature.cuda()
    sv.token_logprobs(lg, tk, tp, top=8)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = sv.token_logprobs(lg, tk, tp, top=8)
    for seed in (14, 15, 16):
        fresh, _, _ = make(2, 3, 30000, torch.bfloat16, seed)
        lg.copy_(fresh)
        graph.replay()
        eager = sv.token_logprobs(lg, tk, tp, top=8)
        torch.cuda.synchronize()
        for name in ("logprobs", "entropy", "top_ids", "top_logprobs"):
            assert torch.equal(getattr(r, name), getattr(eager, name)), name
    side = torch.cuda.Stream()
    other = sv.token_logprobs(lg, tk, tp, top=8, stream=side)
    side.synchronize()
    assert torch.equal(other.top_ids, eager.top_ids) and torch.equal(other.logprobs, eager.logprobs)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [8, 9, 15, 63, 66, 71, 4097, 4103, 5003, 32765, 70001, 262139])
def test_alternatives_at_the_end_of_a_row(sv, V, dtype):
    """The last logits, whose loads reach back over the row's end, lead; then
    the same with the row's ends -inf, and with equal ones."""
    for top in (1, 5, 20, 32):
        x, tokens, _ = make(2, 2, V, dtype, V + top)
        last = min(V, 40)
        x[:, 0, V - last:] = 20.0 + torch.randperm(last, generator=torch.Generator().manual_seed(V)).to(dtype) / 4
        x[:, 1, V - last:] = 20.0
        x[1, 1, V - last // 2:] = -math.inf
        tokens[1, 1] = V - last // 2 - 1
        check(sv, x, tokens, None, top)


def test_more_candidates_than_a_list(sv):
    """Equal logits in 60 to 70 cells, and 250 to 260 of them in few cells."""
    for cells in (60, 64, 65, 70):
        x = torch.randn(1, 1, 40000, generator=torch.Generator().manual_seed(cells)).to(torch.bfloat16)
        x[0, 0, 37:37 + 64 * 8 * cells:64 * 8] = 9.0
        check(sv, x, torch.tensor([[37]], dtype=torch.int32), None, 32)
    for equal in (250, 256, 257, 260):
        x = torch.randn(1, 1, 40000, generator=torch.Generator().manual_seed(equal)).to(torch.bfloat16)
        x[0, 0, 1001:1001 + equal] = 9.0
        check(sv, x, torch.tensor([[1001]], dtype=torch.int32), None, 32)
