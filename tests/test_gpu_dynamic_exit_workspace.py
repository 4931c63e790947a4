"""The dynamic early exit on a workspace whose memory comes back as an earlier
launch found it: leftover records must never pass for this launch's."""
import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import rejection_sampling_verify_03_amd as m
    return m


B, K, V = 192, 8, 151936


def batch(name, seed):
    return workloads.mixture_inputs(name, B, K, V, torch.bfloat16, seed, torch.device("cuda"), temps=(0.0, 0.6, 1.0),
                                    lam_lo=0.05, lam_hi=0.5)


@pytest.mark.parametrize("counter", [0, 7, 0x40297C9488840000])
def test_records_of_an_earlier_launch_at_the_same_counter(sv, counter):
    """A workspace freed and allocated again at the same address: what stood in
    front of its records is zero (or back to what it was), its launch counter
    is the one that an earlier launch on other inputs ran at, and that
    launch's records still stand."""
    old, new = batch("dyn again, old", 83), batch("dyn again, new", 84)
    a1, t1, _ = sv.verify(new.target, new.draft, new.draft_tokens, new.temperature, seed=4, step=9)
    n = sv.spec_verify_workspace_bytes(B, K, V)
    chunks = 5  # of a row of 151936 logits; a record is 64 bytes, the records are the workspace's end
    head = n - B * (2 * K + 1) * chunks * 64
    assert head > 0
    for trial in range(3):
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        ws[8:16].view(torch.int64).fill_(counter)
        before = ws.clone()
        sv.verify(old.target, old.draft, old.draft_tokens, old.temperature, seed=1, step=3, workspace=ws,
                  phase_starts=sv.SPEC_PHASES_DYNAMIC)
        torch.cuda.synchronize()
        assert bool(ws[head:].any()) and int(ws[8:16].view(torch.int64)) == counter + 1
        ws[:head] = before[:head]
        a2, t2, _ = sv.verify(new.target, new.draft, new.draft_tokens, new.temperature, seed=4, step=9, workspace=ws,
                              phase_starts=sv.SPEC_PHASES_DYNAMIC)
        torch.cuda.synchronize()
        assert bool((a2 >= 0).all()), (trial, int((a2 < 0).sum()))
        assert torch.equal(a1, a2) and torch.equal(t1, t2), trial


def test_replays_and_eager_launches_on_one_workspace(sv):
    """A captured dynamic exit and eager ones in turn, on one workspace and new
    inputs each time, equal to one pass."""
    ins = [batch("dyn mixed %d" % i, 90 + i) for i in range(3)]
    want = [sv.verify(i.target, i.draft, i.draft_tokens, i.temperature, seed=8, step=2)[:2] for i in ins]
    tgt, dft, x, T = (t.clone() for t in (ins[0].target, ins[0].draft, ins[0].draft_tokens, ins[0].temperature))
    acc = torch.empty(B, dtype=torch.int32, device="cuda")
    tok = torch.empty(B, K + 1, dtype=torch.int32, device="cuda")
    ws = sv.make_workspace(B, K, V, torch.device("cuda"))
    a = sv.verify_args(tgt, dft, x, T, acc, tok, None, ws, seed=8, step=2, phase_starts=sv.SPEC_PHASES_DYNAMIC)
    assert sv.spec_verify_launch(a, torch.cuda.current_stream().cuda_stream) == sv.SPEC_OK
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert sv.spec_verify_launch(a, torch.cuda.current_stream().cuda_stream) == sv.SPEC_OK
    for rep in range(9):
        i = ins[rep % 3]
        for d, s in ((tgt, i.target), (dft, i.draft), (x, i.draft_tokens), (T, i.temperature)):
            d.copy_(s)
        acc.fill_(-5)
        if rep % 2:
            assert sv.spec_verify_launch(a, torch.cuda.current_stream().cuda_stream) == sv.SPEC_OK
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(acc, want[rep % 3][0]) and torch.equal(tok, want[rep % 3][1]), rep
