"""Truncation between rows that lie among each other in one buffer, and of rows
into a part of themselves, which is refused."""
import pytest
import torch

import decode_oracle as do

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import rejection_sampling_verify_03_amd as m
    return m


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,R,V", [(3, 2, 333), (1, 4, 5000), (4, 1, 2048)])
def test_views_of_one_buffer(sv, B, R, V, dtype):
    g = torch.Generator().manual_seed(V)
    T = torch.tensor([0.7, 1.0, 0.0, 1.3])[:B]
    cut = dict(top_k=torch.tensor([20, 0, 3, 0], dtype=torch.int32)[:B], top_p=torch.tensor([1.0, 0.8, 1.0, 0.95])[:B])
    dcut = {n: t.cuda() for n, t in cut.items()}
    for shape, of in (((B, 2, R, V), lambda t, i: t[:, i]), ((B, R, 2, V), lambda t, i: t[:, :, i]),
                      ((2, B, R, V), lambda t, i: t[i])):
        buf = (3 * torch.randn(shape, generator=g)).to(dtype).cuda()
        before = buf.clone()
        x, out = of(buf, 0), of(buf, 1)
        assert sv.truncate_logits(x, T.cuda(), out=out, **dcut) is out
        torch.cuda.synchronize()
        assert torch.equal(x, of(before, 0))
        want = do.truncate(x.cpu(), T, cut["top_k"], cut["top_p"])
        assert torch.equal(out.cpu().double(), torch.from_numpy(want))
    wide = torch.zeros(B, R, V + 8, dtype=dtype, device="cuda")
    with pytest.raises(sv.SpecError):
        sv.truncate_logits(wide[..., :V], T.cuda(), out=wide[..., 8:], **dcut)
    with pytest.raises(sv.SpecError):
        sv.truncate_logits(wide[..., 1:V + 1], T.cuda(), out=wide[..., :V], **dcut)
