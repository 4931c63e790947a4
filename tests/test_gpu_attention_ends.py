"""Attention over the 8-bit paged cache on the GPU at the ends of what it
takes: sinks without bound."""
import math

import pytest
import torch

from test_gpu_attention import FAR, Case, compare, sv  # noqa: F401  (sv: the fixture)

pytestmark = pytest.mark.gpu

FMAX = torch.finfo(torch.float32).max


@pytest.mark.parametrize("far", [False, True])
def test_sinks_without_bound(sv, far):  # noqa: F811
    """A sink far below every score leaves the row as it is without one; far
    above, it takes all the weight.  A row that sees nothing has the sink as
    its lse, whichever it is (FAR: in runs, the first request in two or more)."""
    kw = dict(max_ctx=FAR) if far else {}
    low, high = [-math.inf, -FMAX, -2.5e38, -1e30], [math.inf, FMAX, 2.5e38, 1e30]
    c = Case([2, 3, 1], [1700, 2, 0], 8, 1, 64, 16, 16, 92)  # (one of the three tokens over two sees nothing)
    c.sinks = torch.tensor(low + high)
    out, lse = c.call(sv, sinks=True, **kw)
    torch.cuda.synchronize()
    o, z, otol, ltol = c.want()
    nothing = [2, 5]
    for row in range(6):
        for h in range(8):
            if h >= 4 or row in nothing:
                o[row, h], z[row, h] = 0.0, float(c.sinks[h])
                otol[row, h], ltol[row, h] = 0.0, 0.0
    compare(out, lse, o, z, otol, ltol)
    assert torch.equal(lse[nothing].cpu(), c.sinks.expand(2, 8))
    assert torch.equal(lse[:, 4:].cpu(), c.sinks[4:].expand(6, 4)) and not bool(out[:, 4:].any())
