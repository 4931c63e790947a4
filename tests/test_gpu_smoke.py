"""The smoke run's comparison of the 4-bit cache: a scale one off under the right
codes does not pass it."""
import os
import sys

import pytest
import torch

import decode_oracle as do

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("change", [None, "one off", "another place"])
def test_scales_are_compared(monkeypatch, change):
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    sys.path.insert(0, ROOT)
    import __graft_entry__ as entry
    write = do.kv_write

    def planted(codes, scales, x, slots):  # the mistake is the definition's
        write(codes, scales, x, slots)
        if change == "one off":
            scales[scales > 0] += 1
        else:
            scales[:] = scales[..., ::-1].copy()
    if change is None:
        return entry.smoke()
    monkeypatch.setattr(do, "kv_write", planted)
    with pytest.raises(AssertionError, match="4-bit scales"):
        entry.smoke()
