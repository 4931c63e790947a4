"""The HBM traffic that the benchmark reports comes from committed counters,
and only while the row pass is the code that they were taken on (CPU only)."""
import pytest

import bench


@pytest.mark.parametrize("phase_starts", [0, 1, 8])
def test_committed_counters_are_the_row_pass_s(phase_starts):
    """Code that the row pass does not run has no place in its sources: it
    would set the committed counters aside."""
    measured, prov = bench.measured_traffic(phase_starts)
    assert prov["matches_sources"] and measured > 0, prov
