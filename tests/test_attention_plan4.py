"""How an attention over the 4-bit cache is cut into workgroups, on the CPU: as
over the 8-bit one but for how many workgroups the card holds at once."""
import os
import shutil
import subprocess

import pytest

from attention_cases import CASES
from decode_oracle import MANY_SHORT

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "rejection_sampling_verify_03_amd", "csrc")

PROGRAM = """
#include <stdio.h>
#include "attention_plan.hpp"
int main() {
  int B, G, heads, dim, max_q, max_ctx, window, in, four;
  while (scanf("%d %d %d %d %d %d %d %d %d", &B, &G, &heads, &dim, &max_q, &max_ctx, &window, &in, &four) == 9) {
    const specv::AttnPlan p = specv::plan_attn(B, G, heads, dim, max_q, max_ctx, window, in, four);
    printf("%d %d %d %d\\n", p.rt, p.nrb, p.chunks, p.hw);
  }
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("plan4")
    (d / "p.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", CSRC, str(d / "p.cpp"), "-o", str(d / "p")],
                   check=True)

    def run(four, B, G, heads, dim, max_q, max_ctx, window=0, heads_in=False):
        """(rt, nrb, chunks, hw)"""
        line = " ".join(str(int(v)) for v in (B, G, heads, dim, max_q, max_ctx, window, heads_in, four))
        out = subprocess.run([str(d / "p")], input=line, check=True, capture_output=True, text=True).stdout.split()
        return tuple(map(int, out))
    return run


@pytest.mark.parametrize("dim,rows,four,eight", [(64, 16, 4, 3), (64, 17, 3, 3), (64, 33, 2, 2), (128, 16, 3, 2),
                                                 (128, 17, 2, 2), (256, 16, 2, 2)])
def test_runs_by_what_is_resident(ask, dim, rows, four, eight):
    """Few long contexts: as many runs as workgroups are resident, by the row
    tiles and dims, 256 CUs of them over 8 heads."""
    for form, per_cu in ((True, four), (False, eight)):
        rt, nrb, chunks, hw = ask(form, 3, 1, 8, dim, rows, 131072)
        assert chunks * 8 == 256 * per_cu if nrb == 1 else chunks > 0, (form, rt, nrb, chunks)


@pytest.mark.parametrize("B,four,eight", [(96, "units", "units"), (97, "units", "runs"), (128, "units", "runs"), (129, "runs", "runs"),
                                          (255, "runs", "units")])
def test_units_where_they_are_resident_together(ask, B, four, eight):
    """Contexts of 2048 tokens: a unit each while all are resident at once, and
    where there are two to each place; runs between."""
    for form, mode in ((True, four), (False, eight)):
        assert ("runs" if ask(form, B, 8, 8, 64, 1, 2048)[2] else "units") == mode


def test_batches_take_every_cut(ask):
    """The batches of the GPU tests reach units and runs, of one head and of several."""
    seen = set()
    for c in CASES + [MANY_SHORT]:
        _, _, chunks, hw = ask(True, len(c["ctx"]), c["G"], c["heads"], (c["dim"] + 31) // 32 * 32, max(c["lens"]),
                               c["max_ctx"], c["window"], c["order"] == "tokens")
        seen.add((bool(chunks), hw))
    assert seen >= {(False, 1), (True, 1), (False, 4), (True, 4), (False, 2), (True, 2)}, seen
