"""How an attention's rows and keys are cut into workgroups, on the CPU: the
plan's header compiled by itself, asked on both sides of each of its rules and
for the batches whose results the GPU tests check."""
import os
import shutil
import subprocess

import pytest

from attention_cases import CASES, FAR

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "rejection_sampling_verify_03_amd", "csrc")

PROGRAM = """
#include <stdio.h>
#include "attention_plan.hpp"
int main() {
  int B, G, heads, dim, max_q, max_ctx, window, in;
  long long total;
  while (scanf("%d %d %d %d %d %d %d %d %lld", &B, &G, &heads, &dim, &max_q, &max_ctx, &window, &in, &total) == 9) {
    const specv::AttnPlan p = specv::plan_attn(B, G, heads, dim, max_q, max_ctx, window, in);
    printf("%d %d %d %d %lld\\n", p.rt, p.nrb, p.chunks, p.hw,
           p.chunks ? (long long)specv::attn_run_tiles(total, p.chunks) : 0LL);
  }
  printf("%d %d %d\\n", specv::kTileKeys, specv::kAttnWaves, specv::kAttnWindow);
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("plan")
    (d / "p.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", CSRC, str(d / "p.cpp"), "-o", str(d / "p")],
                   check=True)

    def run(B, G, heads, dim, max_q, max_ctx, window=0, heads_in=True, total=1):
        """(rt, nrb, chunks, hw, tiles of a run), (tile, waves, window)"""
        line = " ".join(str(int(v)) for v in (B, G, heads, dim, max_q, max_ctx, window, heads_in, total))
        out = subprocess.run([str(d / "p")], input=line, check=True, capture_output=True, text=True).stdout.split()
        return tuple(map(int, out[:5])), tuple(map(int, out[5:]))
    return run


def unit_tiles(c, rt, nrb, tile):
    """Key tiles of each unit of a batch: request by request, block by block."""
    out = []
    for n, ctx in zip(c["lens"], c["ctx"]):
        for rb in range(nrb):
            m0, rows = rb * rt * 16, n * c["G"]
            if m0 >= rows:
                continue
            t0, t1 = m0 // c["G"], (min(rows, m0 + rt * 16) - 1) // c["G"]
            lo = max(0, ctx - n + t0 - c["window"] + 1) // tile * tile if c["window"] else 0
            out.append(max(1, -(-(max(ctx - n + t1 + 1, lo) - lo) // tile)))
    return out


@pytest.mark.parametrize("c", CASES, ids=[c["name"] for c in CASES])
def test_batches_take_the_cut_that_they_are_for(ask, c):
    args = (len(c["ctx"]), c["G"], c["heads"], c["dim"], max(c["lens"]), c["max_ctx"], c["window"],
            c["order"] == "tokens")
    (rt, nrb, _, _, _), (tile, waves, window) = ask(*args)
    tiles = unit_tiles(c, rt, nrb, tile)
    (_, _, chunks, hw, run), _ = ask(*args, sum(tiles))
    assert ("runs" if chunks else "units") == c["mode"] and hw == c["hw"]
    per_wave = -(-min(run or max(tiles), max(tiles)) // (waves // hw))
    assert per_wave >= c["tiles"], per_wave
    assert tile == 32 and window == 32  # (what the cases' numbers of tiles are chosen by)


@pytest.mark.parametrize("args,mode,hw", [
    # short contexts
    (dict(B=3, heads=8, max_ctx=1024), "units", 1), (dict(B=3, heads=8, max_ctx=1025), "units", 1),
    (dict(B=200, heads=8, max_ctx=1024), "units", 2), (dict(B=400, heads=8, max_ctx=1024), "units", 4),
    (dict(B=200, heads=8, max_ctx=FAR, window=1000), "units", 2),
    # few requests of up to 2048
    (dict(B=96, heads=8, max_ctx=2048), "units", 1), (dict(B=97, heads=8, max_ctx=2048), "runs", 1),
    (dict(B=96, heads=8, max_ctx=2049), "runs", 1),
    # full cards of up to 4096, by the heads that a workgroup takes
    (dict(B=768, heads=8, max_ctx=4096), "units", 4), (dict(B=767, heads=8, max_ctx=4096), "runs", 4),
    (dict(B=768, heads=8, max_ctx=4097), "runs", 4), (dict(B=768, heads=2, max_ctx=4096), "runs", 2),
    (dict(B=192, heads=8, max_ctx=4096, heads_in=False), "units", 1),
    # many units
    (dict(B=65536, heads=1, max_ctx=FAR), "runs", 1), (dict(B=65537, heads=1, max_ctx=FAR), "units", 1),
    # many blocks of rows
    (dict(B=2, heads=8, max_ctx=FAR, max_q=640, G=8), "units", 1),
    (dict(B=2, heads=8, max_ctx=FAR, max_q=630, G=8), "runs", 1),
    # a head to a wave for long runs of few rows
    (dict(B=3, heads=8, dim=128, max_ctx=131072), "runs", 4),
    (dict(B=3, heads=8, dim=128, max_ctx=131072, heads_in=False), "runs", 1),
    (dict(B=1, heads=8, dim=128, max_ctx=8192), "runs", 1)])
def test_rules(ask, args, mode, hw):
    (_, _, chunks, got, _), _ = ask(**{**dict(G=1, dim=64, max_q=1), **args})
    assert (("runs" if chunks else "units"), got) == (mode, hw)
