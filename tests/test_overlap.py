"""Outputs whose elements share a place, among themselves or with another tensor of
the call: the host's rule against counting bytes, and the entry points' refusals
(the pointers here are never dereferenced)."""
import os
import random
import shutil
import subprocess

import pytest

from test_decode_abi import P, rope_args, truncate_args, write_args

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "rejection_sampling_verify_03_amd", "csrc")

PROGRAM = """
#include <stdio.h>
#include "overlap.hpp"
int main() {
  long long v[12];
  for (;;) {
    for (int i = 0; i < 12; ++i)
      if (scanf("%lld", v + i) != 1) return 0;
    const specv::MemRows a{(uintptr_t)v[0], v[1], v[2], v[3], v[4], v[5]}, b{(uintptr_t)v[6], v[7], v[8], v[9], v[10], v[11]};
    printf("%d %d\\n", specv::rows_share(b), specv::rows_meet(a, b));
  }
}
"""


@pytest.fixture(scope="module")
def sv():
    import rejection_sampling_verify_03_amd as m
    return m


def places(r):
    base, n, outer, m, inner, ln = r
    return [base + i * outer + j * inner + k for i in range(n) for j in range(m) for k in range(ln)]


def test_the_rule_against_bytes(tmp_path):
    cxx = shutil.which("g++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    (tmp_path / "o.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", CSRC, str(tmp_path / "o.cpp"), "-o",
                    str(tmp_path / "o")], check=True)
    rng = random.Random(1)
    cases = []
    for _ in range(20000):
        ln, n, m = rng.randint(1, 6), rng.randint(1, 5), rng.randint(1, 5)
        kind = rng.randrange(4)
        inner = ln + rng.randint(0, 8) if kind else rng.randint(0, 8)
        outer = rng.choice([m * inner + rng.randint(0, 40), rng.randint(0, 30)])
        if rng.random() < 0.3:
            inner, outer = outer, inner
        a = (1000 + rng.randint(-60, 60), n, outer, m, inner, ln)
        if kind == 1:      # parts of the same rows
            b = (1000 + rng.randint(-60, 60), n, outer, rng.randint(1, 5), rng.choice([inner, rng.randint(0, 12)]), rng.randint(1, 6))
        else:
            l2, n2, m2 = rng.randint(1, 6), rng.randint(1, 5), rng.randint(1, 5)
            i2 = l2 + rng.randint(0, 8)
            b = (1000 + rng.randint(-60, 60), n2, m2 * i2 + rng.randint(0, 9), m2, i2, l2)
            if rng.random() < 0.3:
                b = (b[0], m2, i2, n2, b[2], l2)
        cases.append((a, b))
    far = 1 << 62          # strides whose products pass 64 bits
    cases += [((1000, 3, far, 3, far, 4), (1000 + 2, 1, 0, 1, 0, 1)), ((1000, 3, far, 1, 0, 4), (1004, 3, far, 1, 0, 4))]
    want_far = [("0", "1"), ("0", "0")]
    text = "\n".join(" ".join(map(str, a + b)) for a, b in cases)
    out = subprocess.run([str(tmp_path / "o")], input=text, check=True, capture_output=True, text=True).stdout.split()
    got = list(zip(out[::2], out[1::2]))
    assert got[-2:] == want_far
    met = shared = 0
    for (a, b), (share, meet) in zip(cases[:-2], got):
        pb = places(b)
        assert int(share) == (len(set(pb)) < len(pb)), b
        if share == "0":
            want = bool(set(places(a)) & set(pb))
            nested = a[1] == b[1] and (a[1] == 1 or a[2] == b[2])
            nested |= b[1] == 1 or b[3] == 1 or b[2] >= (b[3] - 1) * b[4] + b[5] or b[4] >= (b[1] - 1) * b[2] + b[5]
            assert int(meet) == want or (meet == "1" and not nested), (a, b)
            met += want
        else:
            shared += 1
    assert 1000 < met < 19000 and shared > 200


@pytest.mark.parametrize("kw", [
    dict(q_out_head_stride=0), dict(q_out_token_stride=0), dict(k_out_head_stride=32), dict(k_out_token_stride=64),
    dict(k_out=2 * P), dict(k_out=2 * P + 64), dict(q_out=P + 2, k=4 * P), dict(k_out=P, q=P, k=8 * P),
    dict(q=P, k=8 * P, q_out=8 * P), dict(q_out=2 * P, k_out=2 * P + 3 * 1024 + 1022), dict(k_out=2 * P - 3 * 256 - 254),
    dict(q=P, q_out=P, q_head_stride=0, q_out_head_stride=0)])
def test_rotations_into_one_place(sv, kw):
    base = dict(k=4 * P, k_out=6 * P)
    assert sv.spec_rope_launch(rope_args(sv, **{**base, **kw}), None) == sv.SPEC_EINVAL


@pytest.mark.parametrize("kw", [dict(q_out_head_stride=0), dict(q_out_token_stride=448), dict(q_out=P + 16),
                                dict(key=16 * P, q_out=16 * P), dict(value=16 * P, q_out=16 * P + 128)])
def test_rotated_queries_of_a_write_into_one_place(sv, kw):
    assert sv.spec_kv4_write_launch(write_args(sv, **{**dict(q=8 * P, q_out=32 * P), **kw}), None) == sv.SPEC_EINVAL


@pytest.mark.parametrize("kw", [dict(out=P + 2), dict(out=P + 2000 * 2), dict(out=P - 5998, out_req_stride=3500),
                                dict(req_stride=0, out=P - 6000 * 2 + 2, out_row_stride=1000, out_req_stride=3000)])
def test_truncation_into_what_it_reads(sv, kw):
    assert sv.spec_truncate_launch(truncate_args(sv, **kw), None) == sv.SPEC_EINVAL
