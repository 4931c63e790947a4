"""The C ABI and the binding of sampling, truncation, rotation, the 4-bit cache
and attention over it, on the CPU: struct layouts, workspace sizes, every
refusal before anything is enqueued (the pointers here are never
dereferenced), the rotation tables, and the 64-bit oracle."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

import decode_oracle as do

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20  # a well-aligned address that nothing reads


@pytest.fixture(scope="module")
def sv():
    import rejection_sampling_verify_03_amd as m
    return m


def test_struct_layouts_match_the_header(sv, tmp_path):
    pairs = (("spec_sample_args", sv.SpecSampleArgs), ("spec_truncate_args", sv.SpecTruncateArgs),
             ("spec_rope_args", sv.SpecRopeArgs), ("spec_kv4_cache", sv.SpecKV4Cache),
             ("spec_kv4_write_args", sv.SpecKV4WriteArgs), ("spec_kv4_read_args", sv.SpecKV4ReadArgs),
             ("spec_attn4_args", sv.SpecAttn4Args))
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "spec_verify.h"', "int main(void) {"]
    want = []
    for cname, py in pairs:
        lines.append('printf("%%zu\\n", sizeof(%s));' % cname)
        want.append(ctypes.sizeof(py))
        for f, _ in py._fields_:
            lines.append('printf("%%zu\\n", offsetof(%s, %s));' % (cname, f))
            want.append(getattr(py, f).offset)
    lines.append("return 0; }")
    src, exe = tmp_path / "l.c", tmp_path / "l"
    src.write_text("\n".join(lines))
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == want


def put(a, kw):
    for k, v in kw.items():
        setattr(a, k, v)
    return a


# ------------------------------------------------------ sampling, truncation
def sample_args(sv, **kw):
    a = sv.SpecSampleArgs()
    a.B, a.R, a.V, a.dtype = 2, 3, 1000, sv.SPEC_BF16
    a.logits, a.req_stride, a.row_stride = P, 3000, 1000
    a.temperature = a.uniforms = a.tokens = a.workspace = P
    a.workspace_bytes = 1 << 20
    return put(a, kw)


def truncate_args(sv, **kw):
    a = sv.SpecTruncateArgs()
    a.B, a.R, a.V, a.dtype = 2, 3, 1000, sv.SPEC_BF16
    a.logits, a.req_stride, a.row_stride, a.out, a.out_req_stride, a.out_row_stride = P, 3000, 1000, 2 * P, 3000, 1000
    a.temperature = a.workspace = P
    a.workspace_bytes = 1 << 20
    return put(a, kw)


BOTH = [
    (dict(B=-1), "SPEC_EINVAL"), (dict(R=-1), "SPEC_EINVAL"), (dict(V=0), "SPEC_EINVAL"), (dict(V=2 ** 31 - 1), "SPEC_EINVAL"),
    (dict(dtype=2), "SPEC_EDTYPE"), (dict(logits=None), "SPEC_EINVAL"), (dict(temperature=None), "SPEC_EINVAL"),
    (dict(row_stride=999), "SPEC_EINVAL"), (dict(req_stride=2999), "SPEC_EINVAL"), (dict(req_stride=-3000), "SPEC_EINVAL"),
    (dict(workspace=None), "SPEC_EINVAL"), (dict(workspace=P + 8), "SPEC_EALIGN"), (dict(workspace_bytes=8), "SPEC_EWORKSPACE"),
    (dict(B=2 ** 16, R=2 ** 15, req_stride=0), "SPEC_EINVAL"), (dict(B=2 ** 16, R=100, req_stride=0), "SPEC_EINVAL")]


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(uniforms=None), "SPEC_EINVAL"), (dict(tokens=None), "SPEC_EINVAL"), (dict(row_index=P, rows=-1), "SPEC_EINVAL")])
def test_sample_refusals(sv, kw, status):
    assert sv.spec_sample_launch(sample_args(sv, **kw), None) == getattr(sv, status)


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(out=None), "SPEC_EINVAL"), (dict(out_row_stride=999), "SPEC_EINVAL"), (dict(out_req_stride=2999), "SPEC_EINVAL"),
    (dict(out_req_stride=0), "SPEC_EINVAL"), (dict(out=P, out_req_stride=6000), "SPEC_EINVAL"),
    (dict(out=P, out_row_stride=1001, out_req_stride=3003), "SPEC_EINVAL"), (dict(out=P, req_stride=0), "SPEC_EINVAL")])
def test_truncate_refusals(sv, kw, status):
    assert sv.spec_truncate_launch(truncate_args(sv, **kw), None) == getattr(sv, status)


def test_sampling_of_nothing_and_workspaces(sv):
    for n in ("B", "R"):
        assert sv.spec_sample_launch(sample_args(sv, **{n: 0, "logits": None}), None) == sv.SPEC_OK
        assert sv.spec_truncate_launch(truncate_args(sv, **{n: 0, "out": None}), None) == sv.SPEC_OK
    assert sv.lib.spec_sample_launch(None, None) == sv.lib.spec_truncate_launch(None, None) == sv.SPEC_EINVAL
    assert sv.spec_sample_workspace_bytes(2, 3, 1000) > 0
    for bad in ((-1, 1, 10), (1, -1, 10), (1, 1, 0), (1, 1, 2 ** 31 - 1), (2 ** 33, 1, 10), (2 ** 20, 2 ** 20, 10)):
        assert sv.spec_sample_workspace_bytes(*bad) == 0


# ------------------------------------------------------------------ rotation
def rope_args(sv, **kw):
    a = sv.SpecRopeArgs()
    a.N, a.q_heads, a.k_heads, a.head_dim, a.rot_dim, a.dtype, a.scale = 4, 8, 2, 64, 32, sv.SPEC_BF16, 1.0
    a.inv_freq = a.positions = a.q = a.k = P
    a.q_out = a.k_out = 2 * P
    a.q_token_stride = a.q_out_token_stride = 512
    a.k_token_stride = a.k_out_token_stride = 128
    a.q_head_stride = a.k_head_stride = a.q_out_head_stride = a.k_out_head_stride = 64
    return put(a, kw)


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), "SPEC_EINVAL"), (dict(q_heads=-1), "SPEC_EINVAL"), (dict(k_heads=1025), "SPEC_EINVAL"),
    (dict(head_dim=0), "SPEC_EINVAL"), (dict(head_dim=60), "SPEC_EINVAL"), (dict(head_dim=264), "SPEC_EINVAL"),
    (dict(rot_dim=0), "SPEC_EINVAL"), (dict(rot_dim=24), "SPEC_EINVAL"), (dict(rot_dim=80), "SPEC_EINVAL"),
    (dict(dtype=3), "SPEC_EDTYPE"), (dict(scale=math.inf), "SPEC_EINVAL"), (dict(scale=math.nan), "SPEC_EINVAL"),
    (dict(inv_freq=None), "SPEC_EINVAL"), (dict(positions=None), "SPEC_EINVAL"), (dict(q=None), "SPEC_EINVAL"),
    (dict(k_out=None), "SPEC_EINVAL"), (dict(q_token_stride=-1), "SPEC_EINVAL"), (dict(k_out_head_stride=-64), "SPEC_EINVAL"),
    (dict(q_out=P, q_out_token_stride=1024), "SPEC_EINVAL"), (dict(k_out=P, k_out_head_stride=128), "SPEC_EINVAL"),
    (dict(N=2 ** 31 - 1, q_heads=1024), "SPEC_EINVAL")])
def test_rope_refusals(sv, kw, status):
    assert sv.spec_rope_launch(rope_args(sv, **kw), None) == getattr(sv, status)


def test_rope_of_nothing(sv):
    assert sv.spec_rope_launch(rope_args(sv, N=0, q=None), None) == sv.SPEC_OK
    assert sv.spec_rope_launch(rope_args(sv, q_heads=0, k_heads=0, q=None, k=None), None) == sv.SPEC_OK
    assert sv.lib.spec_rope_launch(None, None) == sv.SPEC_EINVAL


# --------------------------------------------------------------- 4-bit cache
def cache_args(sv, **kw):
    c = sv.SpecKV4Cache()
    c.num_blocks, c.block_size, c.heads, c.head_dim = 10, 16, 2, 64
    c.k_codes, c.v_codes, c.k_scales, c.v_scales = P, 2 * P, 3 * P, 4 * P
    c.block_stride, c.token_stride, c.head_stride = 1024, 32, 512
    c.scale_block_stride, c.scale_head_stride = 64, 32
    return put(c, kw)


BAD_CACHES = [
    (dict(num_blocks=0), "SPEC_EINVAL"), (dict(block_size=8), "SPEC_EINVAL"), (dict(block_size=48), "SPEC_EINVAL"),
    (dict(block_size=2048), "SPEC_EINVAL"), (dict(heads=0), "SPEC_EINVAL"), (dict(heads=1025), "SPEC_EINVAL"),
    (dict(head_dim=0), "SPEC_EINVAL"), (dict(head_dim=48), "SPEC_EINVAL"), (dict(head_dim=288), "SPEC_EINVAL"),
    (dict(k_codes=None), "SPEC_EINVAL"), (dict(v_scales=None), "SPEC_EINVAL"), (dict(k_codes=P + 8), "SPEC_EALIGN"),
    (dict(token_stride=40), "SPEC_EALIGN"), (dict(block_stride=1032), "SPEC_EALIGN"), (dict(token_stride=16), "SPEC_EINVAL"),
    (dict(head_stride=496), "SPEC_EINVAL"), (dict(block_stride=1008), "SPEC_EINVAL"), (dict(token_stride=-32), "SPEC_EINVAL"),
    (dict(head_stride=2 ** 50), "SPEC_EINVAL"), (dict(scale_head_stride=31), "SPEC_EINVAL"),
    (dict(scale_block_stride=63), "SPEC_EINVAL")]


def write_args(sv, cache=None, **kw):
    a = sv.SpecKV4WriteArgs()
    a.cache = cache_args(sv) if cache is None else cache
    a.N, a.dtype, a.key, a.value, a.slots = 4, sv.SPEC_BF16, P, P, P
    a.k_token_stride = a.v_token_stride = 128
    a.k_head_stride = a.v_head_stride = 64
    a.rot_dim, a.inv_freq, a.scale, a.positions = 32, P, 1.0, P
    a.q_heads, a.q, a.q_out = 8, P, 2 * P
    a.q_token_stride = a.q_out_token_stride = 512
    a.q_head_stride = a.q_out_head_stride = 64
    return put(a, kw)


def read_args(sv, cache=None, **kw):
    a = sv.SpecKV4ReadArgs()
    a.cache = cache_args(sv) if cache is None else cache
    a.N, a.dtype, a.key, a.value, a.slots = 4, sv.SPEC_BF16, P, P, P
    return put(a, kw)


def attn_args(sv, cache=None, **kw):
    a = sv.SpecAttn4Args()
    a.cache = cache_args(sv) if cache is None else cache
    a.B, a.N, a.q_heads, a.max_q, a.max_ctx, a.window, a.dtype, a.scale = 2, 4, 8, 2, 64, 0, sv.SPEC_BF16, 0.125
    a.q = a.q_start = a.ctx_len = a.block_table = a.out = P
    a.q_token_stride, a.q_head_stride, a.bt_row_stride, a.max_blocks = 512, 64, 4, 4
    return put(a, kw)


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_cache_refusals(sv, kw, status):
    c = cache_args(sv, **kw)
    assert sv.spec_kv4_write_launch(write_args(sv, c), None) == getattr(sv, status)
    assert sv.spec_kv4_read_launch(read_args(sv, c), None) == getattr(sv, status)
    assert sv.spec_attn4_launch(attn_args(sv, c), None) == getattr(sv, status)


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), "SPEC_EINVAL"), (dict(dtype=5), "SPEC_EDTYPE"), (dict(key=None), "SPEC_EINVAL"),
    (dict(value=None), "SPEC_EINVAL"), (dict(slots=None), "SPEC_EINVAL"), (dict(k_token_stride=-1), "SPEC_EINVAL"),
    (dict(rot_dim=-16), "SPEC_EINVAL"), (dict(rot_dim=24), "SPEC_EINVAL"), (dict(rot_dim=80), "SPEC_EINVAL"),
    (dict(rot_dim=0), "SPEC_EINVAL"), (dict(q_heads=1025), "SPEC_EINVAL"), (dict(q_heads=-1), "SPEC_EINVAL"),
    (dict(scale=math.nan), "SPEC_EINVAL"), (dict(inv_freq=None), "SPEC_EINVAL"), (dict(positions=None), "SPEC_EINVAL"),
    (dict(q=None), "SPEC_EINVAL"), (dict(q_out=None), "SPEC_EINVAL"), (dict(q_out=P, q_out_token_stride=1024), "SPEC_EINVAL"),
    (dict(N=2 ** 31 - 1, q_heads=1024), "SPEC_EINVAL")])
def test_write_refusals(sv, kw, status):
    assert sv.spec_kv4_write_launch(write_args(sv, **kw), None) == getattr(sv, status)


def test_writes_to_keys_and_values_in_one_place(sv):
    for kw in (dict(v_codes=P), dict(v_scales=3 * P)):
        assert sv.spec_kv4_write_launch(write_args(sv, cache_args(sv, **kw)), None) == sv.SPEC_EINVAL


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), "SPEC_EINVAL"), (dict(dtype=5), "SPEC_EDTYPE"), (dict(key=None), "SPEC_EINVAL"),
    (dict(value=None), "SPEC_EINVAL"), (dict(slots=None), "SPEC_EINVAL")])
def test_read_refusals(sv, kw, status):
    assert sv.spec_kv4_read_launch(read_args(sv, **kw), None) == getattr(sv, status)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), "SPEC_EINVAL"), (dict(N=-1), "SPEC_EINVAL"), (dict(q_heads=7), "SPEC_EINVAL"), (dict(q_heads=130), "SPEC_EINVAL"),
    (dict(max_q=0), "SPEC_EINVAL"), (dict(max_ctx=-1), "SPEC_EINVAL"), (dict(max_ctx=2 ** 30 + 1), "SPEC_EINVAL"),
    (dict(window=-1), "SPEC_EINVAL"), (dict(dtype=0), "SPEC_EDTYPE"), (dict(scale=math.inf), "SPEC_EINVAL"),
    (dict(scale=math.nan), "SPEC_EINVAL"), (dict(q=None), "SPEC_EINVAL"), (dict(q_start=None), "SPEC_EINVAL"),
    (dict(ctx_len=None), "SPEC_EINVAL"), (dict(block_table=None), "SPEC_EINVAL"), (dict(out=None), "SPEC_EINVAL"),
    (dict(out=P + 8), "SPEC_EALIGN"), (dict(bt_row_stride=3), "SPEC_EINVAL"), (dict(q_head_stride=-1), "SPEC_EINVAL"),
    (dict(max_ctx=1 << 20, max_blocks=4), "SPEC_EINVAL")])
def test_attention_refusals(sv, kw, status):
    assert sv.spec_attn4_launch(attn_args(sv, **kw), None) == getattr(sv, status)


def test_of_nothing_and_attention_workspace(sv):
    assert sv.spec_kv4_write_launch(write_args(sv, N=0, key=None), None) == sv.SPEC_OK
    assert sv.spec_kv4_read_launch(read_args(sv, N=0, key=None), None) == sv.SPEC_OK
    assert sv.spec_attn4_launch(attn_args(sv, B=0, q=None), None) == sv.SPEC_OK
    assert sv.spec_attn4_launch(attn_args(sv, N=0, q=None), None) == sv.SPEC_OK
    for f in (sv.lib.spec_kv4_write_launch, sv.lib.spec_kv4_read_launch, sv.lib.spec_attn4_launch):
        assert f(None, None) == sv.SPEC_EINVAL
    assert sv.lib.spec_attn4_workspace_bytes(None) == 0
    assert sv.spec_attn4_workspace_bytes(attn_args(sv)) == 0
    far = attn_args(sv, max_ctx=1 << 20, max_blocks=1 << 16, bt_row_stride=1 << 16)
    need = sv.spec_attn4_workspace_bytes(far)
    assert need > 0
    far.workspace, far.workspace_bytes = P, need - 1
    assert sv.spec_attn4_launch(far, None) == sv.SPEC_EWORKSPACE
    far.workspace, far.workspace_bytes = P + 8, need
    assert sv.spec_attn4_launch(far, None) == sv.SPEC_EALIGN
    assert sv.spec_attn4_workspace_bytes(attn_args(sv, cache_args(sv, head_dim=48), max_ctx=1 << 20)) == 0


# ------------------------------------------------------------------- binding
def test_binding_refusals(sv):
    x, t = torch.zeros(1, 1, 8), torch.zeros(1)
    for call in (lambda: sv.sample(x, torch.zeros(1, 1), t), lambda: sv.truncate_logits(x, t),
                 lambda: sv.rope(torch.zeros(1, 1, 16), None, torch.zeros(1, dtype=torch.int32), None),
                 lambda: sv.Rope(torch.zeros(8, dtype=torch.float64)), lambda: sv.truncate_logits(torch.zeros(2, 8), t),
                 lambda: sv.Rope(torch.zeros(8)), lambda: sv.Rope(torch.zeros(2, 8, dtype=torch.float64)),
                 lambda: sv.make_kv4_cache(1, 16, 1, 48, device="cpu"), lambda: sv.make_kv4_cache(1, 16, 1, 64, device="cpu"),
                 lambda: sv.make_rope(24), lambda: sv.make_rope(32, base=1.0), lambda: sv.make_rope(32, factor=0.5),
                 lambda: sv.make_rope(32, scaling="other"), lambda: sv.make_rope(32, scaling="yarn", factor=2.0)):
        with pytest.raises(ValueError):
            call()
    codes, scales = torch.zeros(1, 16, 1, 32, dtype=torch.uint8), torch.zeros(1, 1, 2, 16, dtype=torch.uint8)
    with pytest.raises(TypeError):
        sv.KVCache4(codes.float(), codes.float(), scales, scales)
    with pytest.raises(TypeError):
        sv.rope_kv_write(object(), None, None, None, None, None, None)


# -------------------------------------------------------------------- oracle
def test_oracle_conversions():
    y = np.linspace(-6, 6, 4801)
    c = do.encode(y)
    v = np.where(c >= 8, -1.0, 1.0) * do.GRID[c & 7]
    signed = np.concatenate([-do.GRID, do.GRID])
    assert np.all(np.abs(v - y) <= np.abs(signed[None] - y[:, None]).min(1))
    assert np.array_equal(do.GRID[do.encode(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]))], [0, 1, 1, 2, 2, 4, 4])
    k, v, ks, vs = (np.zeros(s, np.uint8) for s in ((2, 16, 1, 16), (2, 16, 1, 16), (2, 1, 1, 16), (2, 1, 1, 16)))
    x = np.zeros((3, 1, 32))
    x[0, 0, :3], x[1, 0, 0], x[2, 0, 5] = [6.0, -2.5, 5.0], 6.001, np.inf
    do.kv_write(k, ks, x, [3, 20, 31])
    assert ks[0, 0, 0, 3] == 127 and ks[1, 0, 0, 4] == 128 and ks[1, 0, 0, 15] == 255
    got = do.kv_values(k, ks, [3, 20, 31, -1])
    assert got[0, 0, :3].tolist() == [6.0, -2.0, 4.0] and got[1, 0, 0] == 6.0
    assert np.isnan(got[2]).all() and not got[3].any()


def test_oracle_cuts():
    x = np.log(np.array([0.1, 0.4, 0.2, 0.2, 0.1]))
    assert do.cut(x, 1.0, 3, 1.0, 0.0)[0].tolist() == [False, True, True, True, False]
    assert do.cut(x, 1.0, 2, 1.0, 0.0)[0].tolist() == [False, True, True, False, False]
    assert do.cut(x, 1.0, 0, 0.5, 0.0)[0].tolist() == [False, True, True, False, False]
    assert do.cut(x, 1.0, 0, 0.39, 0.0)[0].tolist() == [False, True, False, False, False]
    assert do.cut(x, 1.0, 0, 1.0, 0.45)[0].tolist() == [False, True, True, True, False]
    assert do.cut(x, 1.0, 3, 0.7, 0.0)[0].tolist() == [False, True, True, False, False]
    assert do.one_token(x, 0.0, 1.0) == 0 and do.one_token(x, 0.11, 1.0) == 1 and do.one_token(x, 0.95, 1.0) == 4
    assert do.one_token(x, 0.6, 1.0, k=3) == 2
    assert do.one_token(x, 0.99, 0.0) == 1 and do.one_token(x, 1.0, 1.0) == -1


@pytest.mark.parametrize("scaling,kw", [(None, {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=8.0)),
                                        ("yarn", dict(factor=8.0, trained=4096))])
def test_rotation_tables(sv, scaling, kw, monkeypatch):
    """The angles against the formulas."""
    class Table:
        def __init__(self, inv_freq, scale, interleaved):
            self.inv_freq, self.scale, self.interleaved = inv_freq, scale, interleaved
    monkeypatch.setattr(sv, "Rope", Table)
    rot, base = 64, 10000.0
    r = sv.make_rope(rot, base, scaling=scaling, device="cpu", **kw)
    f = kw.get("factor", 1.0)
    i = np.arange(rot // 2)
    plain = base ** (-2.0 * i / rot)
    got = r.inv_freq.numpy()
    assert got[0] == 1.0 if scaling != "linear" else got[0] == 0.25
    if scaling is None:
        want = plain
    elif scaling == "linear":
        want = plain / f
    elif scaling == "ntk":
        want = (base * f ** (rot / (rot - 2.0))) ** (-2.0 * i / rot)
        assert abs(got[-1] * f / plain[-1] - 1) < 1e-12  # the slowest pair is divided by the factor
    else:
        turns = 4096 * plain / (2 * math.pi)
        want = None
        assert np.allclose(got[turns > 40], plain[turns > 40], rtol=1e-13)
        assert np.allclose(got[turns < 0.9], plain[turns < 0.9] / f, rtol=1e-13)
        assert np.all(np.diff(got) < 0) and np.all(got <= plain * (1 + 1e-13)) and np.all(got >= plain / f * (1 - 1e-13))
        assert abs(r.scale - (0.1 * math.log(f) + 1)) < 1e-15
    if want is not None:
        assert np.allclose(got, want, rtol=1e-13) and r.scale == 1.0
