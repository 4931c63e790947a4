"""Rotation at its ends: keys that leave fp32's range on their way into the 4-bit
cache, and tensors in and out of place next to each other."""
import math

import numpy as np
import pytest
import torch

import decode_oracle as do

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def sv():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import rejection_sampling_verify_03_amd as m
    return m


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("inter", [False, True])
def test_turned_keys_past_fp32_count_as_infinite(sv, inter, dtype):
    """Pairs near the largest number turned by an eighth of a circle, so that one
    of them grows by up to 2^(1/2): what fp32 holds has the definition's codes, a
    group with an element that it does not hold is NaN."""
    dim, N = 64, 40
    big = torch.finfo(dtype).max
    g = torch.Generator().manual_seed(3)
    key = torch.randn(N, 1, dim, generator=g)
    i, j = (slice(0, dim, 2), slice(1, dim, 2)) if inter else (slice(0, dim // 2), slice(dim // 2, dim))
    for n in range(N):                                   # one pair of each token, from half of the range up
        p = n % (dim // 2)
        key[n, 0, i][p] = key[n, 0, j][p] = big * (0.5 + n / (2 * N - 2))
        if n % 3 == 1:
            key[n, 0, i][p] *= -1
    key = key.to(dtype)
    f = np.full(dim // 2, math.pi / 4)
    pos = torch.ones(N, dtype=torch.int32)
    want = do.rotate(key.double().numpy(), pos.numpy(), f, 1.0, inter)
    past = np.abs(want) >= 2.0 ** 128 - 2.0 ** 103       # (what rounds to 2^128)
    assert 5 < past.any((1, 2)).sum() < N - 5
    # cosine, sine, product and sum are off by 2^-53 of |x| + |y| each, on either side:
    # where a pair of these sizes cancels, what is left of it is below 2^-50 of them,
    # its digits are not determined, and so is the scale of a group that holds nothing larger
    size = np.empty_like(want)
    x = np.abs(key.double().numpy())
    size[..., i] = size[..., j] = x[..., i] + x[..., j]
    sure = (np.abs(want).reshape(N, 2, 32).max(2) > 2.0 ** -20 * size.reshape(N, 2, 32).max(2))  # [N, group]
    assert sure[past.reshape(N, 2, 32).any(2)].all() and sure.sum() >= N
    want[past] = np.inf
    cache = sv.make_kv4_cache(3, 16, 1, dim)
    host = [torch.zeros_like(t, device="cpu").numpy() for t in (cache.k, cache.k_scale)]
    slots = torch.arange(N)
    sv.rope_kv_write(cache, None, key.cuda(), key.cuda(), pos.cuda(), slots.cuda(),
                     sv.Rope(torch.from_numpy(f).cuda(), 1.0, inter))
    torch.cuda.synchronize()
    do.kv_write(host[0], host[1], want, slots.tolist())
    t = slots.numpy()
    got_scale, scale = (a[t // 16, 0, :, t % 16] for a in (cache.k_scale.cpu().numpy(), host[1]))    # [N, group]
    got, codes = (a[t // 16, t % 16, 0].reshape(N, 2, 16) for a in (cache.k.cpu().numpy(), host[0]))
    assert np.array_equal(got_scale[sure], scale[sure]) and np.array_equal(got[sure], codes[sure])
    assert ((scale == 255) == past.reshape(N, 2, 32).any(2)).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_in_place_with_queries_and_keys_side_by_side(sv, dtype):
    """Queries, keys and values of a head next to each other, tokens outside or
    inside: rotated where they stand, equal to new outputs, the rest untouched; the
    same tensor twice, or a shared head, as an output is refused."""
    g = torch.Generator().manual_seed(5)
    N, H, D = 19, 5, 64
    r = sv.make_rope(D)
    pos = torch.arange(N, dtype=torch.int32).cuda()
    for shape, of in (((N, H, 3, D), lambda t, i: t[:, :, i]), ((3, H, N, D), lambda t, i: t[i].transpose(0, 1))):
        buf = torch.randn(shape, generator=g).to(dtype).cuda()
        before = buf.clone()
        q, k, v = (of(buf, i) for i in range(3))
        want = sv.rope(q, k, pos, r)
        got = sv.rope(q, k, pos, r, out=(q, k))
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(v, of(before, 2))
        cache = sv.make_kv4_cache(2, 16, H, D)
        q.copy_(of(before, 0))
        out = sv.rope_kv_write(cache, q, k, v, pos, pos.long(), r, q_out=q)
        torch.cuda.synchronize()
        assert out is q and torch.equal(q, want[0])
        for call in (lambda: sv.rope(q, k, pos, r, out=(want[0], want[0])), lambda: sv.rope(q, k, pos, r, out=(k, q)),
                     lambda: sv.rope(q, k, pos, r, out=(q[:, :1].expand(N, H, D), want[1])),
                     lambda: sv.rope_kv_write(cache, q, k, v, pos, pos.long(), r, q_out=v)):
            with pytest.raises(sv.SpecError):
                call()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("scale", [1.0, 1.2079, 4.0, -0.5])
def test_bf16_rotation_within_its_documented_error(sv, scale, inter):
    """Off by 2^-22 |scale| (|x| + |y|) at most before the rounding to bf16: pairs
    of any angle, and such that almost cancel, where that rounding is small."""
    N, H, D = 300, 4, 64
    g = torch.Generator().manual_seed(11)
    pos = torch.randint(-1000, 100000, (N,), generator=g).to(torch.int32)
    f = 10000.0 ** (-2.0 * np.arange(D // 2) / D)
    i, j = (slice(0, D, 2), slice(1, D, 2)) if inter else (slice(0, D // 2), slice(D // 2, D))
    x = torch.randn(N, H, D, generator=g)
    a = pos.double()[:, None, None] * torch.from_numpy(f)
    y = x[..., i].double() * a.cos() / a.sin()
    near = torch.rand(N, H, D // 2, generator=g) < 0.5
    x[..., j] = torch.where(near & (y.abs() < 100), y.float(), x[..., j])
    x = x.to(BF16)
    got, _ = sv.rope(x.cuda(), None, pos.cuda(), sv.Rope(torch.from_numpy(f).cuda(), scale, inter))
    torch.cuda.synchronize()
    want = do.rotate(x.double().numpy(), pos.numpy(), f, scale, inter)
    size = np.empty_like(want)
    x = np.abs(x.double().numpy())
    size[..., i] = size[..., j] = 2.0 ** -22 * abs(scale) * (x[..., i] + x[..., j])
    assert (np.abs(want) < 2.0 ** -8 * abs(scale) * x.max()).mean() > 0.2  # (many cancel)
    assert np.all(np.abs(got.cpu().double().numpy() - want) <= size + 2.0 ** -8 * (np.abs(want) + size))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("hq,heads,dim,rot,N", [(2, 1, 64, 64, 17003), (6, 2, 128, 32, 16390), (3, 2, 96, 80, 18001), (1, 1, 256, 256, 16385),
                                                (0, 1, 32, 16, 20011), (33, 4, 64, 48, 16400)])
def test_many_tokens(sv, hq, heads, dim, rot, N, inter, dtype):
    """Several tokens to a workgroup: queries against the definition, keys and
    values in the cache against writes of few tokens at a time, some entries
    skipped, some slots given to two entries next to each other."""
    g = torch.Generator().manual_seed(N)
    f = 10000.0 ** (-2.0 * np.arange(rot // 2) / rot)
    r = sv.Rope(torch.from_numpy(f).cuda(), 1.1, inter)
    q = torch.randn(N, hq, dim, generator=g).to(dtype) if hq else None
    key, val = ((torch.randn(N, heads, dim, generator=g) * 3).to(dtype) for _ in range(2))
    pos = torch.randint(0, 100000, (N,), generator=g).long()
    slots = torch.randperm(N, generator=g)
    slots[torch.rand(N, generator=g) < 0.1] = -1
    twice = torch.arange(0, N - 1, 10)
    slots[twice] = slots[twice + 1]
    dq, dk, dv, dp, ds = (None if t is None else t.cuda() for t in (q, key, val, pos, slots))
    one, two = (sv.make_kv4_cache(-(-N // 16), 16, heads, dim) for _ in range(2))
    out = sv.rope_kv_write(one, dq, dk, dv, dp, ds, r)
    for i in range(0, N, 1000):  # (no pair of equal slots is parted)
        sv.rope_kv_write(two, None, dk[i:i + 1000], dv[i:i + 1000], dp[i:i + 1000], ds[i:i + 1000], r)
    turned = sv.rope(dk if q is None else dq, dk, dp, r)
    torch.cuda.synchronize()
    for n in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(getattr(one, n), getattr(two, n)), n
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    for x, got in ((q, out), (q, turned[0] if hq else None), (key, turned[1])):
        if got is None:
            continue
        x, got = x.double().numpy(), got.cpu().double().numpy()
        want, size = do.rotate(x, pos.numpy(), f, 1.1, inter), np.zeros_like(x)
        size[..., i] = size[..., j] = 1.1 * (np.abs(x[..., i]) + np.abs(x[..., j]))
        early = 2.0 ** -22 * size if dtype == BF16 else 1e-12
        assert np.all(np.abs(got - want) <= torch.finfo(dtype).eps / 2 * (np.abs(want) + early) + early)
