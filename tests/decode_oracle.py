"""Plain 64-bit implementations of sampling from cut distributions, rotary
positions, the 4-bit paged cache and attention over it, from their
definitions: CPU tensors or numpy arrays in and out."""
import math

import numpy as np
import torch

U = 2.0 ** -24  # half a step of fp32
E_MIN = -117
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])  # e2m1 magnitudes by code


# --------------------------------------------------------- cut distributions
def cut(x, T, k, p, mn):
    """(which logits of a row stay, their weights in 80 bits): x 64-bit, T > 0."""
    V = len(x)
    order = np.lexsort((np.arange(V), -x))
    w = np.exp((x - x.max()).astype(np.longdouble) / np.longdouble(T))
    s = w[order]
    keep = np.arange(V) < (k if k > 0 else V)
    s = np.where(keep, s, 0)
    if p < 1:
        front = np.concatenate([[0], np.cumsum(s)[:-1]])
        keep &= front < np.longdouble(p) * s.sum()
    keep &= s >= mn
    kept = np.zeros(V, bool)
    kept[order[keep]] = True
    return kept, w


def usable(T, k, p, mn):
    return (T == 0 or 2.0 ** -126 <= T < math.inf) and k >= 0 and p > 0 and 0 <= mn <= 1


def one_token(x, u, T, k=0, p=1.0, mn=0.0):
    """The token of a row (64-bit logits), -1 where it or its settings cannot be used."""
    if not usable(T, k, p, mn) or not 0 <= u < 1:
        return -1
    if T == 0:
        y = np.where(np.isnan(x), -math.inf, x)
        return int(y.argmax()) if y.max() > -math.inf else 0
    if np.isnan(x).any() or not math.isfinite(x.max()):
        return -1
    kept, w = cut(x, T, k, p, mn)
    c = np.cumsum(np.where(kept, w, 0))
    return int(np.argmax(c > np.longdouble(u) * c[-1]))


def settings(B, T, k=None, p=None, mn=None):
    """The settings of each request, as the binding's arguments hold them, as Python numbers."""
    f = lambda t, d: [d] * B if t is None else [v for v in t.tolist()]  # noqa: E731
    return list(zip(T.tolist(), f(k, 0), f(p, 1.0), f(mn, 0.0)))


def sample(x, u, T, k=None, p=None, mn=None):
    """Tokens [B, R] for logits [B, R, V] and uniforms [B, R]."""
    B, R, _ = x.shape
    s, u = settings(B, T, k, p, mn), np.asarray(u)
    x = x.double().numpy()
    return np.array([[one_token(x[b, r], float(u[b, r]), *s[b]) for r in range(R)] for b in range(B)])


def truncate(x, T, k=None, p=None, mn=None):
    """logits [B, R, V] (64-bit array) with -inf where a token is left out."""
    B, R, _ = x.shape
    s = settings(B, T, k, p, mn)
    out = x.double().numpy().copy()
    for b in range(B):
        for r in range(R):
            row = out[b, r]
            if not usable(*s[b]):
                row[:] = np.nan
            elif s[b][0] > 0 and not np.isnan(row).any() and math.isfinite(row.max()):
                row[~cut(row, *s[b])[0]] = -math.inf
    return out


# ----------------------------------------------------------------- rotation
def rotate(x, positions, inv_freq, scale, interleaved):
    """x [N, heads, dim] in 64 bits turned to positions [N]."""
    rot = 2 * len(inv_freq)
    a = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    c, s = (np.cos(a) * scale)[:, None], (np.sin(a) * scale)[:, None]
    y = np.array(x, np.float64)
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    u, v = y[..., i].copy(), y[..., j].copy()
    y[..., i], y[..., j] = u * c - v * s, v * c + u * s
    return y


# -------------------------------------------------------------- 4-bit cache
def encode(y):
    """e2m1 codes of 64-bit values with |y| <= 6, to nearest, ties to even."""
    a = np.abs(y)
    mid = (GRID[1:] + GRID[:-1]) / 2
    up, down = np.searchsorted(mid, a, side="right"), np.searchsorted(mid, a, side="left")
    c = np.where(up % 2 == 0, up, down)
    return (c + np.where(np.signbit(y), 8, 0)).astype(np.uint8)


def kv_write(codes, scales, x, slots):
    """codes [blocks, bs, heads, dim / 2] and scales [blocks, heads, dim / 32,
    bs] uint8 arrays, changed in place; x [N, heads, dim] 64-bit, slots [N]."""
    blocks, bs, heads, half = codes.shape
    for i, s in enumerate(int(v) for v in slots):
        if not 0 <= s < blocks * bs:
            continue
        for h in range(heads):
            for g in range(half // 16):
                y = x[i, h, 32 * g:32 * g + 32]
                if not np.isfinite(y).all():
                    e, c = 128, np.zeros(32, np.uint8)
                else:
                    fr, ex = math.frexp(np.abs(y).max())
                    e = max(E_MIN, ex - 3 + (fr > 0.75)) if fr > 0 else E_MIN
                    c = encode(y * 2.0 ** -e)
                codes[s // bs, s % bs, h, 16 * g:16 * g + 16] = c[0::2] | (c[1::2] << 4)
                scales[s // bs, h, g, s % bs] = e + 127


def kv_values(codes, scales, slots):
    """Values [N, heads, dim] at slots, zeros outside the cache."""
    blocks, bs, heads, half = codes.shape
    slots = np.asarray(slots)
    on = (slots >= 0) & (slots < blocks * bs)
    s = np.where(on, slots, 0)
    c = codes[s // bs, s % bs]
    c = np.stack([c & 15, c >> 4], -1).reshape(len(s), heads, 2 * half)
    e = scales[s // bs, :, :, s % bs].astype(np.float64) - 127
    v = np.where(c >= 8, -1.0, 1.0) * GRID[c & 7] * np.repeat(2.0 ** e, 32, axis=-1)
    v[np.repeat(e == 128, 32, axis=-1)] = np.nan
    return np.where(on[:, None, None], v, 0.0)


def random_cache(blocks, bs, heads, dim, seed, order="heads"):
    """Filled codes and scales as CPU tensors: (k, v, k_scale, v_scale)."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(2):
        shape = (blocks, heads, bs, dim // 2) if order == "heads" else (blocks, bs, heads, dim // 2)
        t = torch.randint(0, 256, shape, generator=g).to(torch.uint8)
        out.append(t.transpose(1, 2) if order == "heads" else t)
    for _ in range(2):
        out.append(torch.randint(124, 129, (blocks, heads, dim // 32, bs), generator=g).to(torch.uint8))
    return out


def up(t):
    """A copy on the GPU with the tensor's strides."""
    return torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda").copy_(t)


def attention(q, codes, k_scale, v_codes, v_scale, block_table, q_start, ctx_len, scale, window=0, sinks=None):
    """out [N, Hq, D], lse [N, Hq] (NaN rows: not computed), and their
    tolerances: scores are a sum of D products in 32 bits, |ds| <= 2 D U scale
    sum|q k|, with two more roundings of the scaled score; weights in bf16 for
    the second product: half a step, 2^-8, each; the output's own half step."""
    N, Hq, D = q.shape
    blocks, bs, heads = codes.shape[:3]
    G = Hq // heads
    out, lse = np.full((N, Hq, D), np.nan), np.full((N, Hq), np.nan)
    otol, ltol = np.zeros((N, Hq, D)), np.zeros((N, Hq))
    q = q.double().numpy()
    for b in range(len(ctx_len)):
        q0, q1, L = int(q_start[b]), int(q_start[b + 1]), int(ctx_len[b])
        pos = np.arange(L)
        phys = np.asarray(block_table[b])[pos // bs] if L else np.zeros(0, np.int64)
        there = (phys >= 0) & (phys < blocks)
        slots = np.where(there, phys.astype(np.int64) * bs + pos % bs, -1)
        K, V = kv_values(codes, k_scale, slots), kv_values(v_codes, v_scale, slots)
        for i in range(q1 - q0):
            p = L - (q1 - q0) + i
            see = there & (pos <= p)
            if window:
                see &= pos > p - window
            for h in range(Hq):
                k, v = K[see, h // G], V[see, h // G]
                s = (k @ q[q0 + i, h]) * scale
                tops = list(s) + ([float(sinks[h])] if sinks is not None else [])
                if not tops:
                    out[q0 + i, h], lse[q0 + i, h] = 0.0, -np.inf
                    continue
                m = max(tops)
                w = np.exp(s - m)
                l = w.sum() + (math.exp(float(sinks[h]) - m) if sinks is not None else 0.0)
                w = w / l
                out[q0 + i, h] = w @ v if len(s) else 0.0
                lse[q0 + i, h] = m + math.log(l)
                ds = 2 * D * U * abs(scale) * (np.abs(k) @ np.abs(q[q0 + i, h])).max() if len(s) else 0.0
                ds += 8 * U * (np.abs(s).max() if len(s) else 0.0) + 8 * U * abs(m) + 64 * U
                mag = np.abs(v).T @ w if len(s) else 0.0
                otol[q0 + i, h] = 2.0 ** -8 * (np.abs(out[q0 + i, h]) + mag) + 2 * ds * mag + 1e-30
                ltol[q0 + i, h] = ds + 2 * U * abs(lse[q0 + i, h])
    return out, lse, otol, ltol


# single tokens of a full card of contexts: a unit each, four heads to a workgroup
MANY_SHORT = dict(name="full_card_of_4_bits", lens=[1] * 520, ctx=[1025 + i * 977 % 3001 for i in range(520)], G=1,
                  heads=16, dim=32, bs=16, max_ctx=4096, order="tokens", window=0, holes=True)
