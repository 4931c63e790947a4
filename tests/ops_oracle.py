"""Plain 64-bit implementations of the operators around a verification step,
from their definitions: token log probabilities, the 8-bit paged cache and the
attention over it.  CPU tensors in, CPU tensors out; the second value of the
computed operators is how far a kernel with 32-bit sums may be off."""
import math

import numpy as np
import torch

U = 2.0 ** -24  # half a step of fp32
E_MIN = -117


# ------------------------------------------------------------------ logprobs
def logprobs(logits, tokens, temperature, top):
    """(logprobs, entropy, ids, top logprobs), (tolerances of the three real
    ones).  The kernel's exponents t = (x - m) log2(e) / T carry three
    roundings (difference, scale, product), its 2^t one step and its sums a few
    more: dS / S <= sum p (3 ln2 |t| + 32) U, and so on for W."""
    B, R, V = logits.shape
    x = logits.double().numpy()
    lp, ent = np.zeros((B, R)), np.zeros((B, R))
    ids, tlp = np.full((B, R, top), -1, np.int64), np.zeros((B, R, top))
    tol, etol = np.zeros((B, R)), np.zeros((B, R))
    for b in range(B):
        T = 1.0 if temperature is None else float(temperature[b])
        ok_t = T == 0 or (math.isfinite(T) and T >= 2.0 ** -126)
        T = 1.0 if T == 0 else T
        for r in range(R):
            t = int(tokens[b, r])
            if t == -1:
                continue
            row = x[b, r]
            m = row.max()
            if not ok_t or not 0 <= t < V or not math.isfinite(m):
                lp[b, r] = ent[b, r] = np.nan
                tlp[b, r] = np.nan
                continue
            z = (row - m) / T
            p = np.exp(z)
            S = p.sum()
            p = p / S
            fin = np.isfinite(z)
            lp[b, r] = z[t] - math.log(S)
            zf = np.where(fin, z, 0.0)
            ent[b, r] = math.log(S) - (p * zf).sum()
            a1, a2 = (p * -zf).sum(), (p * zf * zf).sum()
            tol[b, r] = (3 * a1 + 32 + 2 * (abs(lp[b, r]) if np.isfinite(lp[b, r]) else 0)) * U
            # dH <= dS / S (1 + a1) + dW / S: S is summed in 32 bits together with the exact 1 of the row's
            # maximum, six sums deep in the lane that holds it (6 U, whatever the other logits are), and with
            # the others' own errors; W, to which the maximum adds 0, carries those alone
            etol[b, r] = (6 + 3 * a1 + 32 * (1 - p.max() + a1) + 3 * a2 + 3 * a1 + 2 * ent[b, r]) * U + 1e-13
            order = np.lexsort((np.arange(V), -row))[:top]
            order = order[np.isfinite(row[order])]
            n = len(order)
            ids[b, r, :n] = order
            tlp[b, r, n:] = -np.inf
            tlp[b, r, :n] = z[order] - math.log(S)
    # the outputs are fp32: what is past its largest value rounds to infinity
    for a in (lp, tlp):
        a[a <= -2.0 ** 128 * (1 - 2.0 ** -25)] = -np.inf
    return (lp, ent, ids, tlp), (tol, etol)


# --------------------------------------------------------------------- cache
def _decode_table():
    c = np.arange(256)
    e, m = c >> 3 & 15, (c & 7).astype(np.float64)
    mag = np.where(e > 0, (8 + m) * 2.0 ** (e - 10.0), m * 2.0 ** -9)
    v = np.where(c >= 128, -mag, mag)
    v[[0x7F, 0xFF]] = np.nan
    return v


DECODE = _decode_table()
_POS = DECODE[:127]


def encode(x):
    """e4m3 codes of 64-bit values with |x| <= 448, to nearest, ties to even."""
    a = np.abs(x)
    hi = np.searchsorted(_POS, np.where(np.isnan(a), 0, a), side="left").clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    dh, dl = _POS[hi] - a, a - _POS[lo]
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    c = np.where(np.isnan(a), 0x7F, c)
    return (c + np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def kv_write(codes, scales, x, slots, scale_tokens):
    """codes [blocks, bs, heads, dim] and scales [blocks, heads, groups] uint8
    arrays, changed in place; x [N, heads, dim] 64-bit, slots [N]."""
    blocks, bs, heads, _ = codes.shape
    groups = {}
    for i, s in enumerate(int(v) for v in slots):
        if 0 <= s < blocks * bs:
            groups.setdefault(s // scale_tokens, {})[s % scale_tokens] = i  # of equal slots the last
    for g, at in groups.items():
        blk, t0 = divmod(g * scale_tokens, bs)
        first = min(at)
        for h in range(heads):
            rows = np.stack([x[i, h] for i in at.values()])
            fin = rows[np.isfinite(rows)]
            amax = np.abs(fin).max() if fin.size else 0.0
            e = E_MIN
            if amax > 0:
                fr, ex = math.frexp(amax)
                e = max(E_MIN, ex - 9 + (fr > 0.875))
            if first > 0:
                old = int(scales[blk, h, t0 // scale_tokens]) - 127
                if e > old:
                    keep = codes[blk, t0:t0 + first, h]
                    keep[...] = encode(DECODE[keep] * 2.0 ** (old - e))
                else:
                    e = old
            for o, i in at.items():
                y = np.where(np.isfinite(x[i, h]), x[i, h], np.nan) * 2.0 ** -e
                codes[blk, t0 + o, h] = encode(y)
            scales[blk, h, t0 // scale_tokens] = e + 127


def kv_values(codes, scales, slots, scale_tokens):
    """Values [N, heads, dim] at slots, zeros outside the cache."""
    blocks, bs, heads, dim = codes.shape
    slots = np.asarray(slots)
    on = (slots >= 0) & (slots < blocks * bs)
    s = np.where(on, slots, 0)
    e = scales[s // bs, :, s % bs // scale_tokens].astype(np.float64) - 127
    with np.errstate(invalid="ignore"):
        v = DECODE[codes[s // bs, s % bs]] * 2.0 ** e[..., None]
    return np.where(on[:, None, None], v, 0.0)


def same_codes(a, b):
    """Codes that stand for the same values (any NaN as any NaN, -0 as 0)."""
    return np.array_equal(DECODE[a], DECODE[b], equal_nan=True)


# ----------------------------------------------------------------- attention
def attention(q, codes, k_scale, v_codes, v_scale, scale_tokens, block_table, q_start, ctx_len, scale, window=0,
              sinks=None):
    """out [N, Hq, D], lse [N, Hq] (NaN rows: not computed), and their
    tolerances.  Scores: a sum of D products in 32 bits, |ds| <= 2 D U scale
    sum|q k|, and two more roundings of the scaled score; weights in bf16 for
    the second product: half a step, 2^-8, each; the output's own half step."""
    N, Hq, D = q.shape
    heads = codes.shape[2]
    blocks, bs = codes.shape[:2]
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
        K = kv_values(codes, k_scale, slots, scale_tokens)
        V = kv_values(v_codes, v_scale, slots, scale_tokens)
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


def to_numpy(cache):
    return [t.cpu().numpy().copy() for t in (cache.k, cache.k_scale, cache.v, cache.v_scale)]


def random_cache(blocks, bs, heads, dim, st, seed, spread=4):
    """Filled codes and scales as CPU tensors: (k, v, k_scale, v_scale)."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(2):
        x = (torch.randn(blocks, bs, heads, dim, generator=g) * 90).clamp(-448, 448)
        out.append(x.to(torch.float8_e4m3fn).view(torch.uint8))
    for _ in range(2):
        out.append(torch.randint(120 - spread // 2, 121 + spread // 2, (blocks, heads, bs // st),
                                 generator=g).to(torch.uint8))
    return out
