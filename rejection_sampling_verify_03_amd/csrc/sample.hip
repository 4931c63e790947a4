// sample.hip -- tokens from distributions cut by top k, top p and min p, and
// the same cut applied to logits, on gfx950.
//
// With m a row's largest logit, w_v = exp((x_v - m) / T), and the tokens in the
// order of falling logits (equal ones: the lower index first), a row keeps the
// shortest of three prefixes of that order: the first top_k; the tokens in front
// of which less than top_p of the first top_k's sum of w stands; those with
// w >= min_p.  A token is the first one, by index, whose sum of kept w up to and
// with itself is above u times the sum of all.
//
// Whole numbers decide.  A token is a border found in sums of up to V weights,
// and fp32 sums would often put it one place off; so a weight is a whole number
// of 2^-P.frac, from an fp64 exponential rounded once (an error of 2^-46 of the
// largest weight for 2^17 tokens), and sums of whole numbers do not depend on
// their order: histograms by atomic additions in LDS give the same bits every
// time.
//
// Three kernels, the first reads each row once:
//
//  cut_stats   a wave to a segment of 4096 logits: the largest logit of each
//      cell (the 64 logits of a lane), of the segment, whether there is a NaN,
//      and where no top_k bounds the row the sum of its weights (fp64).
//
//  cut_finish  a workgroup to a row.  The k-th largest cell bounds the k-th
//      largest logit from below, so only the cells above it are read again, and
//      their logits above the bound (a few more than k) are candidates in LDS.
//      Every border is then found by a radix search: a histogram of the weights
//      (or of ones) over 2048 ranges of the key, a scan for the range in which
//      the sum crosses the border, and so on inside it.  The key is the place
//      in the order (distance of the logit from the largest, then the index), or
//      the index for the token.  Where the candidates are too many for LDS, the
//      same searches go over the row itself, and continue in LDS inside the range found.
//
//  truncate    writes the row, with -inf behind the last kept token.
#include <limits.h>

#include "ops_kernels.hpp"
#include "unaligned.hpp"

namespace specv {

constexpr int kCutThreads = 1024;             // of cut_finish
constexpr int kCutWaves = kCutThreads / 64;
constexpr int kBins = 2048;
constexpr int kCand = 4096;                   // candidates held in LDS
constexpr int kGuess = 512;                   // cells taken at first where only the mass bounds the row
typedef unsigned long long u64;

// What a request asks for.
struct Cut {
  float T, p, mn;
  int k;          // 0: all
  bool ok;        // usable
  bool greedy, all;  // T = 0; nothing is left out
  bool mass;      // the sum of all weights is needed
};

__device__ __forceinline__ Cut cut_of(const CutParams& P, int b) {
  Cut c;
  c.T = P.temperature[b];
  c.k = P.top_k ? P.top_k[b] : 0;
  c.p = P.top_p ? P.top_p[b] : 1.0f;
  c.mn = P.min_p ? P.min_p[b] : 0.0f;
  c.ok = temperature_valid(c.T) && c.k >= 0 && c.p > 0.0f && c.mn >= 0.0f && c.mn <= 1.0f;
  if (c.k >= P.V) c.k = 0;
  c.greedy = c.T == 0.0f;
  c.all = c.k == 0 && c.p >= 1.0f && c.mn == 0.0f;
  c.mass = !c.greedy && c.k == 0 && (c.p < 1.0f || c.mn == 0.0f);
  return c;
}

// The row's logits, or null where its entry of the row table is outside.
__device__ __forceinline__ const char* row_of(const CutParams& P, int b, int r, int es) {
  if (P.row_index) {
    const int row = P.row_index[(int64_t)b * P.R + r];
    return row >= 0 && row < P.rows ? P.logits + (int64_t)row * P.row * es : nullptr;
  }
  return P.logits + ((int64_t)b * P.req + (int64_t)r * P.row) * es;
}

// 2^(t + add) for t <= 0 (from -1100 on as 0 for every add below 48): by the
// nearest whole exponent and the power series of 2^f, |f| <= 1/2, whose terms
// left out are below 2^-47 of it.
__device__ __forceinline__ double pow2(double t, int add) {
  constexpr double L = 0.693147180559945309417;
  constexpr double c2 = L * L / 2, c3 = c2 * L / 3, c4 = c3 * L / 4, c5 = c4 * L / 5, c6 = c5 * L / 6, c7 = c6 * L / 7,
                   c8 = c7 * L / 8, c9 = c8 * L / 9, c10 = c9 * L / 10, c11 = c10 * L / 11;
  t = fmax(t, -1100.0);
  const double n = __builtin_rint(t), f = t - n;
  double y = c11;
  y = __builtin_fma(y, f, c10);
  y = __builtin_fma(y, f, c9);
  y = __builtin_fma(y, f, c8);
  y = __builtin_fma(y, f, c7);
  y = __builtin_fma(y, f, c6);
  y = __builtin_fma(y, f, c5);
  y = __builtin_fma(y, f, c4);
  y = __builtin_fma(y, f, c3);
  y = __builtin_fma(y, f, c2);
  y = __builtin_fma(y, f, L);
  y = __builtin_fma(y, f, 1.0);
  return ldexp(y, (int)n + add);
}

// A value below 2^52 as a whole number, rounded to nearest.
__device__ __forceinline__ u64 whole(double y) {
  return (u64)__double_as_longlong(y + 0x1p52) & ((1ull << 52) - 1);
}

// The place of a logit among all values of its type, larger for a larger one
// (-0 as +0): 16 bits of a bf16, 32 of an fp32.
template <int ES>
__device__ __forceinline__ uint32_t place(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  const uint32_t o = u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
  return ES == 2 ? o >> 16 : o;
}
template <int ES>
__device__ __forceinline__ float value_at(uint32_t o) {
  if (ES == 2) o <<= 16;
  if (ES == 2 && !(o >> 31)) o |= 0xffffu;  // (a negative bf16's low half is all ones here)
  return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}

// ------------------------------------------------------------- statistics --
template <int ES>
__device__ __forceinline__ uint32_t magnitude(const RawGroup<ES, true>& g) {  // the largest, as bits
  uint32_t a = 0;
  if constexpr (ES == 2) {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 m{0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, g.v[i] & 0x7fff7fffu));
    a = (uint32_t)(m.x > m.y ? m.x : m.y) << 16;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      a = max(max(a, __float_as_uint(g.a[i]) & 0x7fffffffu), __float_as_uint(g.b[i]) & 0x7fffffffu);
  }
  return a;
}

// 8 logits from e on, -inf past the row's end.
template <int ES>
__device__ __forceinline__ RawGroup<ES, true> load_end(const char* lg, int64_t e, int V) {
  if (e + 8 <= V) return load_any<ES>(lg, e);
  RawGroup<ES, true> g = neg_inf_group<ES, true>();
  if constexpr (ES == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (e + i < V) {
        const uint32_t w = load_bits<2>(lg, e + i);
        g.v[i >> 1] = (i & 1) ? (g.v[i >> 1] & 0xffffu) | (w << 16) : (g.v[i >> 1] & 0xffff0000u) | w;
      }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (e + i < V) g.a[i] = load_one<4>(lg, e + i);
      if (e + 4 + i < V) g.b[i] = load_one<4>(lg, e + 4 + i);
    }
  }
  return g;
}

// x to the 8 places from e on that the row has (values of the type).
template <int ES>
__device__ __forceinline__ void store_end(char* dst, int64_t e, int V, const float x[8]) {
  if constexpr (ES == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = (__float_as_uint(x[2 * i]) >> 16) | (__float_as_uint(x[2 * i + 1]) & 0xffff0000u);
    if (e + 8 <= V) {
      *reinterpret_cast<u32x4_any*>(dst + e * 2) = u32x4{w[0], w[1], w[2], w[3]};
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (e + i < V) reinterpret_cast<uint16_t*>(dst)[e + i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
  } else {
    if (e + 8 <= V) {
      *reinterpret_cast<f32x4_any*>(dst + e * 4) = f32x4{x[0], x[1], x[2], x[3]};
      *reinterpret_cast<f32x4_any*>(dst + e * 4 + 16) = f32x4{x[4], x[5], x[6], x[7]};
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (e + i < V) reinterpret_cast<float*>(dst)[e + i] = x[i];
  }
}

template <int ES>
__global__ __launch_bounds__(kWG) void cut_stats_kernel(CutParams P) {
  const int i = (int)P.by_C.of(blockIdx.x), chunk = blockIdx.x - i * P.C;
  const int b = (int)P.by_R.of((uint32_t)i), r = i - b * P.R;
  const Cut cut = cut_of(P, b);
  if (!cut.ok || (P.tokens == nullptr && (cut.greedy || cut.all))) return;  // (the finish does not read them)
  const char* lg = row_of(P, b, r, ES);
  if (!lg) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int j1 = min(P.nseg, (chunk + 1) * kCutChunkSegs);
  const double s = cut.mass ? 1.4426950408889634074 / (double)cut.T : 0.0;
  for (int j = chunk * kCutChunkSegs + wave; j < j1; j += kWaves) {
    const int64_t s0 = (int64_t)j * kSeg;
    RawGroup<ES, true> g[kSegGroups];
    if (s0 + kSeg <= P.V) {  // eight loads in a row, none under a branch
#pragma unroll
      for (int q = 0; q < kSegGroups; ++q) g[q] = load_any<ES>(lg, s0 + (q * 64 + lane) * 8);
    } else {
#pragma unroll
      for (int q = 0; q < kSegGroups; ++q) g[q] = load_end<ES>(lg, s0 + (q * 64 + lane) * 8, P.V);
    }
    float gm = -INFINITY;
    uint32_t big = 0;
#pragma unroll
    for (int q = 0; q < kSegGroups; ++q) {
      float x[8];
      unpack_group<ES, true>(g[q], x);
#pragma unroll
      for (int e = 0; e < 8; ++e) gm = fmaxf(gm, x[e]);
      big = max(big, magnitude<ES>(g[q]));
    }
    P.cells[((int64_t)i * P.nseg + j) * 64 + lane] = gm;
    CutRecord rec{wave_max_f(gm), __ballot(big > 0x7f800000u) != 0 ? 1 : 0, 0.0};
    if (cut.mass && rec.m > -INFINITY) {
      const double m = rec.m;
      double sum = 0.0;
#pragma unroll 1
      for (int q = 0; q < kSegGroups; ++q) {
        float x[8];
        unpack_group<ES, true>(g[q], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += pow2(((double)x[e] - m) * s, 0);
      }
      rec.s = wave_total_d(sum);
    }
    if (lane == 0) P.rec[(int64_t)i * P.nseg + j] = rec;
  }
}

// --------------------------------------------------------------- searches --
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ u64 dpp_u64(u64 x) {  // fill 0
  const uint32_t lo = (uint32_t)dpp_i<CTRL, ROW_MASK>((int)(uint32_t)x, 0);
  const uint32_t hi = (uint32_t)dpp_i<CTRL, ROW_MASK>((int)(uint32_t)(x >> 32), 0);
  return ((u64)hi << 32) | lo;
}
__device__ __forceinline__ u64 wave_scan_u64(u64 x) {  // inclusive, in lane order
  x += dpp_u64<0x111, 0xf>(x);
  x += dpp_u64<0x112, 0xf>(x);
  x += dpp_u64<0x114, 0xf>(x);
  x += dpp_u64<0x118, 0xf>(x);
  x += dpp_u64<0x142, 0xa>(x);
  x += dpp_u64<0x143, 0xc>(x);
  return x;
}

struct CutShared {
  u64 hist[kBins];
  u64 cand[kCand];      // keys of rank
  u64 wave[kCutWaves];
  double wave_d[kCutWaves];
  float wave_f[kCutWaves];
  u64 before, total, lo, hi;
  int bin, count;
  uint32_t far;
};

// A border: the smallest prefix whose weight reaches it.
struct Border {
  enum Kind { kFixed, kShare, kAbove } kind;
  u64 fixed;      // kFixed
  double share;   // kShare: of the total, rounded up (at least 1); kAbove: the first whole number above share * total
  __device__ u64 of(u64 total) const {
    if (kind == kFixed) return fixed;
    const double y = share * (double)total;
    return kind == kShare ? max((u64)ceil(y), 1ull) : (u64)y + 1;
  }
};

// What the searches of a row share.
struct RowView {
  const char* lg;
  int V, ibits, frac;
  float m;
  uint32_t top;  // place of m
  double s;      // log2(e) / T
};

// The key of rank of logit x at index e: 0.. for the row's largest.
template <int ES>
__device__ __forceinline__ u64 rank_key(const RowView& w, float x, int e) {
  return ((u64)(w.top - place<ES>(x)) << w.ibits) | (uint32_t)e;
}
template <int ES>
__device__ __forceinline__ float key_logit(const RowView& w, u64 key) {
  return value_at<ES>(w.top - (uint32_t)(key >> w.ibits));
}
template <bool MASS>
__device__ __forceinline__ u64 weight_of(const RowView& w, float x) {
  return MASS ? whole(pow2(((double)x - (double)w.m) * w.s, w.frac)) : 1;
}

struct Crossing {
  int bin;  // -1: the border is above the total
  u64 before, total, border;
};

// The range of the histogram in which the sum reaches the border (all threads;
// the histogram is complete when it is called, and free when it returns).
__device__ __forceinline__ Crossing find_crossing(CutShared& S, const Border& border, u64 offset) {
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  __syncthreads();
  const u64 h0 = S.hist[2 * t], h1 = S.hist[2 * t + 1], v = h0 + h1;
  const u64 x = wave_scan_u64(v);
  if (lane == 63) S.wave[wave] = x;
  if (t == 0) S.bin = -1;
  __syncthreads();
  u64 base = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kCutWaves; ++w) {
    const u64 y = S.wave[w];
    base += w < wave ? y : 0;
    total += y;
  }
  const u64 at = border.of(total) - offset, before = base + x - v;
  if (before < at && at <= before + v) {
    S.bin = at <= before + h0 ? 2 * t : 2 * t + 1;
    S.before = at <= before + h0 ? before : before + h0;
  }
  __syncthreads();
  const Crossing c{S.bin, S.before, total, at + offset};
  __syncthreads();
  return c;
}

__device__ __forceinline__ void clear_hist(CutShared& S) {
  S.hist[threadIdx.x] = 0;
  S.hist[threadIdx.x + kCutThreads] = 0;
  __syncthreads();
}

constexpr u64 kNone = ~0ull;

__device__ __forceinline__ int bits_of(u64 x) { return 64 - __clzll((long long)x); }

// Among the candidates in LDS with a key of rank up to `last`, the key (of
// rank, or the index) at which the sum of weights (or the count) reaches the
// border; kNone if it never does.  Keys lie in [lo, hi]; `offset` stands in
// front of them.
template <int ES, bool INDEX, bool MASS>
__device__ __forceinline__ u64 search_lds(CutShared& S, const RowView& w, int n, u64 last, u64 lo, u64 hi, Border border,
                          u64 offset) {
  for (;;) {
    const int shift = max(bits_of(hi - lo) - 11, 0);
    clear_hist(S);
    for (int i = threadIdx.x; i < n; i += kCutThreads) {
      const u64 rank = S.cand[i];
      const u64 key = INDEX ? rank & ((1ull << w.ibits) - 1) : rank;
      if (rank <= last && key >= lo && key <= hi)
        atomicAdd(&S.hist[(key - lo) >> shift], weight_of<MASS>(w, key_logit<ES>(w, rank)));
    }
    const Crossing c = find_crossing(S, border, offset);
    if (c.bin < 0) return kNone;
    border = Border{Border::kFixed, c.border, 0.0};
    offset += c.before;
    lo += (u64)c.bin << shift;
    if (shift == 0) return lo;
    hi = min(hi, lo + (1ull << shift) - 1);
  }
}

// f(x, e) for every logit of the row.
template <int ES, class F>
__device__ __forceinline__ void each_logit(const RowView& w, F f) {
  constexpr int kAhead = ES == 2 ? 4 : 2;
  const int groups = (w.V + 7) >> 3;
  for (int g0 = threadIdx.x; g0 < groups; g0 += kCutThreads * kAhead) {
    RawGroup<ES, true> raw[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int g = g0 + q * kCutThreads;
      if (g < groups) raw[q] = load_end<ES>(w.lg, (int64_t)g * 8, w.V);
    }
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int g = g0 + q * kCutThreads;
      if (g >= groups) break;
      float x[8];
      unpack_group<ES, true>(raw[q], x);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (g * 8 + e < w.V) f(x[e], g * 8 + e);
    }
  }
}

// Candidates gathered into LDS, with the range of their keys.
struct Gather {
  u64 lo = kNone, hi = 0;
  __device__ __forceinline__ void take(CutShared& S, u64 rank, u64 key) {
    const int at = atomicAdd(&S.count, 1);
    if (at < kCand) S.cand[at] = rank;
    lo = min(lo, key);
    hi = max(hi, key);
  }
};
__device__ __forceinline__ void gather_begin(CutShared& S) {
  if (threadIdx.x == 0) {
    S.count = 0;
    S.lo = kNone;
    S.hi = 0;
  }
  __syncthreads();
}
__device__ __forceinline__ void gather_end(CutShared& S, const Gather& g) {
  if (g.lo <= g.hi) {
    atomicMin(&S.lo, g.lo);
    atomicMax(&S.hi, g.hi);
  }
  __syncthreads();
}

// search_lds over the row itself: a histogram of all its logits, the logits of
// the range found gathered into LDS, and so on there.  `span`: the first
// histogram over ranks has its ranges evenly over logits from m down to m -
// span (all below in the last).
template <int ES, bool INDEX, bool MASS>
__device__ __forceinline__ u64 search_row(CutShared& S, const RowView& w, u64 last, float span, Border border) {
  const float inv = INDEX ? 0.f : fminf((float)(kBins - 1) / span, FLT_MAX);
  const int ishift = max(w.ibits - 11, 0);
  auto bin_of = [&](float x, int e) {
    if constexpr (INDEX) return e >> ishift;
    return (int)fminf((w.m - x) * inv, (float)(kBins - 1));
  };
  clear_hist(S);
  if constexpr (INDEX) {  // a group's logits mostly have one range
    u64 sum = 0;
    int at = -1;
    each_logit<ES>(w, [&](float x, int e) {
      const int bin = bin_of(x, e);
      if (bin != at) {
        if (sum) atomicAdd(&S.hist[at], sum);
        sum = 0;
        at = bin;
      }
      if (rank_key<ES>(w, x, e) <= last) sum += weight_of<MASS>(w, x);
    });
    if (sum) atomicAdd(&S.hist[at], sum);
  } else {
    each_logit<ES>(w, [&](float x, int e) {
      if (rank_key<ES>(w, x, e) <= last) {
        const u64 q = weight_of<MASS>(w, x);
        if (q) atomicAdd(&S.hist[bin_of(x, e)], q);
      }
    });
  }
  Crossing c = find_crossing(S, border, 0);
  if (c.bin < 0) return kNone;
  border = Border{Border::kFixed, c.border, 0.0};
  u64 offset = c.before;
  const int bin = c.bin;
  gather_begin(S);
  Gather g;
  each_logit<ES>(w, [&](float x, int e) {
    const u64 rank = rank_key<ES>(w, x, e);
    if (rank <= last && bin_of(x, e) == bin) g.take(S, rank, INDEX ? (u64)e : rank);
  });
  gather_end(S, g);
  u64 lo = S.lo, hi = S.hi;
  int n = S.count;
  while (n > kCand) {  // (many equal logits) the range's keys in finer ranges, over the row again
    const int shift = max(bits_of(hi - lo) - 11, 0);
    clear_hist(S);
    each_logit<ES>(w, [&](float x, int e) {
      const u64 rank = rank_key<ES>(w, x, e), key = INDEX ? (u64)e : rank;
      if (rank <= last && key >= lo && key <= hi) {
        const u64 q = weight_of<MASS>(w, x);
        if (q) atomicAdd(&S.hist[(key - lo) >> shift], q);
      }
    });
    c = find_crossing(S, border, offset);
    if (c.bin < 0) return kNone;
    offset += c.before;
    lo += (u64)c.bin << shift;
    hi = min(hi, lo + (1ull << shift) - 1);
    gather_begin(S);
    Gather h;
    each_logit<ES>(w, [&](float x, int e) {
      const u64 rank = rank_key<ES>(w, x, e), key = INDEX ? (u64)e : rank;
      if (rank <= last && key >= lo && key <= hi) h.take(S, rank, key);
    });
    gather_end(S, h);
    lo = max(lo, S.lo);
    hi = min(hi, S.hi);
    n = S.count;
  }
  return search_lds<ES, INDEX, MASS>(S, w, n, last, lo, hi, border, offset);
}

// Reductions over the workgroup, the same in every thread.
__device__ __forceinline__ float block_max_f(CutShared& S, float x) {
  x = wave_max_f(x);
  if ((threadIdx.x & 63) == 0) S.wave_f[threadIdx.x >> 6] = x;
  __syncthreads();
  float y = S.wave_f[0];
#pragma unroll
  for (int w = 1; w < kCutWaves; ++w) y = fmaxf(y, S.wave_f[w]);
  __syncthreads();
  return y;
}
__device__ __forceinline__ double block_sum_d(CutShared& S, double x) {
  x = wave_total_d(x);
  if ((threadIdx.x & 63) == 0) S.wave_d[threadIdx.x >> 6] = x;
  __syncthreads();
  double y = 0.0;
#pragma unroll
  for (int w = 0; w < kCutWaves; ++w) y += S.wave_d[w];
  __syncthreads();
  return y;
}

// ----------------------------------------------------------------- finish --
template <int ES, bool DRAW>
__global__ __launch_bounds__(kCutThreads) void cut_finish_kernel(CutParams P) {
  __shared__ CutShared S;
  const int i = blockIdx.x, tid = threadIdx.x;
  const int b = (int)P.by_R.of((uint32_t)i), r = i - b * P.R;
  const Cut cut = cut_of(P, b);
  const float u = DRAW ? P.uniforms[i] : 0.f;
  RowView w;
  w.lg = row_of(P, b, r, ES);
  w.V = P.V;
  w.ibits = P.ibits;
  w.frac = P.frac;
  auto end = [&](int token, u64 last) {  // of the row
    if (tid == 0) {
      if constexpr (DRAW)
        P.tokens[i] = token;
      else
        P.last[i] = last;
    }
  };
  if (!cut.ok || !w.lg || (DRAW && !(u >= 0.0f && u < 1.0f))) return end(-1, kCutBad);
  if (!DRAW && (cut.greedy || cut.all)) return end(-1, kCutAll);
  const CutRecord* rec = P.rec + (int64_t)i * P.nseg;
  float m = -INFINITY;
  bool nan = false;
  for (int j = tid; j < P.nseg; j += kCutThreads) {
    const CutRecord q = rec[j];
    m = fmaxf(m, q.m);
    nan |= q.nan != 0;
  }
  m = block_max_f(S, m);
  nan = __syncthreads_or(nan);
  if (cut.greedy ? m == -INFINITY : nan || !(fabsf(m) <= FLT_MAX)) return end(cut.greedy ? 0 : -1, kCutAll);
  w.m = m;
  w.top = place<ES>(m);
  w.s = cut.greedy ? 0.0 : 1.4426950408889634074 / (double)cut.T;
  const u64 index_mask = (1ull << w.ibits) - 1;
  const float reach = (float)fmin((w.frac + 2) / fmax(w.s, 1e-300), (double)FLT_MAX);  // (no weight beyond)

  if (DRAW && cut.all && !cut.greedy) {
    // nothing left out: the segment from the segments' sums, then the token in it
    auto units = [&](int j) { return (u64)ldexp(rec[j].s * pow2(((double)rec[j].m - (double)m) * w.s, 0), w.frac); };
    int lo = 0, hi = P.nseg - 1;
    u64 offset = 0;
    Border at{Border::kAbove, 0, (double)u};
    for (;;) {
      const int shift = max(bits_of((u64)(hi - lo)) - 11, 0);
      clear_hist(S);
      for (int j = lo + tid; j <= hi; j += kCutThreads) atomicAdd(&S.hist[(j - lo) >> shift], units(j));
      const Crossing c = find_crossing(S, at, offset);
      at = Border{Border::kFixed, c.border, 0.0};
      offset += c.before;
      lo += c.bin << shift;
      if (shift == 0) break;
      hi = min(hi, lo + (1 << shift) - 1);
    }
    // in the segment the weights count from its own largest, 4096 of them in 62 bits
    constexpr int kSegFrac = 50;
    const double far = pow2(((double)rec[lo].m - (double)m) * w.s, 0);
    const double rest = ldexp((double)(at.fixed - offset), kSegFrac - w.frac) / far;
    w.m = rec[lo].m;
    w.top = place<ES>(w.m);
    w.frac = kSegFrac;
    const int first = lo * kSeg, n = min(kSeg, P.V - first);
    gather_begin(S);
    u64 sum = 0;
    for (int e = tid; e < n; e += kCutThreads) {
      const float x = load_one<ES>(w.lg, first + e);
      S.cand[e] = rank_key<ES>(w, x, first + e);
      sum += weight_of<true>(w, x);
    }
    if (sum) atomicAdd(&S.hi, sum);
    __syncthreads();
    // (the segment's sum of rounded weights may fall short of the place found)
    const u64 border = min(max((u64)ceil(fmin(rest, 0x1p62)), 1ull), S.hi);
    __syncthreads();
    const u64 e = search_lds<ES, true, true>(S, w, n, kNone, first, first + n - 1, Border{Border::kFixed, border, 0.0}, 0);
    return end((int)e, 0);
  }

  const int k = cut.greedy ? 1 : cut.k;
  const float p = cut.greedy ? 1.0f : cut.p;
  // how far (in places) from the largest logit the kept ones can be
  uint32_t min_far = ~0u;  // by min_p
  if (!cut.greedy && cut.mn > 0.0f) {
    const double low = (double)m + (double)cut.T * log((double)cut.mn);
    const float f = fmaxf(__double2float_ru(low), -FLT_MAX);
    uint32_t q = place<ES>(f);
    if (ES == 2 && value_at<2>(q) < f) ++q;  // (the bf16 values not below it)
    min_far = w.top - min(q, w.top);
  }
  // by the k-th largest cell, or where only the mass bounds the row, by a number of cells that mostly hold it
  const float* cells = P.cells + (int64_t)i * P.nseg * 64;
  const int ncell = P.nseg * 64;
  const int want = k > 0 ? k : p < 1.0f ? min(kGuess, ncell) : 0;
  uint32_t cell_far = ~0u;
  if (want > 0 && want <= ncell) {
    float least = INFINITY;
    for (int c = tid; c < ncell; c += kCutThreads) {
      const float x = cells[c];
      least = fminf(least, x > -INFINITY ? x : INFINITY);
    }
    least = -block_max_f(S, -least);
    const float inv = fminf((float)(kBins - 1) / (m - least), FLT_MAX);  // (0 / 0 for equal cells: range 0)
    clear_hist(S);
    auto bin_of = [&](float x) { return (int)fmaxf(fminf((m - x) * inv, (float)(kBins - 1)), 0.f); };
    for (int c = tid; c < ncell; c += kCutThreads) atomicAdd(&S.hist[bin_of(cells[c])], 1ull);
    const Crossing c = find_crossing(S, Border{Border::kFixed, (u64)want, 0.0}, 0);
    if (tid == 0) S.far = 0;
    __syncthreads();
    uint32_t far = 0;
    for (int j = tid; j < ncell; j += kCutThreads)
      if (bin_of(cells[j]) <= c.bin) far = max(far, w.top - place<ES>(cells[j]));
    if (far) atomicMax(&S.far, far);
    __syncthreads();
    cell_far = S.far;
  }
  // (a top_p of a top_k is a share of all its tokens, min_p or not)
  const bool by_min = !(k > 0 && p < 1.0f);
  const uint32_t far = by_min ? min(cell_far, min_far) : cell_far;
  bool held = false;
  gather_begin(S);
  if (far != ~0u) {
    Gather g;
    for (int c = tid; c < ncell; c += kCutThreads) {
      const float x = cells[c];
      if (!(x >= -FLT_MAX) && !(x == m)) continue;
      if (w.top - place<ES>(x) > far) continue;
      const int s0 = (c >> 6) * kSeg + (c & 63) * 8;
      RawGroup<ES, true> raw[kSegGroups];
#pragma unroll
      for (int q = 0; q < kSegGroups; ++q)
        raw[q] = s0 + q * 512 < P.V ? load_end<ES>(w.lg, (int64_t)s0 + q * 512, P.V) : neg_inf_group<ES, true>();
#pragma unroll 1
      for (int q = 0; q < kSegGroups; ++q) {
        float y[8];
        unpack_group<ES, true>(raw[q], y);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (y[e] <= m && w.top - place<ES>(y[e]) <= far && s0 + q * 512 + e < P.V) {
            const u64 key = rank_key<ES>(w, y[e], s0 + q * 512 + e);
            g.take(S, key, key);
          }
      }
    }
    gather_end(S, g);
    held = S.count <= kCand;
  }
  __syncthreads();
  const int n = S.count;
  const u64 lo = S.lo, hi = S.hi;
  __syncthreads();

  u64 last = held ? hi : kNone;  // the rank of the last kept token
  if (k > 0) {
    const Border at{Border::kFixed, (u64)k, 0.0};
    if (!held)
      last = search_row<ES, false, false>(S, w, cut.greedy ? index_mask : kNone, reach, at);
    else if (n > k)
      last = search_lds<ES, false, false>(S, w, n, kNone, lo, hi, at, 0);
  }
  if (cut.greedy) return end((int)(last & index_mask), 0);
  if (p < 1.0f) {
    u64 at = kNone;
    if (k > 0) {
      const Border border{Border::kShare, 0, (double)p};
      at = held ? search_lds<ES, false, true>(S, w, n, last, lo, hi, border, 0)
                : search_row<ES, false, true>(S, w, last, reach, border);
    } else {
      if (held) {
        double total = 0.0;
        for (int j = tid; j < P.nseg; j += kCutThreads)
          total += rec[j].s * pow2(((double)rec[j].m - (double)m) * w.s, 0);
        total = ldexp(block_sum_d(S, total), w.frac);
        const Border border{Border::kFixed, max((u64)ceil((double)p * total), 1ull), 0.0};
        at = search_lds<ES, false, true>(S, w, n, kNone, lo, hi, border, 0);
      }
      // (not among the candidates: behind them, which matters where min_p did not bound them)
      if (at == kNone && !(held && far == min_far)) {
        at = search_row<ES, false, true>(S, w, kNone, reach, Border{Border::kShare, 0, (double)p});
        last = kNone;
        held = false;
      }
    }
    last = min(last, at);
  }
  if (min_far != ~0u) last = min(last, ((u64)min_far << w.ibits) | index_mask);
  if constexpr (!DRAW) return end(0, last);
  const Border at{Border::kAbove, 0, (double)u};
  const u64 e = held ? search_lds<ES, true, true>(S, w, n, last, 0, (u64)P.V - 1, at, 0)
                     : search_row<ES, true, true>(S, w, last, 0.f, at);
  end((int)e, 0);
}

// --------------------------------------------------------------- truncate --
template <int ES>
__global__ __launch_bounds__(kWG) void truncate_kernel(CutParams P) {
  const int i = (int)P.by_C.of(blockIdx.x), chunk = blockIdx.x - i * P.C;
  const int b = (int)P.by_R.of((uint32_t)i), r = i - b * P.R;
  const u64 last = P.last[i];
  const char* src = P.logits + ((int64_t)b * P.req + (int64_t)r * P.row) * ES;
  char* dst = P.out + ((int64_t)b * P.out_req + (int64_t)r * P.out_row) * ES;
  if (last == kCutAll && src == dst) return;
  RowView w;
  w.ibits = P.ibits;
  w.top = 0;
  if (last < kCutAll) {
    float m = -INFINITY;
    const CutRecord* rec = P.rec + (int64_t)i * P.nseg;
    for (int j = threadIdx.x & 63; j < P.nseg; j += 64) m = fmaxf(m, rec[j].m);
    w.m = wave_max_f(m);
    w.top = place<ES>(w.m);
  }
  const float fill = last == kCutBad ? __builtin_nanf("") : -INFINITY;
  const int64_t e1 = min((int64_t)P.V, ((int64_t)chunk + 1) * kCutChunkSegs * kSeg);
  for (int64_t e = (int64_t)chunk * kCutChunkSegs * kSeg + threadIdx.x * 8; e < e1; e += kWG * 8) {
    RawGroup<ES, true> g = load_end<ES>(src, e, P.V);
    bool some = false;
    float x[8];
    unpack_group<ES, true>(g, x);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const bool keep = last == kCutAll || (last < kCutAll && rank_key<ES>(w, x[q], (int)e + q) <= last);
      some |= !keep;
      x[q] = keep ? x[q] : fill;
    }
    if (!some && src == dst) continue;
    store_end<ES>(dst, e, P.V, x);
  }
}

template <int ES>
static hipError_t launch_cut_typed(const CutParams& P, hipStream_t stream) {
  const unsigned rows = (unsigned)(P.B * P.R), chunks = rows * (unsigned)P.C;
  hipLaunchKernelGGL((cut_stats_kernel<ES>), dim3(chunks), dim3(kWG), 0, stream, P);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (P.tokens) {
    hipLaunchKernelGGL((cut_finish_kernel<ES, true>), dim3(rows), dim3(kCutThreads), 0, stream, P);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((cut_finish_kernel<ES, false>), dim3(rows), dim3(kCutThreads), 0, stream, P);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((truncate_kernel<ES>), dim3(chunks), dim3(kWG), 0, stream, P);
  return hipGetLastError();
}

hipError_t launch_cut(const CutParams& P, int dtype, hipStream_t stream) {
  return dtype == SPEC_BF16 ? launch_cut_typed<2>(P, stream) : launch_cut_typed<4>(P, stream);
}

}  // namespace specv
