// logprobs.hip -- log probabilities of given tokens, the entropy of their
// rows and the rows' most likely tokens, on gfx950.
//
// With x the row's logits, m its maximum, s = log2(e) / T and
// t_v = (x_v - m) * s:  S = sum 2^t_v,  W = sum 2^t_v t_v,
//   ln p(v) = (x_v - m) / T - ln S,   entropy = ln S - ln 2 * W / S,
// so one pass that keeps (m, S, W) gives both.  A lane sums its 64 terms in
// fp32, and so do the lanes of a segment; segments are joined in double.
//
// Two kernels, one read of each row whose logits are finite (a segment that
// holds one of -inf is read and summed a second time):
//
//  logprobs_stats   one 256-thread workgroup per (row, 8 segments), a wave per
//      4096-logit segment: the segment stays in registers while its maximum
//      is taken and then summed against it.  For the alternatives it also
//      writes the maximum of every cell of 64 consecutive logits, 1/64 of the
//      row.
//
//  logprobs_finish  one wave per row (for rows that one workgroup holds, its
//      first wave): merges the segments' records and finds
//      the alternatives through the cells: the n largest logits lie in the n
//      cells with the largest maxima (lower cell first on ties: a cell's
//      logits all stand in front of the next cell's).  A threshold that at
//      least n of the 64 lanes' maxima reach picks a few more than n cells,
//      whose logits are read again; those that reach it are sorted.
//
// Bounds, measured (MI355X): the statistics pass is bound by its vector
// instructions (a logit costs 8 of them and an exponential, which takes four
// slots; they fill 96 % of the slots) just above the rate of memory: 2304 rows
// of 151936 bf16 logits without alternatives take 123 us (6.4 TB/s), the 1327
// live rows of a verified batch with 5 alternatives 84 us (4.8 TB/s), of which
// the finish is 11 us, one wave's chain of steps: 4 to the joined sums, 3 to the
// threshold, the rest to find, read and sort the candidates.  Masked rows cost
// more: the same 1327 rows with a logit of -inf in every segment take 157 us,
// with 8 such logits to a row 106.  Segments of 4096 logits, as
// in draft.hip: 64 registers of logits a lane leave five waves to a SIMD.
// Four segments to a workgroup were 7 % slower there, sixteen 3 %.
#include <limits.h>

#include <type_traits>

#include "device_common.hpp"
#include "ops_kernels.hpp"
#include "unaligned.hpp"

namespace specv {

// x of another lane of the same 8 (every lane has a source: no fill).
template <int CTRL>
__device__ __forceinline__ float dpp_all(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(x), __float_as_int(x), CTRL, 0xf, 0xf, true));
}

// Lane i of each 8 gets the maximum of v[i] over the 8: the lanes exchange
// the half of the values that they do not keep, three times.
__device__ __forceinline__ float max8_scatter(const float (&v)[8], int lane) {
  float a[4], b[2];
  const bool h4 = lane & 4, h2 = lane & 2, h1 = lane & 1;
#pragma unroll
  for (int i = 0; i < 4; ++i)  // lane i with 7 - i
    a[i] = fmaxf(h4 ? v[i + 4] : v[i], dpp_all<0x141>(h4 ? v[i] : v[i + 4]));
#pragma unroll
  for (int i = 0; i < 2; ++i)  // quad [2, 3, 0, 1]
    b[i] = fmaxf(h2 ? a[i + 2] : a[i], dpp_all<0x4e>(h2 ? a[i] : a[i + 2]));
  return fmaxf(h1 ? b[1] : b[0], dpp_all<0xb1>(h1 ? b[0] : b[1]));  // quad [1, 0, 3, 2]
}

// Sum over the 64 lanes in a fixed order, the same in every lane.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ float add_dpp(float x) {
  return x + __int_as_float(dpp_i<CTRL, ROW_MASK>(__float_as_int(x), 0));
}
__device__ __forceinline__ float wave_total_f(float x) {
  x = add_dpp<0x111, 0xf>(x);
  x = add_dpp<0x112, 0xf>(x);
  x = add_dpp<0x114, 0xf>(x);
  x = add_dpp<0x118, 0xf>(x);
  x = add_dpp<0x142, 0xa>(x);
  x = add_dpp<0x143, 0xc>(x);
  return lane_f(x, 63);
}

__device__ __forceinline__ float row_temperature(const LogprobsParams& P, int b) {
  const float T = P.temperature ? P.temperature[b] : 1.0f;
  return T == 0.0f ? 1.0f : T;
}

// 8 logits as stored, with -inf for those past the end of the row.
template <int ES>
__device__ __forceinline__ RawGroup<ES, true> load_any_bounded(const char* row, int e0, int V) {
  if (e0 < V && e0 + 8 <= V) return load_any<ES>(row, e0);
  RawGroup<ES, true> r = neg_inf_group<ES, true>();
  if (e0 < V) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = e0 + i < V ? load_one<ES>(row, e0 + i) : -INFINITY;
    if constexpr (ES == 2) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = (__float_as_uint(x[2 * i]) >> 16) | (__float_as_uint(x[2 * i + 1]) & 0xffff0000u);
      r.v = u32x4{w[0], w[1], w[2], w[3]};
    } else {
      r.a = f32x4{x[0], x[1], x[2], x[3]};
      r.b = f32x4{x[4], x[5], x[6], x[7]};
    }
  }
  return r;
}

// The largest of 8 logits, three to an instruction (a NaN shows in S).
__device__ __forceinline__ float group_max(const float (&x)[8]) {
  const float a = fmaxf(fmaxf(x[0], x[1]), x[2]), b = fmaxf(fmaxf(x[3], x[4]), x[5]);
  return fmaxf(fmaxf(fmaxf(x[6], x[7]), a), b);
}

// What 8 exponents t add to S and W.
__device__ __forceinline__ void add_group(const float (&e)[8], const float (&t)[8], float& S, float& W) {
  S += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
  float a = e[0] * t[0], b = e[4] * t[4];
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    a = __builtin_fmaf(e[i], t[i], a);
    b = __builtin_fmaf(e[4 + i], t[4 + i], b);
  }
  W += a + b;
}

// A float's place in the order of floats as a signed integer (-0 as +0).
__device__ __forceinline__ int order_key(float x) {
  const int k = __float_as_int(x + 0.0f);
  return k < 0 ? (int)0x80000000 - k : k;
}
__device__ __forceinline__ float order_value(int k) {
  return __int_as_float(k < 0 ? (int)0x80000000 - k : k);
}

// A bound that at least n of the 64 * K keys of a wave reach (1 <= n <=
// 64 * K), and as few more as kSpare where the keys differ: the range below
// the largest key is widened until it holds n, then halved.
constexpr int kSpare = 8;
template <int K>
__device__ __forceinline__ int reach_bound(const int (&k)[K], int n) {
  auto count = [&](int bound) {
    int c = 0;
#pragma unroll
    for (int q = 0; q < K; ++q) c += __builtin_popcountll(__ballot(k[q] >= bound));
    return c;
  };
  int most = k[0];
#pragma unroll
  for (int q = 1; q < K; ++q) most = max(most, k[q]);
  int64_t hi = wave_max_i(most), lo = hi;
  int c = 0;
  for (int64_t step = 1 << 20;; step <<= 2) {  // an eighth of a power of two first
    lo = max(hi - step, (int64_t)INT_MIN);
    c = count((int)lo);
    if (c >= n) break;  // (at INT_MIN all 64 * K do)
    hi = lo - 1;
  }
  while (c > n + kSpare && lo < hi) {
    const int64_t mid = (lo + hi + 1) >> 1;
    const int m = count((int)mid);
    if (m >= n) {
      lo = mid;
      c = m;
    } else {
      hi = mid - 1;
    }
  }
  return (int)lo;
}

constexpr int kLpList = 256;  // candidates a wave can hold, 4 per lane

// Candidates in LDS, in ascending order of their ids: all whose key is above
// the threshold, and of those equal to it the first n.  What the list cannot
// hold is counted all the same.
struct LpList {
  int* keys;
  int* ids;
  int count, equal;  // appended (or past the end), of them equal to the threshold
};

__device__ __forceinline__ int lanes_below(uint64_t mask) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

// Appends from each lane Q items with consecutive ids from `id` on; lanes in
// ascending order hold ascending ids.
template <int Q>
__device__ __forceinline__ void collect(LpList& st, const int (&key)[Q], int id, int thr, int n) {
  int most = key[0];
#pragma unroll
  for (int q = 1; q < Q; ++q) most = max(most, key[q]);
  if (!__ballot(most >= thr)) return;
  int rank = st.equal, equal = 0;  // of this lane's first item among those equal to the threshold
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const uint64_t b = __ballot(key[q] == thr);
    rank += lanes_below(b);
    equal += __builtin_popcountll(b);
  }
  st.equal += equal;
  bool take[Q];
  int at = st.count;
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    take[q] = key[q] > thr || (key[q] == thr && rank < n);
    rank += key[q] == thr;
    const uint64_t b = __ballot(take[q]);
    at += lanes_below(b);
    st.count += __builtin_popcountll(b);
  }
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    if (take[q] && at < kLpList) {
      st.keys[at] = key[q];
      st.ids[at] = id + q;
    }
    at += take[q];
  }
}

// A bound that at least n of a full list's keys reach, and not all of them: a
// threshold above the one that the list was collected with.
__device__ __forceinline__ int raise_threshold(const int* keys, int lane, int n) {
  int k[kLpList / 64];
#pragma unroll
  for (int q = 0; q < kLpList / 64; ++q) k[q] = keys[q * 64 + lane];
  return reach_bound<kLpList / 64>(k, n);
}

// The alternatives of one row: ids and values of the n largest logits above
// -inf (lane p the p-th), -1 where there are fewer.  A row is one wave's chain
// of steps.  top_short takes rows whose cells fit a window and whose
// candidates are few, all others (ties of thousands, very long rows) top_long.
constexpr int kLpWindow = 16;  // loads of 256 cells held at a time: 4096 cells, a row of up to 262144 logits
constexpr int kLpShort = 8;    // loads of 8 cells that top_short holds: 64 candidate cells
template <int ES>
struct LpLists {  // a wave's room in LDS
  alignas(16) int keys[2][kLpList];
  alignas(16) int ids[2][kLpList];  // candidate cells, candidate logits
  union {
    typename std::conditional<ES == 2, uint2, uint4>::type cells[kLpWindow * 64];  // four to a lane, as stored
    RawGroup<ES, true> logits[kLpShort * 64];                                      // eight to a lane, as stored
  };
};

__device__ __forceinline__ int wave_scan_i(int x) {
  x += dpp_i<0x111, 0xf>(x, 0);
  x += dpp_i<0x112, 0xf>(x, 0);
  x += dpp_i<0x114, 0xf>(x, 0);
  x += dpp_i<0x118, 0xf>(x, 0);
  x += dpp_i<0x142, 0xa>(x, 0);
  x += dpp_i<0x143, 0xc>(x, 0);
  return x;
}

// The first window of a row's cells, four to a lane and load; -inf past them.
struct LpCellWindow {
  f32x4 c[kLpWindow];
};
__device__ __forceinline__ void load_cells(LpCellWindow& w, const float* cells, int first, int ncell, int lane) {
#pragma unroll
  for (int j = 0; j < kLpWindow; ++j) {
    const int at = first + j * 256 + lane * 4;
    w.c[j] = f32x4{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    if (at < ncell) w.c[j] = *reinterpret_cast<const f32x4*>(cells + at);
  }
}

// The keys of a row's cells, the lanes' largest: a threshold that at least n
// cells reach (or every cell above -inf).
__device__ __forceinline__ int cell_threshold(const f32x4& head, float lm, int ncell, int n) {
  int thr;
  if (ncell <= 256) {
    const int mk[4] = {order_key(head.x), order_key(head.y), order_key(head.z), order_key(head.w)};
    thr = reach_bound<4>(mk, n);
  } else {
    const int mk[1] = {order_key(lm)};
    thr = reach_bound<1>(mk, n);
  }
  return max(thr, order_key(-INFINITY) + 1);
}

// The candidates of a row in any order into L.keys[1], L.ids[1]; their number,
// or -1 where there are too many.  A lane marks what it holds in a mask, and a
// sum over the lanes gives each its places: no step waits for another's count
// (appending 256 cells at a time cost 5 us of the finish's 16, and eight cells'
// logits at a time another 5).
template <int ES>
__device__ __forceinline__ int top_short(const LogprobsParams& P, const char* row, const LpCellWindow& win, int n,
                                         int lane, LpLists<ES>& L) {
  float lm = -INFINITY;
#pragma unroll
  for (int j = 0; j < kLpWindow; ++j)
    lm = fmaxf(fmaxf(fmaxf(win.c[j].x, win.c[j].y), fmaxf(win.c[j].z, win.c[j].w)), lm);
  int thr = cell_threshold(win.c[0], lm, P.nseg * kLpCells, n);
  auto places = [&](uint64_t hit, int& total) {  // where this lane's hits go
    const int mine = __builtin_popcountll(hit), end = wave_scan_i(mine);
    total = lane_i(end, 63);
    return end - mine;
  };
  uint32_t lo = 0, hi = 0;
  const float t0 = order_value(thr);
#pragma unroll
  for (int j = 0; j < kLpWindow; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) (j < 8 ? lo : hi) |= win.c[j][q] >= t0 ? 1u << (4 * (j & 7) + q) : 0u;
  uint64_t hit = ((uint64_t)hi << 32) | lo;
  int ncand, at = places(hit, ncand);
  if (ncand > kLpShort * 8) return -1;
  for (; hit; hit &= hit - 1, ++at) {
    const int k = __builtin_ctzll(hit);
    L.ids[0][at] = (k >> 2) * 256 + lane * 4 + (k & 3);
  }
  __builtin_amdgcn_wave_barrier();
  // the cells' logits, 8 lanes to a cell: the last 8 of the row where a lane's
  // would pass its end, of which it takes what is its own
  RawGroup<ES, true> r[kLpShort];
  int first[kLpShort];
#pragma unroll
  for (int j = 0; j < kLpShort; ++j) {
    const int c = j * 8 + (lane >> 3);
    first[j] = INT_MAX;
    if (j * 8 < ncand) {
      if (c < ncand) first[j] = L.ids[0][c] * 64 + (lane & 7) * 8;
      r[j] = load_any<ES>(row, min(first[j], P.V - 8));
    }
  }
  float most = -INFINITY;
#pragma unroll
  for (int j = 0; j < kLpShort; ++j)
    if (j * 8 < ncand) {
      float x[8];
      unpack_group<ES, true>(r[j], x);
      L.logits[j * 64 + lane] = r[j];
      if (__ballot(first[j] > P.V - 8)) {
#pragma unroll
        for (int q = 0; q < 8; ++q) x[q] = first[j] - q > P.V - 8 ? -INFINITY : x[q];
      }
      most = fmaxf(most, group_max(x));
    }
  // the threshold may rise to what n lanes reach
  const int mk[1] = {order_key(most)};
  thr = max(thr, reach_bound<1>(mk, n));
  const float t1 = order_value(thr);
  lo = hi = 0;
#pragma unroll
  for (int j = 0; j < kLpShort; ++j)
    if (j * 8 < ncand) {
      float x[8];
      uint32_t m = 0;
      unpack_group<ES, true>(r[j], x);
#pragma unroll
      for (int q = 0; q < 8; ++q) m |= x[q] >= t1 ? 1u << q : 0u;
      const int own = min(max(first[j] - (P.V - 8), 0), 8);  // the first of them that is its own
      m = (m >> own) << own;
      (j < 4 ? lo : hi) |= m << (8 * (j & 3));
    }
  hit = ((uint64_t)hi << 32) | lo;
  int ne;
  at = places(hit, ne);
  if (ne > kLpList) return -1;
  __builtin_amdgcn_wave_barrier();
  for (; hit; hit &= hit - 1, ++at) {
    const int k = __builtin_ctzll(hit), j = k >> 3, q = k & 7;
    const int c = j * 8 + (lane >> 3);
    const char* g = reinterpret_cast<const char*>(&L.logits[j * 64 + lane]);
    uint32_t bits = 0;  // (bf16: its upper half)
    __builtin_memcpy(reinterpret_cast<char*>(&bits) + 4 - ES, g + q * ES, ES);
    L.keys[1][at] = order_key(__uint_as_float(bits));
    L.ids[1][at] = min(L.ids[0][c] * 64 + (lane & 7) * 8, P.V - 8) + q;
  }
  __builtin_amdgcn_wave_barrier();
  return ne;
}

// The same for any row, the candidates in ascending order of their ids and of
// those equal to the threshold the first n; the loops are kept rolled
// (unrolled, the wave waits for its own instructions).
template <int ES>
__device__ __forceinline__ int top_long(const LogprobsParams& P, const char* row, const float* cells, int n, int lane,
                                        LpLists<ES>& L) {
  const int ncell = P.nseg * kLpCells;  // at most 2^25, a multiple of 64
  const int windows = (ncell + kLpWindow * 256 - 1) / (kLpWindow * 256);
  float lm = -INFINITY;   // the lane's largest
  f32x4 head;             // its first four
  auto load_window = [&](int w) {
    LpCellWindow win;
    load_cells(win, cells, w * kLpWindow * 256, ncell, lane);
    if (w == 0) head = win.c[0];
#pragma unroll
    for (int j = 0; j < kLpWindow; ++j) {
      const f32x4 c = win.c[j];
      lm = fmaxf(fmaxf(fmaxf(c.x, c.y), fmaxf(c.z, c.w)), lm);
      if constexpr (ES == 2)  // exact in bf16
        L.cells[j * 64 + lane] = uint2{(__float_as_uint(c.x) >> 16) | (__float_as_uint(c.y) & 0xffff0000u),
                                       (__float_as_uint(c.z) >> 16) | (__float_as_uint(c.w) & 0xffff0000u)};
      else
        L.cells[j * 64 + lane] = uint4{__float_as_uint(c.x), __float_as_uint(c.y), __float_as_uint(c.z),
                                       __float_as_uint(c.w)};
    }
  };
#pragma unroll 1
  for (int w = 0; w < windows; ++w) load_window(w);
  int thr = cell_threshold(head, lm, ncell, n);
  LpList lc{L.keys[0], L.ids[0], 0, 0};
  for (;;) {
    lc.count = lc.equal = 0;
    for (int w = 0; w < windows; ++w) {
      if (windows > 1) load_window(w);
      const int loads = min(kLpWindow, (ncell - w * kLpWindow * 256 + 255) / 256);
#pragma unroll 1
      for (int j = 0; j < loads; ++j) {
        int key[4];
        if constexpr (ES == 2) {
          const uint2 v = L.cells[j * 64 + lane];
          key[0] = order_key(__uint_as_float(v.x << 16));
          key[1] = order_key(__uint_as_float(v.x & 0xffff0000u));
          key[2] = order_key(__uint_as_float(v.y << 16));
          key[3] = order_key(__uint_as_float(v.y & 0xffff0000u));
        } else {
          const uint4 v = L.cells[j * 64 + lane];
          key[0] = order_key(__uint_as_float(v.x));
          key[1] = order_key(__uint_as_float(v.y));
          key[2] = order_key(__uint_as_float(v.z));
          key[3] = order_key(__uint_as_float(v.w));
        }
        collect<4>(lc, key, (w * kLpWindow + j) * 256 + lane * 4, thr, n);
      }
    }
    __builtin_amdgcn_wave_barrier();
    if (lc.count <= kLpList) break;
    thr = raise_threshold(lc.keys, lane, n);
  }
  // the cells' logits that reach the threshold: 8 lanes to a cell, 8 cells a
  // load, the next load on its way; the cells stand in ascending order
  LpList le{L.keys[1], L.ids[1], 0, 0};
  auto first_of = [&](int c0) {
    const int at = c0 + (lane >> 3);
    return at < lc.count ? lc.ids[at] * 64 + (lane & 7) * 8 : P.V;
  };
  for (;;) {
    le.count = le.equal = 0;
    int e1 = first_of(0);
    RawGroup<ES, true> r1 = load_any_bounded<ES>(row, e1, P.V);
#pragma unroll 1
    for (int c0 = 0; c0 < lc.count; c0 += 8) {
      const int e0 = e1;
      float x[8];
      int key[8];
      unpack_group<ES, true>(r1, x);
      if (c0 + 8 < lc.count) {
        e1 = first_of(c0 + 8);
        r1 = load_any_bounded<ES>(row, e1, P.V);
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) key[q] = order_key(x[q]);
      // before anything is collected the threshold may rise to what n lanes reach
      if (c0 == 0) {
        int most = key[0];
#pragma unroll
        for (int q = 1; q < 8; ++q) most = max(most, key[q]);
        const int mk[1] = {most};
        thr = max(thr, reach_bound<1>(mk, n));
      }
      collect<8>(le, key, e0, thr, n);
    }
    __builtin_amdgcn_wave_barrier();
    if (le.count <= kLpList) break;
    thr = raise_threshold(le.keys, lane, n);
  }
  return le.count;
}

template <int ES>
__device__ __forceinline__ void top_of_row(const LogprobsParams& P, const char* row, const float* cells,
                                           const LpCellWindow& win, int n, int lane, LpLists<ES>& L, int& out_id,
                                           float& out_x) {
  int ne = -1;
  if (P.nseg * kLpCells <= kLpWindow * 256 && P.V >= 8) ne = top_short<ES>(P, row, win, n, lane, L);
  if (ne < 0) ne = top_long<ES>(P, row, cells, n, lane, L);
  // sorted by rank: the place of an item is the number of items in front
  const int* keys = L.keys[1];
  const int* ids = L.ids[1];
  L.keys[0][lane] = order_key(-INFINITY);
  L.ids[0][lane] = -1;
  __builtin_amdgcn_wave_barrier();
  for (int at = lane; at < ne; at += 64) {
    const int key = keys[at], id = ids[at];
    int rank = 0;
#pragma unroll 8
    for (int o = 0; o < ne; ++o) rank += keys[o] > key || (keys[o] == key && ids[o] < id);
    if (rank < n) {
      L.keys[0][rank] = key;
      L.ids[0][rank] = id;
    }
  }
  __builtin_amdgcn_wave_barrier();
  out_id = L.ids[0][lane];
  out_x = order_value(L.keys[0][lane]);
}

// One wave: row i's records joined, its outputs written.
template <int ES, bool TOP>
__device__ __forceinline__ void finish_row(const LogprobsParams& P, int i, int lane, LpLists<ES>* lists) {
  const int b = (int)P.by_R.of((uint32_t)i), r = i - b * P.R;
  const int tok = P.tokens[i];
  const float T = row_temperature(P, b);
  const float nan = __builtin_nanf("");
  const bool usable = tok >= 0 && tok < P.V && temperature_valid(T);
  const char* row = P.logits + (b * P.req + r * P.row) * ES;
  double M = -INFINITY, S = 0.0, W = 0.0;
  float x_tok = 0.f;
  LpCellWindow win;
  if (usable) {
    // what the row needs first is on its way together: its records, the
    // token's logit, the cells
    const LpRecord* rec = P.rec + (int64_t)i * P.nseg;
    LpRecord q = rec[min(lane, P.nseg - 1)];
    x_tok = load_one<ES>(row, tok);
    if constexpr (TOP) load_cells(win, P.cells + (int64_t)i * P.nseg * kLpCells, 0, P.nseg * kLpCells, lane);
    if (lane >= P.nseg) q = LpRecord{-INFINITY, 0.f, 0.f, 0.f};
    // the records' sums, each brought to the row's maximum: the exponents
    // shift by d = (m - M) * s <= 0, so S by 2^d and W to 2^d (W + d S)
    const double s = 1.4426950408889634074 / (double)T;
    float mm = q.m;
    for (int j = lane + 64; j < P.nseg; j += 64) mm = fmaxf(mm, rec[j].m);
    mm = wave_max_f(mm);
    M = mm;
    double S1 = 0.0, W1 = 0.0;
    for (int j = lane;;) {
      if (q.m > -INFINITY) {
        const double d = fmax(((double)q.m - M) * s, -4000.0);
        const double f = exp2(d);
        S1 += f * q.s;
        W1 += f * (q.w + d * q.s);
      } else {
        S1 += (double)q.s;  // 0, or NaN
      }
      j += 64;
      if (j >= P.nseg) break;
      q = rec[j];
    }
    S = wave_total_d(S1);
    W = wave_total_d(W1);
  }
  const bool good = usable && S > 0.0 && S <= DBL_MAX && fabs(M) <= FLT_MAX;
  const double lnS = good ? log(S) : 0.0;
  if (lane == 0) {
    float lp = tok == -1 ? 0.f : nan, ent = lp;
    if (good) {
      lp = (float)(((double)x_tok - M) / (double)T - lnS);
      ent = (float)fmax(lnS - 0.69314718055994530942 * (W / S), 0.0);
    }
    P.logprobs[i] = lp;
    if (P.entropy) P.entropy[i] = ent;
  }
  if constexpr (TOP) {
    int id = -1;
    float x = -INFINITY;
    if (good)
      top_of_row<ES>(P, row, P.cells + (int64_t)i * P.nseg * kLpCells, win, P.top, lane, *lists, id, x);
    if (lane < P.top) {
      P.top_ids[(int64_t)i * P.top + lane] = id;
      P.top_lp[(int64_t)i * P.top + lane] =
          good ? (float)(((double)x - M) / (double)T - lnS) : (tok == -1 ? 0.f : nan);
    }
  }
}

template <int ES, bool TOP>
__global__ __launch_bounds__(64) void logprobs_finish_kernel(LogprobsParams P) {
  if constexpr (TOP) {
    __shared__ LpLists<ES> lists;
    finish_row<ES, true>(P, blockIdx.x, threadIdx.x, &lists);
  } else {
    finish_row<ES, false>(P, blockIdx.x, threadIdx.x, nullptr);
  }
}

// WHOLE: a workgroup holds a whole row (P.C == 1), and its first wave finishes
// it (no second launch: 4 us less of the 15 us of a small batch).
template <int ES, bool TOP, bool WHOLE>
__global__ __launch_bounds__(kWG) void logprobs_stats_kernel(LogprobsParams P) {
  const int i = (int)P.by_C.of(blockIdx.x);  // row b * R + r
  const int c = (int)blockIdx.x - i * P.C;
  const int b = (int)P.by_R.of((uint32_t)i), r = i - b * P.R;
  const int tok = P.tokens[i];
  const float T = row_temperature(P, b);
  const bool usable = tok >= 0 && tok < P.V && temperature_valid(T);  // the finish reports the others
  if (!WHOLE && !usable) return;
  const char* row = P.logits + (b * P.req + r * P.row) * ES;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const float s = (float)(1.4426950408889634074 / (double)T);
  const int j1 = usable ? min(P.nseg, (c + 1) * kLpChunkSegs) : 0;
  for (int j = c * kLpChunkSegs + wave; j < j1; j += kWaves) {
    const int s0 = j * kSeg;
    RawGroup<ES, true> rg[kSegGroups];
    if (s0 + kSeg <= P.V) {
#pragma unroll
      for (int g = 0; g < kSegGroups; ++g) rg[g] = load_any<ES>(row, s0 + (g * 64 + lane) * 8);
    } else {
#pragma unroll
      for (int g = 0; g < kSegGroups; ++g) {
        const int e = s0 + (g * 64 + lane) * 8;
        rg[g] = load_any_bounded<ES>(row, e, P.V);
      }
    }
    // widened once: the kernel is bound by its vector instructions, and a
    // second widening would be a tenth of them
    float x[kSegGroups][8], gm[kSegGroups], m = -INFINITY;
#pragma unroll
    for (int g = 0; g < kSegGroups; ++g) {
      unpack_group<ES, true>(rg[g], x[g]);
#pragma unroll
      for (int q = 0; q < 8; ++q) asm volatile("" : "+v"(x[g][q]));  // (kept, not widened anew)
      gm[g] = group_max(x[g]);
      m = fmaxf(m, gm[g]);
    }
    m = wave_max_f(m);
    const int64_t rec = (int64_t)i * P.nseg + j;
    if constexpr (TOP) {
      // lane 8j + q holds the maximum of cell 8q + j
      P.cells[rec * kLpCells + (lane & 7) * 8 + (lane >> 3)] = max8_scatter(gm, lane);
    }
    float S = 0.f, W = 0.f;
    // the exponents (x - m) s as x s - c, c = m s rounded: what c is off by
    // (eps) is the same in all of them and taken out of the sums at the end
    const float c = m * s, eps = __builtin_fmaf(m, s, -c);
    if (s0 + kSeg > P.V) {
      // the places past the row's end: so far below the maximum that 2^t is 0,
      // but finite
      const float pad = m - 16384.f / s;
#pragma unroll
      for (int g = 0; g < kSegGroups; ++g)
#pragma unroll
        for (int q = 0; q < 8; ++q) x[g][q] = s0 + (g * 64 + lane) * 8 + q < P.V ? x[g][q] : pad;
    }
    bool again = !(fabsf(c) <= 0x1p24f);
    if (!again) {
#pragma unroll
      for (int g = 0; g < kSegGroups; ++g) {
        float e[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          x[g][q] = __builtin_fmaf(x[g][q], s, -c);
          e[q] = __builtin_amdgcn_exp2f(x[g][q]);
        }
        add_group(e, x[g], S, W);
      }
      const float f = __builtin_amdgcn_exp2f(-eps);
      W = __builtin_fmaf(-eps, S, W) * f;
      S *= f;
      again = __ballot(W != W) != 0;
    }
    if (again) {
      // logits of -inf (0 * -inf in W: exponents no lower than -16384 here), a
      // range that c does not hold, a NaN or +inf, or nothing above -inf: the
      // logits once more, one group after another (a second copy of the sums
      // from registers would double their number)
      S = W = 0.f;
#pragma unroll 1
      for (int g = 0; g < kSegGroups && s0 + g * 512 < P.V; ++g) {
        float y[8], e[8];
        unpack_group<ES, true>(load_any_bounded<ES>(row, s0 + (g * 64 + lane) * 8, P.V), y);
        if (m > -INFINITY) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float t = (y[i] - m) * s;
            e[i] = __builtin_amdgcn_exp2f(t);
            y[i] = fmaxf(t, -16384.f);
          }
          add_group(e, y, S, W);
        } else {
          // only -inf adds nothing, but a NaN or +inf may hide among it
#pragma unroll
          for (int i = 0; i < 8; ++i) S = y[i] == -INFINITY ? S : __builtin_nanf("");
        }
      }
    }
    S = wave_total_f(S);
    W = wave_total_f(W);
    if (lane == 0) P.rec[rec] = LpRecord{m, S, W, 0.f};
  }
  if constexpr (WHOLE) {
    __threadfence_block();
    __syncthreads();
    if constexpr (TOP) {
      __shared__ LpLists<ES> lists;
      if (wave == 0) finish_row<ES, true>(P, i, lane, &lists);
    } else {
      if (wave == 0) finish_row<ES, false>(P, i, lane, nullptr);
    }
  }
}

template <int ES, bool TOP>
static hipError_t launch_logprobs_typed(const LogprobsParams& P, hipStream_t stream) {
  const int64_t rows = (int64_t)P.B * P.R;
  if (P.C == 1) {
    hipLaunchKernelGGL((logprobs_stats_kernel<ES, TOP, true>), dim3((unsigned)rows), dim3(kWG), 0, stream, P);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((logprobs_stats_kernel<ES, TOP, false>), dim3((unsigned)(rows * P.C)), dim3(kWG), 0, stream, P);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((logprobs_finish_kernel<ES, TOP>), dim3((unsigned)rows), dim3(64), 0, stream, P);
  return hipGetLastError();
}

hipError_t launch_logprobs(const LogprobsParams& P, int dtype, hipStream_t stream) {
  if (dtype == SPEC_BF16)
    return P.top > 0 ? launch_logprobs_typed<2, true>(P, stream) : launch_logprobs_typed<2, false>(P, stream);
  return P.top > 0 ? launch_logprobs_typed<4, true>(P, stream) : launch_logprobs_typed<4, false>(P, stream);
}

}  // namespace specv
