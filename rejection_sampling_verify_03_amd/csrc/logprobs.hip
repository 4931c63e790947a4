// logprobs.hip -- log probabilities of given tokens, the entropy of their
// rows and the rows' most likely tokens, on gfx950.
//
// With x the row's logits, m its maximum, s = log2(e) / T and
// t_v = (x_v - m) * s:  S = sum 2^t_v,  W = sum 2^t_v t_v,
//   ln p(v) = (x_v - m) / T - ln S,   entropy = ln S - ln 2 * W / S,
// so one pass that keeps (m, S, W) gives both.  A lane sums its 64 terms in
// fp32 (the largest logit's are exactly 1 and 0), all further sums are in
// double.  The differences x - m are formed before they are scaled, so no
// range of logits or temperatures is lost.
//
// Two kernels, one read of each row:
//
//  logprobs_stats   one 256-thread workgroup per (row, 8 segments), a wave per
//      4096-logit segment: the segment stays in registers while its maximum
//      is taken and then summed against it.  For the alternatives it also
//      writes the maximum of every cell of 64 consecutive logits, 1/64 of the
//      row.
//
//  logprobs_finish  one wave per row: merges the segments' records and finds
//      the alternatives through the cells: the n largest logits lie in the n
//      cells with the largest maxima (lower cell first on ties: a cell's
//      logits all stand in front of the next cell's).  A threshold that at
//      least n cells reach (the n-th largest of the 64 lanes' maxima) picks
//      a few more than n cells, whose logits are read again; those that reach
//      it are sorted.
#include <limits.h>

#include "device_common.hpp"
#include "ops_kernels.hpp"
#include "sampling.hpp"

namespace specv {

// Maximum over each run of 8 lanes, the same in all of them (DPP: mirrored
// half rows, then quads).
__device__ __forceinline__ float max8_lanes(float x) {
  const int ninf = __float_as_int(-INFINITY);
  x = fmaxf(x, __int_as_float(dpp_i<0x141, 0xf>(__float_as_int(x), ninf)));  // lane i with 7 - i
  x = fmaxf(x, __int_as_float(dpp_i<0xb1, 0xf>(__float_as_int(x), ninf)));   // quad [1, 0, 3, 2]
  x = fmaxf(x, __int_as_float(dpp_i<0x4e, 0xf>(__float_as_int(x), ninf)));   // quad [2, 3, 0, 1]
  return x;
}

__device__ __forceinline__ float row_temperature(const LogprobsParams& P, int b) {
  const float T = P.temperature ? P.temperature[b] : 1.0f;
  return T == 0.0f ? 1.0f : T;
}

// Sums a segment held in registers against its maximum m.  CLAMP: exponents
// no lower than -16384, so that a logit of -inf (or one so far below m that
// its exponent overflows) adds 0 * -16384 and not 0 * -inf to W.
template <int ES, bool VEC, bool CLAMP>
__device__ __forceinline__ void segment_sums(RawGroup<ES, VEC> (&rg)[kSegGroups], float m, float s, float& S,
                                             float& W) {
  float Sg[kSegGroups], Wg[kSegGroups];
#pragma unroll
  for (int g = 0; g < kSegGroups; ++g) {
    opaque_group<ES, VEC>(rg[g]);
    float x[8], e[8], w[8];
    unpack_group<ES, VEC>(rg[g], x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float t = (x[i] - m) * s;
      e[i] = __builtin_amdgcn_exp2f(t);
      if (CLAMP) t = fmaxf(t, -16384.f);
      w[i] = t;
    }
    Sg[g] = ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
    float a = e[0] * w[0], b = e[4] * w[4];
#pragma unroll
    for (int i = 1; i < 4; ++i) {
      a = __builtin_fmaf(e[i], w[i], a);
      b = __builtin_fmaf(e[4 + i], w[4 + i], b);
    }
    Wg[g] = a + b;
  }
  S = ((Sg[0] + Sg[1]) + (Sg[2] + Sg[3])) + ((Sg[4] + Sg[5]) + (Sg[6] + Sg[7]));
  W = ((Wg[0] + Wg[1]) + (Wg[2] + Wg[3])) + ((Wg[4] + Wg[5]) + (Wg[6] + Wg[7]));
}

template <int ES, bool VEC, bool TOP>
__global__ __launch_bounds__(kWG) void logprobs_stats_kernel(LogprobsParams P) {
  const int c = blockIdx.x % P.C;
  const int i = blockIdx.x / P.C;  // row b * R + r
  const int b = i / P.R, r = i - b * P.R;
  const int tok = P.tokens[i];
  const float T = row_temperature(P, b);
  if (tok < 0 || tok >= P.V || !temperature_valid(T)) return;  // the finish reports it
  const char* row = P.logits + (b * P.req + r * P.row) * ES;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const float s = (float)(1.4426950408889634074 / (double)T);
  const int j1 = min(P.nseg, (c + 1) * kLpChunkSegs);
  for (int j = c * kLpChunkSegs + wave; j < j1; j += kWaves) {
    const int s0 = j * kSeg;
    RawGroup<ES, VEC> rg[kSegGroups];
    if (s0 + kSeg <= P.V) {
#pragma unroll
      for (int g = 0; g < kSegGroups; ++g) rg[g] = load_raw<ES, VEC>(row, s0 + (g * 64 + lane) * 8);
    } else {
#pragma unroll
      for (int g = 0; g < kSegGroups; ++g) {
        const int e = s0 + (g * 64 + lane) * 8;
        rg[g] = e < P.V ? load_raw_bounded<ES, VEC>(row, e, P.V) : neg_inf_group<ES, VEC>();
      }
    }
    float gm[kSegGroups], m = -INFINITY;
#pragma unroll
    for (int g = 0; g < kSegGroups; ++g) {
      float x[8];
      unpack_group<ES, VEC>(rg[g], x);
      gm[g] = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
      m = fmaxf(m, gm[g]);
    }
    m = wave_max_f(m);
    const int64_t rec = (int64_t)i * P.nseg + j;
    if constexpr (TOP) {
      // lane 8j + q ends with the maximum of cell 8q + j
      float v = 0.f;
#pragma unroll
      for (int g = 0; g < kSegGroups; ++g) {
        const float cm = max8_lanes(gm[g]);
        v = (lane & 7) == g ? cm : v;
      }
      P.cells[rec * kLpCells + (lane & 7) * 8 + (lane >> 3)] = v;
    }
    float S, W;
    if (m > -INFINITY) {
      segment_sums<ES, VEC, false>(rg, m, s, S, W);
      if (__ballot(W != W)) segment_sums<ES, VEC, true>(rg, m, s, S, W);
    } else {
      // no logit above -inf: nothing to add, unless a NaN hides among them
      bool nan = false;
#pragma unroll
      for (int g = 0; g < kSegGroups; ++g) {
        float x[8];
        unpack_group<ES, VEC>(rg[g], x);
#pragma unroll
        for (int q = 0; q < 8; ++q) nan |= x[q] != x[q];
      }
      S = nan ? __builtin_nanf("") : 0.f;
      W = 0.f;
    }
    const double Sd = wave_total_d((double)S), Wd = wave_total_d((double)W);
    if (lane == 0) P.rec[rec] = LpRecord{Sd, Wd, m, 0};
  }
}

// A float's place in the order of floats as a signed integer (-0 as +0).
__device__ __forceinline__ int order_key(float x) {
  const int k = __float_as_int(x + 0.0f);
  return k < 0 ? (int)0x80000000 - k : k;
}
__device__ __forceinline__ float order_value(int k) {
  return __int_as_float(k < 0 ? (int)0x80000000 - k : k);
}

// The n-th largest of the 64 * K keys of a wave (1 <= n <= 64 * K), by
// halving the range that holds it.
template <int K>
__device__ __forceinline__ int nth_largest(const int (&k)[K], int n) {
  int lo = INT_MIN, hi = INT_MAX;  // the largest bound that at least n keys reach
  while (lo < hi) {
    const int mid = (int)(((int64_t)lo + hi + 1) >> 1);
    int cnt = 0;
#pragma unroll
    for (int q = 0; q < K; ++q) cnt += __builtin_popcountll(__ballot(k[q] >= mid));
    if (cnt >= n)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

constexpr int kLpList = 256;  // candidates a wave can hold, 4 per lane

// Appends the lanes' items (those of ascending lanes first) whose key
// reaches thr to a list in LDS: all above it, and of those equal to it the
// first n.  Counts what it would have appended past the list's end too.
struct LpCollect {
  int count, equal;  // appended (or past the end), of them equal to the threshold
};
__device__ __forceinline__ void collect(LpCollect& st, int* keys, int* ids, int lane, bool in, int key, int id, int thr,
                                        int n) {
  const uint64_t eq = __ballot(in && key == thr);
  const uint64_t below = lane ? (~0ull >> (64 - lane)) : 0ull;
  const bool take = in && (key > thr || (key == thr && st.equal + __builtin_popcountll(eq & below) < n));
  const uint64_t tk = __ballot(take);
  if (tk == 0) return;
  const int at = st.count + __builtin_popcountll(tk & below);
  if (take && at < kLpList) {
    keys[at] = key;
    ids[at] = id;
  }
  st.count += __builtin_popcountll(tk);
  st.equal += __builtin_popcountll(eq);
}

// The n-th largest key of a full list: a threshold above the one it was
// collected with that at least n of all items still reach.
__device__ __forceinline__ int raise_threshold(const int* keys, int lane, int n) {
  int k[kLpList / 64];
#pragma unroll
  for (int q = 0; q < kLpList / 64; ++q) k[q] = keys[q * 64 + lane];
  return nth_largest<kLpList / 64>(k, n);
}

// The alternatives of one row: ids and keys of the n largest logits above
// -inf in out_ids / out_keys (lane p the p-th), -1 where there are fewer.
template <int ES, bool VEC>
__device__ __forceinline__ void top_of_row(const LogprobsParams& P, const char* row, const float* cells, int n,
                                           int lane, int* ck, int* ci, int* ek, int* ei, int& out_id, float& out_x) {
  const int ncell = P.nseg * kLpCells;  // at most 2^25
  const int kNone = order_key(-INFINITY);
  // a threshold that at least n cells reach (or -inf: every cell above it)
  float lm = -INFINITY;
  for (int j = lane; j < ncell; j += 64) lm = fmaxf(lm, cells[j]);
  const int mk[1] = {order_key(lm)};
  int thr = max(nth_largest<1>(mk, n), kNone + 1);
  LpCollect st;
  for (;;) {
    st = LpCollect{0, 0};
    for (int j0 = 0; j0 < ncell; j0 += 64) {
      const int key = order_key(cells[j0 + lane]);
      if (__ballot(key >= thr)) collect(st, ck, ci, lane, true, key, j0 + lane, thr, n);
    }
    __builtin_amdgcn_wave_barrier();
    if (st.count <= kLpList) break;
    thr = raise_threshold(ck, lane, n);
  }
  // the cells' logits that reach the threshold: 8 cells at a time, 8 lanes
  // to a cell; the cells stand in ascending order, and so do the logits
  const int nc = st.count;
  for (;;) {
    st = LpCollect{0, 0};
    for (int c0 = 0; c0 < nc; c0 += 8) {
      const int c = c0 + (lane >> 3);
      int key[8];
      const int e0 = c < nc ? ci[c] * 64 + (lane & 7) * 8 : 0;
      float x[8];
      if (c < nc && e0 < P.V) {
        if (e0 + 8 <= P.V) {
          load_group<ES, VEC>(row, e0, x);
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q) x[q] = e0 + q < P.V ? load_one<ES>(row, e0 + q) : -INFINITY;
        }
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) x[q] = -INFINITY;
      }
      int most = kNone;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        key[q] = order_key(x[q]);
        most = max(most, key[q]);
      }
      // lanes in ascending order hold ascending indexes; a lane's eight come
      // one after another
      uint64_t lanes = __ballot(most >= thr);
      while (lanes) {
        const int L = __builtin_ctzll(lanes);
        lanes &= lanes - 1;
        int kq = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int v = lane_i(key[q], L);
          kq = lane == q ? v : kq;
        }
        collect(st, ek, ei, lane, lane < 8, kq, lane_i(e0, L) + lane, thr, n);
      }
    }
    __builtin_amdgcn_wave_barrier();
    if (st.count <= kLpList) break;
    thr = raise_threshold(ek, lane, n);
  }
  // sorted by rank: the place of an item is the number of items in front
  const int ne = st.count;
  out_id = -1;
  out_x = -INFINITY;
  for (int q = 0; q * 64 < ne; ++q) {
    const int at = q * 64 + lane;
    const int key = at < ne ? ek[at] : INT_MIN;
    const int id = at < ne ? ei[at] : INT_MAX;
    int rank = 0;
    for (int o = 0; o < ne; ++o) rank += ek[o] > key || (ek[o] == key && o < at);
    // the lane whose number is an item's place takes it
    for (uint64_t w = __ballot(at < ne && rank < n); w; w &= w - 1) {
      const int L = __builtin_ctzll(w);
      const int p = lane_i(rank, L), k = lane_i(key, L), d = lane_i(id, L);
      if (lane == p) {
        out_id = d;
        out_x = order_value(k);
      }
    }
  }
}

template <int ES, bool VEC, bool TOP>
__global__ __launch_bounds__(64) void logprobs_finish_kernel(LogprobsParams P) {
  __shared__ int lists[TOP ? 4 * kLpList : 1];
  const int i = blockIdx.x, lane = threadIdx.x;
  const int b = i / P.R, r = i - b * P.R;
  const int tok = P.tokens[i];
  const float T = row_temperature(P, b);
  const float nan = __builtin_nanf("");
  const bool usable = tok >= 0 && tok < P.V && temperature_valid(T);
  double M = -INFINITY, S = 0.0, W = 0.0;
  if (usable) {
    // the records' sums, each brought to the row's maximum: the exponents
    // shift by d = (m - M) * s <= 0, so S by 2^d and W to 2^d (W + d S)
    const LpRecord* rec = P.rec + (int64_t)i * P.nseg;
    const double s = 1.4426950408889634074 / (double)T;
    float mm = -INFINITY;
    for (int j = lane; j < P.nseg; j += 64) mm = fmaxf(mm, rec[j].m);
    mm = wave_max_f(mm);
    M = mm;
    double S1 = 0.0, W1 = 0.0;
    for (int j = lane; j < P.nseg; j += 64) {
      const LpRecord q = rec[j];
      if (q.m > -INFINITY) {
        const double d = fmax(((double)q.m - M) * s, -4000.0);
        const double f = exp2(d);
        S1 += f * q.s;
        W1 += f * (q.w + d * q.s);
      } else {
        S1 += q.s;  // 0, or NaN
      }
    }
    S = wave_total_d(S1);
    W = wave_total_d(W1);
  }
  const bool good = usable && S > 0.0 && S <= DBL_MAX && fabs(M) <= FLT_MAX;
  const char* row = P.logits + (b * P.req + r * P.row) * ES;
  const double lnS = good ? log(S) : 0.0;
  if (lane == 0) {
    float lp = tok == -1 ? 0.f : nan, ent = lp;
    if (good) {
      const double x = load_one<ES>(row, tok);
      lp = (float)((x - M) / (double)T - lnS);
      ent = (float)fmax(lnS - 0.69314718055994530942 * (W / S), 0.0);
    }
    P.logprobs[i] = lp;
    if (P.entropy) P.entropy[i] = ent;
  }
  if constexpr (TOP) {
    int id = -1;
    float x = -INFINITY;
    if (good)
      top_of_row<ES, VEC>(P, row, P.cells + (int64_t)i * P.nseg * kLpCells, P.top, lane, lists, lists + kLpList,
                          lists + 2 * kLpList, lists + 3 * kLpList, id, x);
    if (lane < P.top) {
      P.top_ids[(int64_t)i * P.top + lane] = id;
      P.top_lp[(int64_t)i * P.top + lane] =
          good ? (float)(((double)x - M) / (double)T - lnS) : (tok == -1 ? 0.f : nan);
    }
  }
}

template <int ES, bool VEC, bool TOP>
static hipError_t launch_logprobs_typed(const LogprobsParams& P, hipStream_t stream) {
  const int64_t rows = (int64_t)P.B * P.R;
  hipLaunchKernelGGL((logprobs_stats_kernel<ES, VEC, TOP>), dim3((unsigned)(rows * P.C)), dim3(kWG), 0, stream, P);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((logprobs_finish_kernel<ES, VEC, TOP>), dim3((unsigned)rows), dim3(64), 0, stream, P);
  return hipGetLastError();
}

hipError_t launch_logprobs(const LogprobsParams& P, int dtype, bool vec, hipStream_t stream) {
  if (dtype == SPEC_BF16) {
    if (P.top > 0)
      return vec ? launch_logprobs_typed<2, true, true>(P, stream) : launch_logprobs_typed<2, false, true>(P, stream);
    return vec ? launch_logprobs_typed<2, true, false>(P, stream) : launch_logprobs_typed<2, false, false>(P, stream);
  }
  if (P.top > 0)
    return vec ? launch_logprobs_typed<4, true, true>(P, stream) : launch_logprobs_typed<4, false, true>(P, stream);
  return vec ? launch_logprobs_typed<4, true, false>(P, stream) : launch_logprobs_typed<4, false, false>(P, stream);
}

}  // namespace specv
