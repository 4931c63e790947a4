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
// One workgroup takes a row.  Its first pass counts the logits in bins of their
// upper bits, in the order of the logits: a bin of bf16 logits is a single
// value, so the bins' counts give every sum of weights with one exponential a
// bin; fp32 logits, whose bins hold several values, are weighed one by one in a
// second pass where top p asks for it.  The bin in which the count or the mass
// reaches a border is known from one scan.  Where the tokens up to it are few
// they are gathered into LDS and everything else happens there; otherwise the
// border is found inside its bin (the c-th of equal logits by their index, or
// the logits of the bin gathered), and the token by the sums of kept weights
// over ranges of indices, then inside the range.  Up to kCand logits are
// candidates from the start.
//
// Few rows of many logits are shared out to several workgroups each, in three
// kernels (four with fp32 logits and a top p): each sweeps a part of the row
// and leaves its counts, its candidates or its sums for the next, which goes on
// from the joined ones; what lies between two sweeps every workgroup of a row
// works out by itself.
//
// Bounds, measured (MI355X).  512 rows of 151936 bf16 logits, top p: 87 us, of
// which the bytes need 23; 21 vector instructions a logit fill 60 % of the issue
// slots (the place of a logit among the bins, 4.5 of them, in each of two
// sweeps), and the atomic additions and lookups in LDS, which half collide, 32 %
// of its cycles.  64 rows of 201088 with settings of their own: 53 us (the parts'
// counts 15, their candidates or sums 23, the rest 14), of which the bytes need
// 4: chains of dependent steps on a few waves.  288 such rows cut: 64 to 71 us by
// their settings, and 31 (5.6 TB/s) to write what is left of the logits.  Four rows
// of 1024 fp32 logits, top k: 11 us, a chain of steps again.
//
// Additions in one place of LDS follow one another.  Logits masked with -128 or
// less are spared it: the last bin's count is what the others leave (288 rows of
// 151936 with a hundredth of the logits left, top k: 47 us at -inf or -10000, whole
// rows 46; added one by one 274).  Rows most of whose logits share a value above
// -128 are not: 99 % at -100 or -50, top k 274 us, top p 291 (89 for whole rows); at 0,
// where they have weight, 274 and 1566, uncut 204 (57); fp32 logits 282 and 350 (93 and
// 340 for whole rows), at 0 282 and 2043.
//
// Registers: of the 128 that four waves to a SIMD have, 28 more would be needed in
// the whole draw of bf16 rows with 1024 threads, 24 in its cut, 25 in the shared
// cut's last kernel, 8 with 512 threads, 6 at most with fp32 logits: so many are
// spilled.
//
#include <limits.h>

#include <type_traits>

#include "ops_kernels.hpp"
#include "unaligned.hpp"

namespace specv {

constexpr int kRangeBits = kCutRangeBits, kRanges = kCutRanges;  // of a search's histogram
constexpr int kCand = kCutCand;                                 // candidates held in LDS
typedef unsigned long long u64;
typedef u64 u64x2 __attribute__((ext_vector_type(2)));
constexpr u64 kNone = ~0ull;

// What a request asks for.
struct Cut {
  float T, p, mn;
  int k;          // 0: all
  bool ok;        // usable
  bool greedy, all;  // T = 0; nothing is left out
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

// 2^(t + frac) for t <= 0 as a whole number below 2^52, rounded to nearest: by
// the nearest whole exponent and the power series of 2^f, |f| <= 1/2, whose terms
// left out are below 2^-47 of it.  (Adding 1.5 * 2^52 rounds to a whole number,
// which its low word then holds: conversions and fp64 scaling are slow here.)
__device__ __forceinline__ double whole_pow2(double t, int frac) {
  constexpr double kRound = 0x1.8p52, L = 0.693147180559945309417;
  constexpr double c2 = L * L / 2, c3 = c2 * L / 3, c4 = c3 * L / 4, c5 = c4 * L / 5, c6 = c5 * L / 6, c7 = c6 * L / 7,
                   c8 = c7 * L / 8, c9 = c8 * L / 9, c10 = c9 * L / 10, c11 = c10 * L / 11;
  t = fmax(t, -56.0);  // (below that nothing is left of it: frac is at most 48)
  const double r = t + kRound;
  const int n = (int)(uint32_t)__double_as_longlong(r);
  const double f = t - (r - kRound);
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
  const uint64_t u = (uint64_t)__double_as_longlong(y) + ((uint64_t)(uint32_t)(n + frac) << 52);
  return __longlong_as_double((long long)u) + 0x1p52;  // (rounds)
}

// The whole number that a value between 2^52 and 2^53 is above 2^52.
__device__ __forceinline__ u64 above52(double y) { return (u64)__double_as_longlong(y) & ((1ull << 52) - 1); }
// A value below 2^52 as a whole number, rounded to nearest.
__device__ __forceinline__ u64 whole(double y) { return above52(y + 0x1p52); }

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


// ------------------------------------------------------------------- bins --
// The bins of logits by sign and upper bits, in falling order: 2^kFine to an
// octave from 2^-20 to 2^7 in magnitude, and three that hold what is left: from
// 2^7 on (bin 0), below 2^-20 in magnitude (the middle one), from -2^7 down.
// They are kept by slot, the clamped magnitude of either sign: slots 0 and kHalf
// are both the middle bin's (counts are moved to the first).
template <int ES>
struct Bins {
  static constexpr int kFine = ES == 2 ? 7 : 6, kShift = 23 - kFine;  // (bf16: all the bits there are)
  static constexpr uint32_t kLo = 107u << kFine, kHi = 134u << kFine;
  static constexpr int kMid = (int)(kHi - kLo) + 1, kN = 2 * kMid + 1;
  static constexpr int kHalf = kMid + 1, kSlots = 2 * kHalf;
  static __device__ __forceinline__ int slot(float x) {
    const uint32_t u = __float_as_uint(x);
    return (int)(min(max((u & 0x7fffffffu) >> kShift, kLo - 1), kHi) - (kLo - 1) + (u >> 31) * kHalf);
  }
  static __host__ __device__ __forceinline__ constexpr int slot_of(int bin) { return bin <= kMid ? kMid - bin : kHalf + bin - kMid; }
  static __device__ __forceinline__ int of(float x) {
    const int s = slot(x);
    return s < kHalf ? kMid - s : kMid + s - kHalf;
  }
  // whether all its logits are one value, and that value
  static __device__ __forceinline__ bool single(int bin) { return ES == 2 && bin > 0 && bin < kN - 1 && bin != kMid; }
  static __device__ __forceinline__ float value(int bin) {
    const uint32_t mag = kLo - 1 + (uint32_t)abs(bin - kMid);
    return __uint_as_float((mag << kShift) | (bin > kMid ? 0x80000000u : 0u));
  }
  // the smallest value that the bin can hold
  static __device__ __forceinline__ float least(int bin) {
    if (bin == kN - 1) return -INFINITY;
    if (bin == kMid) return -__uint_as_float((kLo << kShift) - (ES == 2 ? 0x10000u : 1u));
    const uint32_t mag = kLo - 1 + (uint32_t)abs(bin - kMid);
    return bin < kMid ? __uint_as_float(mag << kShift)
                      : -__uint_as_float(ES == 2 ? mag << kShift : ((mag + 1) << kShift) - 1);
  }
};
static_assert((Bins<4>::kSlots + 1) / 2 + Bins<4>::kSlots <= Bins<2>::kSlots,
              "counts and masses of fp32 in the place of bf16's weights");
static_assert(Bins<2>::kSlots % 4 == 0 && Bins<4>::kSlots % 4 == 0, "taken four at a time");
static_assert(Bins<2>::kSlots * 4 <= kSplitPartBytes && Bins<4>::kSlots * 12 <= kSplitPartBytes, "room for a part's");

// SMALL: rows of up to kCand logits, all of them candidates.
template <bool SMALL>
struct CutShared {
  // by slot.  bf16: counts (u32), later weights (double); fp32: counts, and
  // behind them masses
  alignas(16) u64 bins[SMALL ? 1 : Bins<2>::kSlots];
  union {
    u64 ranges[kRanges];
    struct {  // a range's candidates
      u64 few[64], few_mass[64], few_upto[64];
    };
  };
  u64 cand[kCand];  // keys of rank; (bf16) counts of equal logits by range
  u64 wave[2][16];
  float wave_f[16];
  uint32_t wave_u[16];
  alignas(16) float tail[8];  // the row's last group, if that is not whole, filled up with -inf
  u64 before, through, special[3];
  int bin, count;
};

// The slots of 8 bf16 logits, two to an instruction.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void slots8(const RawGroup<2, true>& g, uint32_t (&slot)[8]) {
  using B = Bins<2>;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const u16x2 lo = (uint16_t)(B::kLo - 1), hi = (uint16_t)B::kHi, half = (uint16_t)B::kHalf;
    const uint32_t two = g.v[i];
    u16x2 mag = __builtin_bit_cast(u16x2, two & 0x7fff7fffu);
    uint32_t signs = __builtin_bit_cast(uint32_t, __builtin_bit_cast(u16x2, two) >> (uint16_t)15);
    asm volatile("" : "+v"(signs));  // (kept a factor: a choice between two values takes five instructions for two)
    const u16x2 sign = __builtin_bit_cast(u16x2, signs);
    mag = sign * half + (__builtin_elementwise_min(__builtin_elementwise_max(mag, lo), hi) - lo);
    const uint32_t both = __builtin_bit_cast(uint32_t, mag);
    slot[2 * i] = both & 0xffffu;
    slot[2 * i + 1] = both >> 16;
  }
}

// Whether some of 8 bf16 logits falls into the last bin (as unsigned numbers
// these are the largest).
__device__ __forceinline__ bool lowest8(const RawGroup<2, true>& g) {
  const uint32_t two[4] = {g.v.x, g.v.y, g.v.z, g.v.w};
  u16x2 m = __builtin_bit_cast(u16x2, two[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, two[i]));
  return max(m.x, m.y) >= (uint16_t)(0x8000u | Bins<2>::kHi);
}

// Whether some of 8 bf16 logits falls into a bin of several values, the last one
// counted or not.
__device__ __forceinline__ bool special8(const RawGroup<2, true>& g, bool last) {
  using B = Bins<2>;
  const uint32_t two[4] = {g.v.x, g.v.y, g.v.z, g.v.w};
  const u16x2 cap = (uint16_t)(last ? 0xffffu : 0x8000u | (B::kHi - 1)), lo = (uint16_t)B::kLo;
  u16x2 m{0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const u16x2 a = __builtin_elementwise_min(__builtin_bit_cast(u16x2, two[i]), cap) & (uint16_t)0x7fff;
    m = __builtin_elementwise_max(m, a - lo);
  }
  return max(m.x, m.y) >= (uint16_t)(B::kHi - B::kLo);
}

// A bound from below on logits, as the test of a group of 8 takes it: bf16
// values above zero rise with their bits as signed numbers, those below zero
// fall with them as unsigned ones.
template <int ES>
struct Floor {
  float x;
  uint32_t both;  // (bf16) its bits in both halves
  bool above;     // (bf16) above zero
  __device__ __forceinline__ explicit Floor(float f) : x(f) {
    uint32_t u = __float_as_uint(f) >> 16;
    above = f > 0.f;
    if (f == 0.f) u = 0x8000u;
    both = u | u << 16;
  }
  // whether some logit of the group may reach it
  __device__ __forceinline__ bool reached(const RawGroup<ES, true>& g) const {
    if constexpr (ES == 2) {
      typedef int16_t i16x2 __attribute__((ext_vector_type(2)));
      const uint32_t two[4] = {g.v.x, g.v.y, g.v.z, g.v.w};
      if (above) {
        i16x2 m = __builtin_bit_cast(i16x2, two[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(i16x2, two[i]));
        return max(m.x, m.y) >= (int16_t)(both & 0xffffu);
      }
      u16x2 m = __builtin_bit_cast(u16x2, two[0]);
#pragma unroll
      for (int i = 1; i < 4; ++i) m = __builtin_elementwise_min(m, __builtin_bit_cast(u16x2, two[i]));
      return min(m.x, m.y) <= (uint16_t)(both & 0xffffu);
    } else {
      float m = g.a[0];
#pragma unroll
      for (int i = 1; i < 4; ++i) m = fmaxf(m, g.a[i]);
#pragma unroll
      for (int i = 0; i < 4; ++i) m = fmaxf(m, g.b[i]);
      return m >= x;
    }
  }
};

struct Crossing {
  int bin;  // -1: the border is above the total
  u64 before, border, through;
};

__device__ __forceinline__ u64 lane_u64(u64 x, int l) {
  return ((u64)(uint32_t)lane_i((int)(x >> 32), l) << 32) | (uint32_t)lane_i((int)x, l);
}

__device__ __forceinline__ int bits_of(u64 x) { return 64 - __clzll((long long)x); }

// The key of rank of logit x at index e, rising in a row's order.
template <int ES>
__device__ __forceinline__ u64 key_of(float x, int e, int ibits) {
  return ((u64)((ES == 2 ? 0xffffu : 0xffffffffu) - place<ES>(x)) << ibits) | (uint32_t)e;
}

// A row and what its passes share; NT: threads of the workgroup.
template <int ES, int NT, bool SMALL>
struct CutRow {
  using B = Bins<ES>;
  static constexpr int kWavesNT = NT / 64;
  static constexpr int kPer = (B::kN + NT - 1) / NT;  // bins of a thread

  CutShared<SMALL>& S;
  const char* lg;
  int V, ibits, frac;
  float m;
  double s;  // log2(e) / T

  // by slot
  __device__ __forceinline__ uint32_t* counts() const { return reinterpret_cast<uint32_t*>(S.bins); }
  __device__ __forceinline__ double* weights() const { return reinterpret_cast<double*>(S.bins); }
  __device__ __forceinline__ u64* masses() const { return S.bins + (B::kSlots + 1) / 2; }

  __device__ __forceinline__ u64 rank_key(float x, int e) const { return key_of<ES>(x, e, ibits); }
  __device__ __forceinline__ float key_logit(u64 key) const {
    return value_at<ES>((ES == 2 ? 0xffffu : 0xffffffffu) - (uint32_t)(key >> ibits));
  }
  __device__ __forceinline__ u64 index_mask() const { return (1ull << ibits) - 1; }
  // The key of the last place that a bin's logits can have.
  __device__ __forceinline__ u64 bin_end(int bin) const { return rank_key(B::least(bin), 0) | index_mask(); }

  // The weight of a logit, a whole number.
  __device__ __forceinline__ double exponent(float x) const { return ((double)x - (double)m) * s; }
  __device__ __forceinline__ double weight_of(float x) const { return whole_pow2(exponent(x), frac) - 0x1p52; }
  __device__ __forceinline__ u64 mass_of(float x) const { return above52(whole_pow2(exponent(x), frac)); }

  // Whether logits of -2^7 and below (the last bin's) may have a weight.
  __device__ __forceinline__ bool low_weighs() const { return ((double)m + 128.0) * s < frac + 2; }

  __device__ __forceinline__ void read_tail() const {  // (a barrier stands in front of its use)
    if (threadIdx.x < 8) {
      const int e = (V & ~7) + threadIdx.x;
      S.tail[threadIdx.x] = e < V ? load_one<ES>(lg, e) : -INFINITY;
    }
  }
  __device__ __forceinline__ RawGroup<ES, true> tail() const {
    RawGroup<ES, true> g;
    const f32x4 a = *reinterpret_cast<const f32x4*>(S.tail), b = *reinterpret_cast<const f32x4*>(S.tail + 4);
    if constexpr (ES == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = i < 2 ? a[2 * i] : b[2 * i - 4], y = i < 2 ? a[2 * i + 1] : b[2 * i - 3];
        g.v[i] = (__float_as_uint(x) >> 16) | (__float_as_uint(y) & 0xffff0000u);
      }
    } else {
      g.a = a;
      g.b = b;
    }
    return g;
  }

  // f(raw, e) for the groups of 8 logits from index e on that hold some of
  // [first, last]; past the row's end -inf.
  template <class F>
  __device__ __forceinline__ void each_group(int first, int last, F f) const {
    constexpr int kAhead = ES == 2 ? 4 : 2;
    const int g1 = (last >> 3) + 1, full = V >> 3;
    RawGroup<ES, true> next[kAhead];
    auto load = [&](int g0) {
      if (full > 0) {  // (without a condition on each, so that they are on their way together)
#pragma unroll
        for (int q = 0; q < kAhead; ++q) next[q] = load_any<ES>(lg, (int64_t)min(g0 + q * NT, full - 1) * 8);
      }
      if (g1 > full) {
#pragma unroll
        for (int q = 0; q < kAhead; ++q)
          if (g0 + q * NT == full) next[q] = tail();
      }
    };
    int g0 = (first >> 3) + threadIdx.x;
    if (g0 < g1) load(g0);
    for (; g0 < g1; g0 += NT * kAhead) {
      RawGroup<ES, true> raw[kAhead];
#pragma unroll
      for (int q = 0; q < kAhead; ++q) raw[q] = next[q];
      if (g0 + NT * kAhead < g1) load(g0 + NT * kAhead);
#pragma unroll
      for (int q = 0; q < kAhead; ++q)
        if (g0 + q * NT < g1) f(raw[q], (g0 + q * NT) * 8);
    }
  }

  __device__ __forceinline__ float block_max(float x) const {
    x = wave_max_f(x);
    if ((threadIdx.x & 63) == 0) S.wave_f[threadIdx.x >> 6] = x;
    __syncthreads();
    float y = S.wave_f[0];
#pragma unroll
    for (int w = 1; w < kWavesNT; ++w) y = fmaxf(y, S.wave_f[w]);
    __syncthreads();
    return y;
  }

  // Of the places in thread order (a thread has the values at(0), ..., at(n - 1)
  // and, beside each, other(i)) the one at which the sum reaches the border, with
  // the sum of the others up to and with it.  All threads call it; what at()
  // reads is complete, and free when it returns.
  // (N: at most so many, whose values stay in registers; 0: any number, read again)
  template <int N, class At, class Other>
  __device__ __forceinline__ Crossing find_crossing(const Border& border, u64 offset, int place0, int n, At at,
                                                    Other other) const {
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    __syncthreads();
    u64 v = 0, o = 0, mine[N > 0 ? N : 1];
    if constexpr (N > 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        mine[i] = i < n ? at(i) : 0;
        v += mine[i];
        o += i < n ? other(i) : 0;
      }
    } else {
      for (int i = 0; i < n; ++i) {
        v += at(i);
        o += other(i);
      }
    }
    const u64 x = wave_scan_u64(v), y = wave_scan_u64(o);
    if (lane == 63) {
      S.wave[0][wave] = x;
      S.wave[1][wave] = y;
    }
    if (t == 0) S.bin = -1;
    __syncthreads();
    u64 base = 0, total = 0, obase = 0;
#pragma unroll
    for (int w = 0; w < kWavesNT; ++w) {
      base += w < wave ? S.wave[0][w] : 0;
      obase += w < wave ? S.wave[1][w] : 0;
      total += S.wave[0][w];
    }
    const u64 to = border.of(total) - offset;
    u64 sum = base + x - v, through = obase + y - o;
    if (sum < to && to <= sum + v) {
      int i = 0;
      if constexpr (N > 0) {
        bool past = false;
#pragma unroll
        for (int k = 0; k < N; ++k) {
          if (past) continue;
          i = k;
          through += other(k);
          past = to <= sum + mine[k];
          sum += past ? 0 : mine[k];
        }
      } else {
        for (;; ++i) {
          const u64 one = at(i);
          through += other(i);
          if (to <= sum + one) break;
          sum += one;
        }
      }
      S.bin = place0 + i;
      S.before = sum;
      S.through = through;
    }
    __syncthreads();
    const Crossing c{S.bin, S.before, to + offset, S.through};
    __syncthreads();
    return c;
  }

  __device__ __forceinline__ Crossing find_range(const Border& border, u64 offset) const {
    constexpr int kMine = kRanges / NT;
    const int t = threadIdx.x * kMine;
    return find_crossing<kMine>(border, offset, t, kMine, [&](int i) { return S.ranges[t + i]; }, [](int) { return (u64)0; });
  }

  __device__ __forceinline__ void clear_ranges() const {
    for (int i = threadIdx.x; i < kRanges; i += NT) S.ranges[i] = 0;
    __syncthreads();
  }

  // The same among the n <= 64 in `few`: each one's sum up to itself, the pairs
  // shared out to the waves.
  template <bool INDEX, bool MASS>
  __device__ __forceinline__ u64 search_few(int n, const Border& border, u64 offset) const {
    constexpr int kShare = 64 / kWavesNT;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    auto key_of_place = [&](int j) { return INDEX ? S.few[j] & index_mask() : S.few[j]; };
    if (threadIdx.x < n) {
      S.few_mass[lane] = MASS ? mass_of(key_logit(S.few[lane])) : 1;
      S.few_upto[lane] = 0;
    }
    __syncthreads();
    const u64 key = lane < n ? key_of_place(lane) : 0, mine = lane < n ? S.few_mass[lane] : 0;
    u64 upto = 0;
#pragma unroll
    for (int q = 0; q < kShare; ++q) {
      const int j = wave * kShare + q;
      if (j < n && key_of_place(j) <= key) upto += S.few_mass[j];
    }
    if (lane < n && upto) atomicAdd(&S.few_upto[lane], upto);
    __syncthreads();
    upto = lane < n ? S.few_upto[lane] : 0;
    const u64 to = border.of(lane_u64(wave_scan_u64(mine), 63)) - offset;
    const uint64_t at = __ballot(lane < n && upto >= to && upto - mine < to);
    __syncthreads();  // (they are free)
    return at ? lane_u64(key, __builtin_ctzll(at)) : kNone;
  }

  // Among the candidates in LDS with a key of rank up to `last`, the key (of
  // rank, or the index) at which the sum of weights (or the count) reaches the
  // border; kNone if it never does.  Keys lie in [lo, hi]; `offset` stands in
  // front of them.
  template <bool INDEX, bool MASS>
  __device__ __forceinline__ u64 search_lds(int n, u64 last, u64 lo, u64 hi, Border border, u64 offset) const {
    for (;;) {
      if (threadIdx.x == 0) S.count = 0;
      __syncthreads();
      for (int i = threadIdx.x; i < n; i += NT) {
        const u64 rank = S.cand[i];
        const u64 key = INDEX ? rank & index_mask() : rank;
        if (rank <= last && key >= lo && key <= hi) {
          const int at = atomicAdd(&S.count, 1);
          if (at < 64) S.few[at] = rank;
        }
      }
      __syncthreads();
      if (S.count <= 64) return search_few<INDEX, MASS>(S.count, border, offset);
      const int shift = max(bits_of(hi - lo) - kRangeBits, 0);
      clear_ranges();
      for (int i = threadIdx.x; i < n; i += NT) {
        const u64 rank = S.cand[i];
        const u64 key = INDEX ? rank & index_mask() : rank;
        if (rank <= last && key >= lo && key <= hi)
          atomicAdd(&S.ranges[(key - lo) >> shift], MASS ? mass_of(key_logit(rank)) : 1ull);
      }
      const Crossing c = find_range(border, offset);
      if (c.bin < 0) return kNone;
      border = Border{Border::kFixed, c.border, 0.0};
      offset += c.before;
      lo += (u64)c.bin << shift;
      if (shift == 0) return lo;
      hi = min(hi, lo + (1ull << shift) - 1);
    }
  }

  // A sum of the group at e to its range, 2^shift >= 8 indices wide: the lanes of a
  // range (wide enough, and lane order is index order) joined first, as they
  // would all add in one place.  (The lanes at work are a prefix of the wave's.)
  __device__ __forceinline__ void add_range(u64* ranges, int at, int shift, double sum) const {
    const int lane = threadIdx.x & 63;
    u64 y = whole(sum);  // (a group's 8 weights, below 2^52: 16 groups' would be past a double's bits)
    if (shift >= 7) {
      y += dpp_u64<0x111, 0xf>(y);
      y += dpp_u64<0x112, 0xf>(y);
      y += dpp_u64<0x114, 0xf>(y);
      y += dpp_u64<0x118, 0xf>(y);
      const int last = 63 - __builtin_clzll(__ballot(true));
      if ((lane & 15) != 15 && lane != last) return;
    }
    if (y) atomicAdd(&ranges[at], y);
  }

  // The index in [lo, hi] at which the sum, with `offset` in front, reaches the
  // border: sums over ranges of indices, then inside the range.  pass(lo, hi, f)
  // calls f(e, sum) for the groups of [lo, hi] with their sum (all lanes of a
  // wave that have a group, or none); one(x, e) is the part of a single logit.
  template <class Pass, class One>
  __device__ __forceinline__ int search_index(int lo, int hi, Border border, u64 offset, Pass pass, One one) const {
    for (;;) {
      const int shift = max(bits_of((u64)(hi - lo)) - kRangeBits, 0);
      clear_ranges();
      if (shift >= 3) {  // (ranges of whole groups)
        pass(lo, hi, [&](int e, double sum) { add_range(S.ranges, (e - lo) >> shift, shift, sum); });
      } else {
        each_group(lo, hi, [&](const RawGroup<ES, true>& raw, int e) {
          float x[8];
          unpack_group<ES, true>(raw, x);
#pragma unroll 1
          for (int q = 0; q < 8; ++q)
            if (e + q >= lo && e + q <= hi) {
              const double y = one(x[q], e + q);
              if (y > 0.0) atomicAdd(&S.ranges[(e + q - lo) >> shift], whole(y));
            }
        });
      }
      const Crossing c = find_range(border, offset);
      if (c.bin < 0) return -1;
      border = Border{Border::kFixed, c.border, 0.0};
      offset += c.before;
      lo += c.bin << shift;
      if (shift == 0) return lo;
      hi = lo + min(hi - lo, (1 << shift) - 1);
    }
  }

  // The logits from `floor` up for which take(key) holds gathered into LDS, as
  // many as fit: how many there are.
  template <class Take>
  __device__ __forceinline__ int gather(int first, int last, float floor, Take take) const {
    __syncthreads();
    if (threadIdx.x == 0) S.count = 0;
    __syncthreads();
    const Floor<ES> low(floor);
    each_group(first, last, [&](const RawGroup<ES, true>& raw, int e) {
      if (!low.reached(raw)) return;
      float x[8];
      unpack_group<ES, true>(raw, x);
      uint32_t hits = 0;
#pragma unroll
      for (int q = 0; q < 8; ++q) hits |= x[q] >= floor ? 1u << q : 0u;
      for (; hits; hits &= hits - 1) {
        const int q = __builtin_ctz(hits);
        const u64 key = rank_key(select8(x, q), e + q);
        if (e + q >= V || !take(key)) continue;
        const int at = atomicAdd(&S.count, 1);
        if (at < kCand) S.cand[at] = key;
      }
    });
    __syncthreads();
    const int n = S.count;
    __syncthreads();
    return n;
  }
  static __device__ __forceinline__ float select8(const float (&x)[8], int q) {
    const float a = q & 1 ? x[1] : x[0], b = q & 1 ? x[3] : x[2], c = q & 1 ? x[5] : x[4], d = q & 1 ? x[7] : x[6];
    const float e = q & 2 ? b : a, f = q & 2 ? d : c;
    return q & 4 ? f : e;
  }

  // The key of rank at which the weights (or the count) of the logits of one bin
  // up to `last` reach the border.
  template <bool MASS>
  __device__ __forceinline__ u64 search_bin(int bin, u64 last, u64 border) const {
    const float floor = fmaxf(B::least(bin), -FLT_MAX);  // (-inf stays what it is, kept or not)
    u64 lo = bin > 0 ? bin_end(bin - 1) + 1 : 0, hi = min(last, bin_end(bin)), offset = 0;
    hi = min(hi, rank_key(-FLT_MAX, 0) | index_mask());
    int n = gather(0, V - 1, floor, [&](u64 key) { return key >= lo && key <= hi; });
    if (!MASS && border > (u64)n) return hi;
    const Border to{Border::kFixed, border, 0.0};
    while (n > kCand) {  // their keys in finer ranges, over the row again
      const int shift = max(bits_of(hi - lo) - kRangeBits, 0);
      clear_ranges();
      each_group(0, V - 1, [&](const RawGroup<ES, true>& raw, int e) {
        float x[8];
        unpack_group<ES, true>(raw, x);
#pragma unroll 1
        for (int q = 0; q < 8; ++q) {
          const u64 key = rank_key(x[q], e + q);
          if (key >= lo && key <= hi && e + q < V) atomicAdd(&S.ranges[(key - lo) >> shift], MASS ? mass_of(x[q]) : 1ull);
        }
      });
      const Crossing c = find_range(to, offset);
      if (c.bin < 0) return kNone;
      offset += c.before;
      lo += (u64)c.bin << shift;
      hi = min(hi, lo + (1ull << shift) - 1);
      n = gather(0, V - 1, floor, [&](u64 key) { return key >= lo && key <= hi; });
    }
    return search_lds<false, MASS>(n, last, lo, hi, to, offset);
  }

  // Whether a logit's key is at most `last`.
  struct Upto {
    float x;
    int at;
    __device__ __forceinline__ Upto(const CutRow& w, u64 last)
        : x(last == kNone ? -INFINITY : w.key_logit(last)), at(last == kNone ? INT_MAX : (int)(last & w.index_mask())) {}
    __device__ __forceinline__ bool operator()(float y, int e) const { return y > x || (y == x && e <= at); }
  };

  // The c-th logit, by its index, among those in [lo, hi] equal to the value of a
  // bin: its key of rank.
  __device__ __forceinline__ u64 search_equal(int lo, int hi, int bin, u64 c) const {
    const float v = B::value(bin);
    const int at = search_index(
        lo, hi, Border{Border::kFixed, c, 0.0}, 0,
        [&](int l, int h, auto f) {
          each_group(l, h, [&](const RawGroup<ES, true>& raw, int e) {
            float x[8];
            unpack_group<ES, true>(raw, x);
            int k = 0;
#pragma unroll
            for (int q = 0; q < 8; ++q) k += x[q] == v;
            f(e, (double)k);
          });
        },
        [&](float x, int) { return x == v ? 1.0 : 0.0; });
    return rank_key(v, at);
  }
};

// --------------------------------------------------------------------- cut --
// What a kernel does of a row: all of it, or where few rows are shared out to
// several workgroups each: the counts of its part; (fp32 logits and a top p) the
// masses of its part; its part's candidates or sums of kept weights; or, one
// workgroup to a row again, the rest.  What lies between the sweeps each
// workgroup of a row does by itself, with the same whole numbers.
enum CutPhase { kWhole, kCount, kMass, kSums, kRest };

// What the last kernel finds to do: nothing; the candidates of a row cut by its
// top k, or by its top p; the sums of ranges; these, without the logits of the
// last kept one's bin, which are the candidates.
enum SplitKind { kDone, kFromK, kFromP, kInRanges, kEdge };

template <int ES, int NT, bool SMALL, bool DRAW, CutPhase PHASE>
__global__ __launch_bounds__(NT, 4) void cut_kernel(CutParams P) {
  using B = Bins<ES>;
  using Row = CutRow<ES, NT, SMALL>;
  using Upto = typename Row::Upto;
  __shared__ CutShared<SMALL> S;
  constexpr bool kParts = PHASE == kCount || PHASE == kMass || PHASE == kSums;  // several workgroups to a row
  const int i = kParts ? blockIdx.y : blockIdx.x, part = kParts ? blockIdx.x : 0, tid = threadIdx.x;
  const int a0 = kParts ? part * P.seg : 0, z0 = kParts ? a0 + (min(P.seg, P.V - a0) - 1) : P.V - 1;  // the logits to sweep
  const int b = (int)P.by_R.of((uint32_t)i), r = i - b * P.R;
  const Cut cut = cut_of(P, b);
  const float u = DRAW ? P.uniforms[i] : 0.f;
  Row w{S, row_of(P, b, r, ES), P.V, P.ibits, P.frac, 0.f, 0.0};
  SplitRow* st = PHASE == kWhole ? nullptr : reinterpret_cast<SplitRow*>(P.split + (int64_t)i * P.split_row);
  // parts' counts, and their masses
  auto part_counts = [&](int g) { return reinterpret_cast<uint32_t*>(st + 1) + (int64_t)g * B::kSlots; };
  auto part_masses = [&](int g) {
    return reinterpret_cast<u64*>(reinterpret_cast<uint32_t*>(st + 1) + (int64_t)P.parts * B::kSlots) +
           (int64_t)g * B::kSlots;
  };
  auto leave = [&](SplitKind kind, u64 last, int bin, u64 before, u64 amount, bool one) {
    if (part != 0 || tid != 0) return;
    st->kind = kind;
    st->last = last;
    st->bin = bin;
    st->before = before;
    st->amount = amount;
    st->one = one;
    st->m = w.m;
  };
  auto end = [&](int token, u64 last) {  // of the row
    if (PHASE == kCount || PHASE == kMass) return;
    if (DRAW && PHASE == kSums) leave(kDone, 0, 0, 0, 0, false);
    if (tid == 0 && part == 0) {
      if constexpr (DRAW)
        P.tokens[i] = token;
      else
        P.last[i] = last;
    }
  };
  constexpr bool kTail = DRAW && PHASE == kRest;  // goes on from what the row's workgroups left
  if (kTail && st->kind == kDone) return;
  if (!cut.ok || !w.lg || (DRAW && !(u >= 0.0f && u < 1.0f))) return end(-1, kCutBad);
  if (!DRAW && (cut.greedy || cut.all)) return end(-1, kCutAll);
  if (PHASE == kMass && (cut.greedy || !(cut.p < 1.0f))) return;

  if (!kTail) w.read_tail();

  if (DRAW && !kTail && cut.greedy) {
    VI best{-INFINITY, INT_MAX};
    if constexpr (PHASE != kSums) {
      __syncthreads();
      w.each_group(a0, z0, [&](const RawGroup<ES, true>& raw, int e) {
        float x[8];
        unpack_group<ES, true>(raw, x);
#pragma unroll
        for (int q = 0; q < 8; ++q) best = vi_pick(best, VI{x[q], e + q});
      });
      best = wave_argmax(vi_floor(best, 0));  // (a row with nothing above -inf: 0)
      if ((tid & 63) == 0) {
        S.wave_f[tid >> 6] = best.v;
        S.wave_u[tid >> 6] = (uint32_t)best.i;
      }
      __syncthreads();
      if (tid != 0) return;
      for (int k = 1; k < Row::kWavesNT; ++k) best = vi_pick(best, VI{S.wave_f[k], (int)S.wave_u[k]});
      if constexpr (PHASE == kCount) {
        st->part[part].m = best.v;
        st->part[part].at = best.i;
        return;
      }
    } else if (part == 0) {
      for (int g = 0; g < P.parts; ++g) best = vi_pick(best, VI{st->part[g].m, st->part[g].at});
    }
    return end(best.i, 0);
  }

  const bool counted = !SMALL && (cut.k > 0 || cut.p < 1.0f);
  uint32_t* counts = w.counts();
  const int j0 = tid * Row::kPer, jn = max(0, min(Row::kPer, B::kN - j0));  // this thread's bins
  w.s = 1.4426950408889634074 / (double)cut.T;
  u64 last = kNone;  // the key of the last kept token
  // the candidates in LDS, where they are all that can be kept, and the end of their keys
  bool held = SMALL;
  int n = SMALL ? P.V : 0;
  u64 hi = w.rank_key(-INFINITY, 0) | w.index_mask();
  // of the logits in the bin of the last kept token: how many stay, by their
  // index, where the last one's index is still to be found (the bin, or -1)
  int tie_bin = -1;
  u64 ties = 0;

  // The candidates gathered: of the row, or of its part for the last kernel.
  auto gather = [&](float floor, auto take) __attribute__((always_inline)) {
    const int n = w.gather(a0, z0, floor, take);
    if constexpr (DRAW && PHASE == kSums) {
      if (tid == 0) S.bin = n > 0 ? atomicAdd(&st->count, n) : 0;
      __syncthreads();
      const int at = S.bin;
      for (int k = tid; k < n && at + k < kCand; k += NT) st->cand[at + k] = S.cand[k];
    }
    return n;
  };
  // The candidates up to bin `bin`, in front of which `before` stand, cut to the top k.
  auto cut_k = [&](int bin, u64 before) __attribute__((always_inline)) {
    held = true;
    last = w.bin_end(bin);
    hi = min(hi, last);
    if (n > cut.k)
      last = w.template search_lds<false, false>(n, kNone, bin > 0 ? w.bin_end(bin - 1) + 1 : 0, hi,
                                                 Border{Border::kFixed, (u64)cut.k, 0.0}, before);
  };
  auto cut_p = [&]() __attribute__((always_inline)) {
    last = min(last, w.template search_lds<false, true>(n, last, w.rank_key(w.m, 0), hi,
                                                        Border{Border::kShare, 0, (double)cut.p}, 0));
  };
  // The logits of bin `bin` that are candidates cut to `amount` of their count
  // (of one value) or their weights.
  auto cut_bin = [&](int bin, u64 amount, bool one) __attribute__((always_inline)) {
    const u64 from = bin > 0 ? w.bin_end(bin - 1) + 1 : 0;
    const Border to{Border::kFixed, amount, 0.0};
    hi = min(hi, w.bin_end(bin));
    last = min(last, one ? w.template search_lds<false, false>(n, last, from, hi, to, 0)
                         : w.template search_lds<false, true>(n, last, from, hi, to, 0));
  };
  // The key of the last place that min p leaves.
  auto min_key = [&]() __attribute__((always_inline)) {
    const double low = (double)w.m + (double)cut.T * log((double)cut.mn);
    const float f = fmaxf(__double2float_ru(low), -FLT_MAX);
    uint32_t q = place<ES>(f);
    if (ES == 2 && value_at<2>(q) < f) ++q;  // (the bf16 values not below it)
    return ((u64)((ES == 2 ? 0xffffu : 0xffffffffu) - q) << w.ibits) | w.index_mask();
  };
  const Border above{Border::kAbove, 0, (double)u};
  auto draw_held = [&]() __attribute__((always_inline)) {
    end((int)w.template search_lds<true, true>(n, last, 0, (u64)P.V - 1, above, 0), 0);
  };
  // Sums of weights by ranges of 2^shift indices, and beside them the counts of
  // logits of the tie's bin: whole groups of 8, where the row is long enough.
  const int shift = max(w.ibits - kRangeBits, 0);
  uint32_t* equal = reinterpret_cast<uint32_t*>(S.cand);
  // The token, from those of the whole row.
  auto draw_ranges = [&]() __attribute__((always_inline)) {
    if (shift < 3) {  // (few logits, one by one)
      const Upto stays(w, last);
      auto one = [&](float x, int e) { return stays(x, e) ? w.weight_of(x) : 0.0; };
      return end(w.search_index(0, P.V - 1, above, 0, [](int, int, auto) {}, one), 0);
    }
    constexpr int kMine = kRanges / NT;
    const int t = tid * kMine;
    auto none = [](int) { return (u64)0; };
    Crossing c{INT_MAX, 0, 0, 0};
    u64 stay = 0, weight = 0;
    if (tie_bin >= 0) {
      c = w.template find_crossing<kMine>(Border{Border::kFixed, ties, 0.0}, 0, t, kMine,
                                          [&](int j) { return (u64)equal[t + j]; }, none);
      stay = ties - c.before;
      weight = w.mass_of(B::value(tie_bin));
    }
    const Crossing d = w.template find_crossing<kMine>(
        above, 0, t, kMine,
        [&](int j) {
          const int at = t + j;
          const u64 same = tie_bin < 0 ? 0 : at < c.bin ? equal[at] : at == c.bin ? stay : 0;
          return S.ranges[at] + weight * same;
        },
        none);
    // inside the range a thread has few logits or one
    const int l = d.bin << shift, size = 1 << shift, mine = max(1, size / NT), e0 = l + tid * mine;
    const int n1 = max(0, min(mine, min(size, P.V - l) - tid * mine));
    Upto stays(w, last);
    if (tie_bin >= 0) {
      const float v = B::value(tie_bin);
      stays.at = d.bin < c.bin ? INT_MAX : -1;
      stays.x = v;
      if (d.bin == c.bin) {
        const Crossing f = w.template find_crossing<0>(
            Border{Border::kFixed, stay, 0.0}, 0, e0, n1,
            [&](int k) { return (u64)(load_one<ES>(w.lg, e0 + k) == v); }, none);
        stays.at = f.bin;
      }
    }
    const Crossing f = w.template find_crossing<0>(
        Border{Border::kFixed, d.border, 0.0}, d.before, e0, n1,
        [&](int k) {
          const float x = load_one<ES>(w.lg, e0 + k);
          return stays(x, e0 + k) ? w.mass_of(x) : 0;
        },
        none);
    end(f.bin, 0);
  };

  if constexpr (kTail) {
    const int kind = st->kind;
    w.m = st->m;
    last = st->last;
    n = min(st->count, kCand);
    if (kind != kInRanges) {
      for (int k = tid; k < n; k += NT) S.cand[k] = st->cand[k];
      __syncthreads();
    }
    if (kind == kFromK) {
      cut_k(st->bin, st->before);
      if (cut.p < 1.0f) cut_p();
    } else if (kind == kFromP || kind == kEdge) {
      cut_bin(st->bin, st->amount, st->one);
    }
    if (kind != kInRanges && cut.mn > 0.0f) last = min(last, min_key());
    if (kind == kFromK || kind == kFromP) return draw_held();
    for (int k = tid; k < kRanges; k += NT) S.ranges[k] = st->ranges[k];
    if (kind == kEdge) {
      __syncthreads();
      for (int k = tid; k < n; k += NT) {
        const u64 key = S.cand[k];
        if (key <= last) atomicAdd(&S.ranges[(key & w.index_mask()) >> shift], w.mass_of(w.key_logit(key)));
      }
    } else if (st->bin >= 0) {
      tie_bin = st->bin;
      ties = st->amount;
      for (int k = tid; k < kRanges; k += NT) equal[k] = st->equal[k];
    }
    return draw_ranges();
  }

  // the counts of the bins, the largest logit, and whether there is a NaN
  float m = -INFINITY;
  uint32_t big = 0, small = ~0u;
  bool nan = false, odd = false;
  if (counted && (PHASE == kWhole || PHASE == kCount)) {
    // (the last bin holds what the others do not: masked logits, of which a row may
    // have mostly, would all add in one place)
    constexpr int kLowest = B::kSlots - 1;
    static_assert(B::slot_of(B::kN - 1) == kLowest, "the last bin's");
    for (int j = tid; j < B::kSlots; j += NT) counts[j] = 0;
    __syncthreads();
    w.each_group(a0, z0, [&](const RawGroup<ES, true>& raw, int) {
      if constexpr (ES == 2) {
        uint32_t slot[8];
        slots8(raw, slot);
        u16x2 mag{0, 0};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t two = raw.v[q] & 0x7fff7fffu;
          mag = __builtin_elementwise_max(mag, __builtin_bit_cast(u16x2, two));
        }
        big = max(big, (uint32_t)max(mag.x, mag.y) << 16);
        if (__ballot(lowest8(raw))) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (slot[q] != kLowest) atomicAdd(&counts[slot[q]], 1u);
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q) atomicAdd(&counts[slot[q]], 1u);
        }
      } else {
        float x[8];
        unpack_group<ES, true>(raw, x);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          m = fmaxf(m, x[q]);
          big = max(big, __float_as_uint(x[q]) & 0x7fffffffu);
          const int slot = B::slot(x[q]);
          if (slot != kLowest) atomicAdd(&counts[slot], 1u);
        }
      }
    });
    __syncthreads();
    uint32_t sum = 0;
    for (int j = tid; j < kLowest; j += NT) sum += j != 0 && j != B::kHalf ? counts[j] : 0;
    sum = (uint32_t)wave_scan_u64(sum);
    if (tid == 0) {
      const uint32_t mid = counts[0] + counts[B::kHalf];  // zeros and the like of either sign
      counts[0] = mid;
      counts[B::kHalf] = 0;
      atomicAdd(&counts[kLowest], (uint32_t)(z0 - a0 + 1) - mid);
    }
    if ((tid & 63) == 63) atomicSub(&counts[kLowest], sum);
    __syncthreads();
  }
  if (PHASE != kWhole && PHASE != kCount) {
    if (counted) {
      // (all parts' on their way together)
      for (int j = 4 * tid; j < B::kSlots; j += 4 * NT) {
        u32x4 c[kCutParts], sum{0, 0, 0, 0};
#pragma unroll
        for (int g = 0; g < kCutParts; ++g)
          c[g] = *reinterpret_cast<const u32x4*>(part_counts(min(g, P.parts - 1)) + j);
#pragma unroll
        for (int g = 0; g < kCutParts; ++g) sum += g < P.parts ? c[g] : u32x4{0, 0, 0, 0};
        *reinterpret_cast<u32x4*>(counts + j) = sum;
      }
      __syncthreads();
    }
    uint32_t flags = 0;
#pragma unroll
    for (int g = 0; g < kCutParts; ++g) {
      m = fmaxf(m, st->part[min(g, P.parts - 1)].m);
      flags |= st->part[min(g, P.parts - 1)].flags;
    }
    nan = flags & 1u;
    odd = flags & 2u;
    big = flags & 4u ? ~0u : 0;
  }
  if (ES == 2 && counted && (PHASE == kWhole || PHASE == kCount)) {  // the largest logit from the first bin, where that is one value
    int first = B::kN;
    for (int j = jn - 1; j >= 0; --j)
      if (counts[B::slot_of(j0 + j)]) first = j0 + j;
    first = (int)-w.block_max((float)-first);
    if (B::single(first)) m = B::value(first);
  }
  if ((PHASE == kWhole || PHASE == kCount) && (ES == 2 || !counted) && !(m > -INFINITY)) {
    if (!counted) __syncthreads();
    w.each_group(a0, z0, [&](const RawGroup<ES, true>& raw, int e) {
      float x[8];
      unpack_group<ES, true>(raw, x);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const uint32_t mag = __float_as_uint(x[q]) & 0x7fffffffu;
        m = fmaxf(m, x[q]);
        big = max(big, mag);
        small = min(small, mag);
        if (SMALL && e + q < P.V) S.cand[e + q] = w.rank_key(x[q], e + q);
      }
    });
  }
  w.m = w.block_max(m);
  if (PHASE == kWhole || PHASE == kCount) {
    nan = __syncthreads_or(big > 0x7f800000u);
    if constexpr (!SMALL)  // logits whose bins are of several values, those of -2^7 and below apart
      odd = __syncthreads_or(!counted && small < (B::kLo << B::kShift)) || (!counted && w.m >= 128.0f);
  }
  if constexpr (PHASE == kCount) {
    const bool far = __syncthreads_or(big >= (B::kHi << B::kShift));
    if (counted)
      for (int j = tid; j < B::kSlots; j += NT) part_counts(part)[j] = counts[j];
    if (tid == 0) {
      st->part[part].m = w.m;
      st->part[part].flags = (nan ? 1u : 0u) | (odd ? 2u : 0u) | (far ? 4u : 0u);
      if (part == 0) st->count = 0;
    }
    return;
  }
  if (nan || !(fabsf(w.m) <= FLT_MAX)) return end(-1, kCutAll);
  auto count_of = [&](int j) { return (u64)counts[B::slot_of(j0 + j)]; };

  int k_bin = B::kN;
  u64 k_rest = 0;
  if (cut.k > 0) {
    const Border to{Border::kFixed, (u64)cut.k, 0.0};
    if constexpr (SMALL) {
      last = w.template search_lds<false, false>(n, kNone, w.rank_key(w.m, 0), hi, to, 0);
    } else {
      const Crossing c = w.template find_crossing<0>(to, 0, j0, jn, count_of, count_of);
      k_bin = c.bin;
      k_rest = (u64)cut.k - c.before;
      last = w.bin_end(k_bin);
      if (c.through <= kCand) {
        if (PHASE == kMass) return;
        n = gather(B::least(k_bin), [](u64) { return true; });
        if constexpr (DRAW && PHASE == kSums) return leave(kFromK, last, c.bin, c.before, 0, false);
        cut_k(c.bin, c.before);
      } else if (c.through > (u64)cut.k) {
        if (B::single(k_bin)) {
          tie_bin = k_bin;
          ties = k_rest;
        } else {
          last = w.template search_bin<false>(k_bin, kNone, k_rest);
        }
      }
    }
  }
  int edge_bin = -1;
  u64 edge = 0;
  if (cut.p < 1.0f) {
    if (held) {
      cut_p();
    } else if constexpr (!SMALL) {
      // the masses of bins with several values, logit by logit (those of -2^7 and below mostly have none)
      u64* masses = w.masses();
      if (tid < 3) S.special[tid] = 0;
      if (ES == 4 && PHASE != kSums && PHASE != kRest)
        for (int j = tid; j < B::kSlots; j += NT) masses[j] = 0;
      const bool low = counts[B::slot_of(B::kN - 1)] != 0 && w.low_weighs();
      const bool some = counts[B::slot_of(0)] != 0 || counts[B::slot_of(B::kMid)] != 0 || low;
      __syncthreads();
      const Upto stays(w, last);
      if (ES == 4 && (PHASE == kSums || PHASE == kRest)) {
        for (int j = 2 * tid; j < B::kSlots; j += 2 * NT) {
          u64x2 y[kCutParts], sum{0, 0};
#pragma unroll
          for (int g = 0; g < kCutParts; ++g)
            y[g] = *reinterpret_cast<const u64x2*>(part_masses(min(g, P.parts - 1)) + j);
#pragma unroll
          for (int g = 0; g < kCutParts; ++g) sum += g < P.parts ? y[g] : u64x2{0, 0};
          masses[j] = sum.x;
          masses[j + 1] = sum.y;
        }
      } else if (ES == 4) {
        w.each_group(a0, z0, [&](const RawGroup<ES, true>& raw, int e) {
          float x[8];
          unpack_group<ES, true>(raw, x);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const u64 y = stays(x[q], e + q) ? w.mass_of(x[q]) : 0;
            if (y) atomicAdd(&masses[B::slot(x[q])], y);  // (the slots of the middle bin are added up below)
          }
        });
        __syncthreads();
        if (tid == 0) masses[0] += masses[B::kHalf];
      } else if (some) {
        w.each_group(0, P.V - 1, [&](const RawGroup<ES, true>& raw, int e) {
          if constexpr (ES == 2)
            if (!special8(raw, low)) return;
          float x[8];
          unpack_group<ES, true>(raw, x);
#pragma unroll 1
          for (int q = 0; q < 8; ++q) {
            const int bin = B::of(x[q]);
            if (!B::single(bin) && stays(x[q], e + q))
              atomicAdd(&S.special[bin == 0 ? 0 : bin == B::kMid ? 1 : 2], w.mass_of(x[q]));
          }
        });
      }
      if constexpr (PHASE == kMass) {
        __syncthreads();
        for (int j = tid; j < B::kSlots; j += NT) part_masses(part)[j] = masses[j];
        return;
      }
      auto mass = [&](int j) -> u64 {
        const int bin = j0 + j;
        if constexpr (ES == 4) return masses[B::slot_of(bin)];
        if (!B::single(bin)) return S.special[bin == 0 ? 0 : bin == B::kMid ? 1 : 2];
        const u64 c = bin < k_bin ? counts[B::slot_of(bin)] : bin == k_bin ? k_rest : 0;
        return c ? c * w.mass_of(B::value(bin)) : 0;
      };
      const Crossing c = w.template find_crossing<Row::kPer <= 8 ? Row::kPer : 0>(Border{Border::kShare, 0, (double)cut.p},
                                                                                  0, j0, jn, mass, count_of);
      const u64 rest = c.border - c.before;
      u64 one = 0, stay = 0;
      if (B::single(c.bin)) {  // (of equal logits as many as reach it)
        one = w.mass_of(B::value(c.bin));
        stay = (rest + one - 1) / one;
      }
      if (c.through <= kCand) {
        n = gather(B::least(c.bin), [&](u64 key) { return key <= last; });
        if constexpr (DRAW && PHASE == kSums)
          return leave(kFromP, last, c.bin, 0, one ? stay : rest, one != 0);
        held = true;
        cut_bin(c.bin, one ? stay : rest, one != 0);
        tie_bin = -1;
      } else if (one) {
        if (c.bin < k_bin) {  // (in the k-th token's bin the rest of that is known)
          last = w.bin_end(c.bin);
          tie_bin = -1;
        }
        if (stay < counts[B::slot_of(c.bin)]) {
          tie_bin = c.bin;
          ties = stay;
        }
      } else if (ES == 4 && DRAW && PHASE == kSums && counts[B::slot_of(c.bin)] <= kCand) {
        edge_bin = c.bin;  // (its border is found among its candidates, later)
        edge = rest;
      } else {
        last = w.template search_bin<true>(c.bin, last, rest);
        tie_bin = -1;
      }
    }
  }
  if (cut.mn > 0.0f) {
    const u64 at = min_key();
    if (tie_bin >= 0 && at < w.rank_key(B::value(tie_bin), 0)) tie_bin = -1;
    if (edge_bin > 0 && at <= w.bin_end(edge_bin - 1)) edge_bin = -1;
    if (edge_bin < 0) last = min(last, at);
  }
  // (a draw finds the last index together with its sums, where it goes by ranges of whole groups)
  if (!SMALL && tie_bin >= 0 && (!DRAW || shift < 3)) {
    last = w.search_equal(0, P.V - 1, tie_bin, ties);
    tie_bin = -1;
  }
  if constexpr (!DRAW) return end(0, min(last, (u64)kCutAll - 1));

  if constexpr (PHASE == kWhole)
    if (held) return draw_held();
  if constexpr (!SMALL) {
    if (edge_bin >= 0) {
      const u64 first = edge_bin > 0 ? w.bin_end(edge_bin - 1) + 1 : 0, end = min(last, w.bin_end(edge_bin));
      gather(B::least(edge_bin), [&](u64 key) { return key >= first && key <= end; });
      leave(kEdge, last, edge_bin, 0, edge, false);
      __syncthreads();
      last = edge_bin > 0 ? first - 1 : w.rank_key(INFINITY, 0);  // the sums: of what is in front of it
    }
    const float floor = last == kNone ? -INFINITY : w.key_logit(last);
    const Upto stays(w, last);
    auto one = [&](float x, int e) { return stays(x, e) ? w.weight_of(x) : 0.0; };
    if (shift >= 3) {
      const Floor<ES> kept(floor);
      if constexpr (ES == 2) {
        // the weight of each bin, 0 behind the last kept one's and for bins of
        // several values
        const int end_bin = B::of(floor);
        double* weights = w.weights();
        __syncthreads();
        // whether some of a bin of several values may stay, with a weight
        const bool low = end_bin == B::kN - 1 && w.low_weighs();
        if (counted)
          odd = counts[B::slot_of(0)] != 0 || counts[0] != 0 || (low && counts[B::slot_of(B::kN - 1)] != 0);
        else
          odd = __syncthreads_or(odd || (low && big >= (B::kHi << B::kShift)));
        __syncthreads();
        for (int j = tid; j < B::kN; j += NT)
          weights[B::slot_of(j)] = j <= end_bin && j != tie_bin && B::single(j) ? w.weight_of(B::value(j)) : 0.0;
        if (tid == 0) weights[B::kHalf] = 0.0;
        for (int j = tid; j < kRanges; j += NT) equal[j] = 0;
        w.clear_ranges();
        auto sum_of = [&](const RawGroup<2, true>& raw, const uint32_t (&slot)[8], int e) __attribute__((always_inline)) {
          double sum = 0.0;
#pragma unroll
          for (int q = 0; q < 8; ++q) sum += weights[slot[q]];
          if (odd && special8(raw, low)) {
            float x[8];
            unpack_group<2, true>(raw, x);
#pragma unroll 1
            for (int q = 0; q < 8; ++q)
              if (!B::single(B::of(x[q]))) sum += one(x[q], e + q);
          }
          return sum;
        };
        auto sweep = [&](auto tie) __attribute__((always_inline)) {
          const uint32_t end_slot = (uint32_t)B::slot_of(max(tie_bin, 0));
          w.each_group(a0, z0, [&](const RawGroup<2, true>& raw, int e) {
            if (!__ballot(kept.reached(raw))) return;
            uint32_t slot[8], same = 0;
            slots8(raw, slot);
            if constexpr (tie) {
#pragma unroll
              for (int q = 0; q < 8; ++q) same += slot[q] == end_slot;
            }
            w.add_range(S.ranges, e >> shift, shift, sum_of(raw, slot, e));
            if (tie && same) atomicAdd(&equal[e >> shift], same);
          });
        };
        if (tie_bin >= 0)
          sweep(std::true_type{});
        else
          sweep(std::false_type{});
      } else {
        w.clear_ranges();
        w.each_group(a0, z0, [&](const RawGroup<4, true>& raw, int e) {
          if (!__ballot(kept.reached(raw))) return;
          float x[8];
          unpack_group<4, true>(raw, x);
          double sum = 0.0;
#pragma unroll 4
          for (int q = 0; q < 8; ++q) sum += one(x[q], e + q);
          w.add_range(S.ranges, e >> shift, shift, sum);
        });
      }
    }
    if constexpr (PHASE == kSums) {
      __syncthreads();
      for (int k = (a0 >> shift) + tid; k <= z0 >> shift; k += NT) {
        st->ranges[k] = S.ranges[k];
        if (tie_bin >= 0) st->equal[k] = equal[k];
      }
      if (part == 0)
        for (int k = (P.V - 1 >> shift) + 1 + tid; k < kRanges; k += NT) {
          st->ranges[k] = 0;
          st->equal[k] = 0;
        }
      if (edge_bin < 0) leave(kInRanges, last, tie_bin, 0, ties, false);
      return;
    }
    draw_ranges();
  }
}

// --------------------------------------------------------------- truncate --
// The rows with what was left out at -inf: memory's rate (a copy's in effect, 5.6
// TB/s for 288 rows of 151936).  In place, groups that stay whole are not written.
template <int ES>
__global__ __launch_bounds__(kWG) void truncate_kernel(CutParams P) {
  const int i = (int)P.by_C.of(blockIdx.x), chunk = blockIdx.x - i * P.C;
  const int b = (int)P.by_R.of((uint32_t)i), r = i - b * P.R;
  const u64 last = P.last[i];
  const char* src = P.logits + ((int64_t)b * P.req + (int64_t)r * P.row) * ES;
  char* dst = P.out + ((int64_t)b * P.out_req + (int64_t)r * P.out_row) * ES;
  if (last == kCutAll && src == dst) return;
  const float fill = last == kCutBad ? __builtin_nanf("") : -INFINITY;
  const int64_t e0 = (int64_t)chunk * P.chunk, e1 = min((int64_t)P.V, e0 + P.chunk);
  for (int64_t e = e0 + threadIdx.x * 8; e < e1; e += kWG * 8) {
    const RawGroup<ES, true> g = load_end<ES>(src, e, P.V);
    bool some = false;
    float x[8];
    unpack_group<ES, true>(g, x);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const bool keep = last == kCutAll || (last < kCutAll && key_of<ES>(x[q], (int)e + q, P.ibits) <= last);
      some |= !keep;
      x[q] = keep ? x[q] : fill;
    }
    if (!some && src == dst) continue;
    store_end<ES>(dst, e, P.V, x);
  }
}

// 1024 threads to a row up to 256 rows, a row to a CU, and 512 beyond, two rows to
// a CU: 256 rows of 151936 bf16 logits 53 us against 58 with 512, of 40000 fp32
// ones 64 against 68; with 1024 beyond, 288 rows of 151936 drawn with settings of
// their own 91 us against 74, uncut 67 against 56, cut 116 against 102 (by top k 97
// against 82), 261 rows cut 89 against 80, 504 rows 141 against 121.
template <int ES, bool DRAW>
static hipError_t launch_rows(const CutParams& P, unsigned rows, hipStream_t stream) {
  if (P.parts > 1) {
    const dim3 grid((unsigned)P.parts, rows);
    hipLaunchKernelGGL((cut_kernel<ES, 1024, false, DRAW, kCount>), grid, dim3(1024), 0, stream, P);
    if constexpr (ES == 4)
      if (P.top_p) hipLaunchKernelGGL((cut_kernel<ES, 1024, false, DRAW, kMass>), grid, dim3(1024), 0, stream, P);
    if constexpr (DRAW)
      hipLaunchKernelGGL((cut_kernel<ES, 1024, false, DRAW, kSums>), grid, dim3(1024), 0, stream, P);
    hipLaunchKernelGGL((cut_kernel<ES, 1024, false, DRAW, kRest>), dim3(rows), dim3(1024), 0, stream, P);
  } else if (P.V <= kCand) {
    hipLaunchKernelGGL((cut_kernel<ES, 256, true, DRAW, kWhole>), dim3(rows), dim3(256), 0, stream, P);
  } else if (rows <= 256) {
    hipLaunchKernelGGL((cut_kernel<ES, 1024, false, DRAW, kWhole>), dim3(rows), dim3(1024), 0, stream, P);
  } else {
    hipLaunchKernelGGL((cut_kernel<ES, 512, false, DRAW, kWhole>), dim3(rows), dim3(512), 0, stream, P);
  }
  return hipGetLastError();
}

template <int ES>
static hipError_t launch_cut_typed(const CutParams& P, hipStream_t stream) {
  const unsigned rows = (unsigned)(P.B * P.R);
  if (P.tokens) return launch_rows<ES, true>(P, rows, stream);
  const hipError_t e = launch_rows<ES, false>(P, rows, stream);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((truncate_kernel<ES>), dim3(rows * (unsigned)P.C), dim3(kWG), 0, stream, P);
  return hipGetLastError();
}

hipError_t launch_cut(const CutParams& P, int dtype, hipStream_t stream) {
  return dtype == SPEC_BF16 ? launch_cut_typed<2>(P, stream) : launch_cut_typed<4>(P, stream);
}

}  // namespace specv
