// cache4.hip -- rotary positions, and the 4-bit paged KV cache: queries and keys
// rotated, keys and values quantised as they are written at the slots of a
// slot mapping, and read back, on gfx950.
//
// Rotation: pair i of a head, (x, y), at position p becomes
//   (x cos a - y sin a, y cos a + x sin a) * scale,  a = p * inv_freq[i],
// pairs (i, i + rot / 2), or (2 i, 2 i + 1) interleaved.  The angle, its cosine
// and sine are taken in fp64: an angle of a far position has no correct fraction
// in fp32.  They are worked out once for all heads of a token.  The products of
// fp32 elements, and of keys that go into the cache, are fp64's too, rounded
// once: the codes are then those of the exact values (an fp32 product next to
// the border of two codes picks the wrong one about once in a million).  Those
// that become bf16 elements are fp32's, off by at most 2^-24 (2 |x cos a| + 3 |y
// sin a|) |scale| (cosine and sine rounded, one product, the sum): far below half a
// step of bf16, 2^-9 of the larger elements, but where the two products cancel.
//
// Cache: 32 consecutive elements of a token's head share the scale 2^e, e the
// smallest exponent with |x| <= 6 * 2^e, and are held as e2m1 codes (0, 0.5, 1,
// 1.5, 2, 3, 4, 6 and a sign), the microscaled format that the widening
// instructions read.  A scale belongs to one token, so every token is written
// by itself: no order among the writers, nothing read back.
//
// Bounds, measured (MI355X): memory.  8190 tokens of 32 + 8 heads of 128, half of
// each rotated: 38 us with inputs past the caches (4.4 TB/s read and written), 30
// with part of them within.  24000 tokens of 32 + 8 + 8 heads of 128 rotated and
// written: 119 us, 4.4 TB/s; the cache's part read back as bf16 22 us, 5.7 TB/s.
// A decode step's 64 tokens take 4 us, what a launch takes.
//
#include <type_traits>

#include "cache_device.hpp"
#include "unaligned.hpp"

namespace specv {

// sin and cos of an fp64 angle by its multiple of pi / 2 (in two parts, so that
// the rest keeps full precision up to 2^31 radians) and the power series: the
// terms left out are below 2^-53 for |r| <= pi / 4.
__device__ __forceinline__ void sin_cos(double a, double& sn, double& cs) {
  constexpr double kTwoOverPi = 0.63661977236758134308, kHi = 0x1.921fb54442d18p+0, kLo = 0x1.1a62633145c07p-54;
  const double n = __builtin_rint(a * kTwoOverPi);
  const double r = __builtin_fma(-n, kLo, __builtin_fma(-n, kHi, a));
  const double z = r * r;
  double s = -1.0 / 1307674368000.0;  // 1 / 15!
  s = __builtin_fma(s, z, 1.0 / 6227020800.0);
  s = __builtin_fma(s, z, -1.0 / 39916800.0);
  s = __builtin_fma(s, z, 1.0 / 362880.0);
  s = __builtin_fma(s, z, -1.0 / 5040.0);
  s = __builtin_fma(s, z, 1.0 / 120.0);
  s = __builtin_fma(s, z, -1.0 / 6.0);
  s = __builtin_fma(s * z, r, r);
  double c = 1.0 / 20922789888000.0;  // 1 / 16!
  c = __builtin_fma(c, z, -1.0 / 87178291200.0);
  c = __builtin_fma(c, z, 1.0 / 479001600.0);
  c = __builtin_fma(c, z, -1.0 / 3628800.0);
  c = __builtin_fma(c, z, 1.0 / 40320.0);
  c = __builtin_fma(c, z, -1.0 / 720.0);
  c = __builtin_fma(c, z, 1.0 / 24.0);
  c = __builtin_fma(c, z, -0.5);
  c = __builtin_fma(c, z, 1.0);
  const int q = (int)__builtin_fma(-4.0, __builtin_floor(n * 0.25), n);  // n mod 4
  const double a0 = (q & 1) ? c : s, b0 = (q & 1) ? s : c;
  sn = (q & 2) ? -a0 : a0;
  cs = ((q + 1) & 2) ? -b0 : b0;
}

// y rounded to fp32 so that a later rounding to fewer bits gives what rounding
// y itself would (inexact: to the neighbour whose last bit is 1).  What rounds
// to 2^128 becomes infinite.
__device__ __forceinline__ float to_odd(double y) {
  const float f = (float)y;
  const double d = y - (double)f;
  uint32_t u = __float_as_uint(f);
  if (d != 0.0 && fabsf(f) <= FLT_MAX && !(u & 1u)) u += (d > 0.0) == (y > 0.0) ? 1u : ~0u;
  return __uint_as_float(u);
}

// The smallest e with amax <= 6 * 2^e, at least kScaleMin; amax finite.
__device__ __forceinline__ int exponent4(float amax) {
  const uint32_t u = __float_as_uint(amax);
  return max((int)(u >> 23) - 127 - 2 + ((u & 0x7fffffu) > 0x400000u ? 1 : 0), kScaleMin);
}

// Eight values at the scale 2^e as codes, the first in the lowest bits, rounded
// to nearest even.
__device__ __forceinline__ uint32_t encode8(const float x[8], float scale) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], scale, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], scale, 3);
}

typedef uint32_t u32x4_any_out __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_any_out __attribute__((ext_vector_type(4), aligned(4)));

// (Written past the caches: 145 us against 152 for 24000 tokens of 32 + 8 + 8 heads
// of 128 rotated, written and read back, 17 against 19 for 2000 fp32 tokens; bf16
// heads of 64, whose pieces are half lines, the other way: 38 against 37.)
template <int ES>
__device__ __forceinline__ void store8(char* dst, const float x[8]) {
  if constexpr (ES == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = round_bf16x2(x[2 * i], x[2 * i + 1]);
    __builtin_nontemporal_store(u32x4{w[0], w[1], w[2], w[3]}, reinterpret_cast<u32x4_any_out*>(dst));
  } else {
    __builtin_nontemporal_store(f32x4{x[0], x[1], x[2], x[3]}, reinterpret_cast<f32x4_any_out*>(dst));
    __builtin_nontemporal_store(f32x4{x[4], x[5], x[6], x[7]}, reinterpret_cast<f32x4_any_out*>(dst + 16));
  }
}

// A pair turned by its cosine and sine.
template <class T>
__device__ __forceinline__ void turn(T& x, T& y, T c, T s) {
  const T u = x;
  x = __builtin_fma(x, c, -(y * s));
  y = __builtin_fma(u, s, y * c);
}

// A lane takes two groups of 8 elements of one head of a token, a and b.  Where
// pairs lie apart: in the rotated part groups half of it apart, whose elements
// are pairs of each other, behind it groups half of the rest apart.  Where they
// lie side by side: groups half of the head apart.  Every pair is one lane's, and
// in place nothing is overwritten that another lane reads; a load or store of a
// head's lanes covers whole lines where it can.
// Grid: x sets of P.tokens tokens, y shares of their heads.  The heads of a
// set's tokens, end to end, go to the lanes in rounds.  (Two rounds' reads on
// their way together: 166 us against 122 for 24000 tokens of 32 + 8 + 8 heads of
// 128; the registers cost more waves than that gains.)
template <int ES, bool WRITE, bool INTER>
__global__ __launch_bounds__(kWG) void rope_kernel(RopeParams P) {
  // cosine and sine of a group's pair q at [token][q][group of the head], in both
  // precisions: neighbouring lanes read neighbouring places
  __shared__ double2 s_turn[kRopeAngles];
  __shared__ float2 s_turn32[kRopeAngles];
  __shared__ __align__(16) float s_max[WRITE ? kWG * 2 : 1];
  const int tid = threadIdx.x;
  // turned: groups of a head whose elements are turned, with pairs apart those of a
  const int half = P.half, turned = INTER ? half >> 2 : half >> 3;
  const int n0 = blockIdx.x * P.tokens;
  const int tokens = min(P.tokens, P.N - n0);
  for (int i = tid; i < tokens * half; i += kWG) {
    const int t = i / half, f = i - t * half;
    const double at = P.wide ? (double)static_cast<const int64_t*>(P.positions)[n0 + t]
                             : (double)static_cast<const int32_t*>(P.positions)[n0 + t];
    double sn, cs;
    sin_cos(at * P.inv_freq[f], sn, cs);
    constexpr int kPairs = INTER ? 4 : 8;  // of a group
    const int place = t * half + f % kPairs * turned + f / kPairs;
    s_turn[place] = double2{cs * P.scale, sn * P.scale};
    s_turn32[place] = float2{(float)(cs * P.scale), (float)(sn * P.scale)};
  }
  __syncthreads();
  const int lanes = (P.dim + 15) >> 4, per = kWG / lanes;
  const int heads = P.heads[0] + (WRITE ? 2 : 1) * P.heads[1];
  const int mine = tid / lanes, lane = tid - mine * lanes;
  const int groups = P.dim >> 3;
  const int front = INTER ? lanes : (groups - 2 * turned + 1) >> 1;  // from a to b, where b is no partner
  const bool turn_a = lane < turned, turn_b = INTER ? lane + front < turned : turn_a;
  const int group_a = INTER || turn_a ? lane : lane + turned, group_b = !INTER && turn_a ? lane + turned : group_a + front;
  const int col_a = 8 * group_a, col_b = 8 * group_b;
  const bool two = group_b < groups;  // (else the second group does not exist)
  const int items = tokens * heads, rounds = (items + per - 1) / per;
  for (int r = blockIdx.y; r < rounds; r += gridDim.y) {
    const int item = r * per + mine;
    const bool on = mine < per && item < items;
    const int token = (int)P.by_heads.of((uint32_t)min(item, items - 1)), h = item - token * heads, n = n0 + token;
    const int what = h < P.heads[0] ? 0 : h < P.heads[0] + P.heads[1] ? 1 : 2;  // queries, keys, values
    const int head = h - (what == 1 ? P.heads[0] : what == 2 ? P.heads[0] + P.heads[1] : 0);
    float a[8], b[8];
    if (on) {
      const char* src = P.src[what] + ((int64_t)n * P.tok[what] + (int64_t)head * P.hd[what]) * ES;
      // (past the caches a line of which each load takes half comes twice: 38 us
      // against 28 for the keys and values of 24000 tokens)
      const RawGroup<ES, true> raw_a = load_cached<ES>(src, col_a), raw_b = load_cached<ES>(src, two ? col_b : col_a);
      unpack_group<ES, true>(raw_a, a);
      unpack_group<ES, true>(raw_b, b);
      if ((turn_a || turn_b) && what < 2) {
        const int at = token * half + lane;
        auto turn16 = [&](auto& a, auto& b, auto* table) {
          using T = std::remove_reference_t<decltype(a[0])>;
          if constexpr (INTER) {
            if (turn_a)
#pragma unroll
              for (int q = 0; q < 4; ++q)
                turn<T>(a[2 * q], a[2 * q + 1], table[at + q * turned].x, table[at + q * turned].y);
            if (turn_b)
#pragma unroll
              for (int q = 0; q < 4; ++q)
                turn<T>(b[2 * q], b[2 * q + 1], table[at + front + q * turned].x, table[at + front + q * turned].y);
          } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) turn<T>(a[q], b[q], table[at + q * turned].x, table[at + q * turned].y);
          }
        };
        if (ES == 2 && (!WRITE || what == 0)) {
          turn16(a, b, s_turn32);
        } else {
          double x[8], y[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            x[q] = a[q];
            y[q] = b[q];
          }
          turn16(x, y, s_turn);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            a[q] = WRITE && what == 1 ? to_odd(x[q]) : (float)x[q];
            b[q] = WRITE && what == 1 ? to_odd(y[q]) : (float)y[q];
          }
        }
      }
      if (!WRITE || what == 0) {
        char* dst = P.dst[what] + ((int64_t)n * P.dtok[what] + (int64_t)head * P.dhd[what]) * ES;
        store8<ES>(dst + col_a * ES, a);
        if (two) store8<ES>(dst + col_b * ES, b);
      }
    }
    if constexpr (WRITE) {
      const bool kept = on && what > 0;
      float* top = s_max + mine * 2 * lanes;  // the largest of each group of 8 of the head
      if (kept) {
        float ma = 0.f, mb = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float x = fabsf(a[q]), y = fabsf(b[q]);
          ma = fmaxf(ma, x <= FLT_MAX ? x : INFINITY);
          mb = fmaxf(mb, y <= FLT_MAX ? y : INFINITY);
        }
        top[col_a >> 3] = ma;
        top[col_b >> 3] = mb;
      }
      // (a head's lanes are in one wave where they divide it)
      if (64 % lanes == 0) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
      } else {
        __syncthreads();
      }
      int64_t slot = -1;
      if (kept) {
        slot = P.slots[n];
        // of equal slots next to each other the last counts
        if (slot >= (int64_t)P.c.num_blocks << P.c.bs_shift || (n + 1 < P.N && P.slots[n + 1] == slot)) slot = -1;
      }
      if (slot >= 0) {
        const int64_t blk = slot >> P.c.bs_shift;
        const int in = (int)(slot & ((1 << P.c.bs_shift) - 1));
        uint8_t* codes = P.c.codes[what - 1] + blk * P.c.block + (int64_t)in * P.c.token + (int64_t)head * P.c.head;
        uint8_t* scales = P.c.scales[what - 1] + blk * P.c.sblock + (int64_t)head * P.c.shead + in;
        auto put = [&](const float (&x)[8], int col) {
          const f32x4 m = *reinterpret_cast<const f32x4*>(&top[(col >> 5) * 4]);
          const float amax = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
          const bool fine = amax <= FLT_MAX;
          const int e = fine ? exponent4(amax) : 0;
          const uint32_t w = encode8(x, two_to(e));
          *reinterpret_cast<uint32_t*>(codes + (col >> 1)) = fine ? w : 0u;
          if ((col & 31) == 0) scales[(col >> 5) << P.c.bs_shift] = (uint8_t)(fine ? e + kScaleBias : 255);
        };
        put(a, col_a);
        put(b, col_b);
      }
      // (the next round writes there)
      if (64 % lanes == 0) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
      } else {
        __syncthreads();
      }
    }
  }
}

template <int ES, bool WRITE>
static hipError_t launch_rope_typed(const RopeParams& P, hipStream_t stream) {
  const dim3 grid((unsigned)((P.N + P.tokens - 1) / P.tokens), (unsigned)P.shares);
  if (P.inter)
    hipLaunchKernelGGL((rope_kernel<ES, WRITE, true>), grid, dim3(kWG), 0, stream, P);
  else
    hipLaunchKernelGGL((rope_kernel<ES, WRITE, false>), grid, dim3(kWG), 0, stream, P);
  return hipGetLastError();
}

hipError_t launch_rope(const RopeParams& P, int dtype, hipStream_t stream) {
  if (P.write) return dtype == SPEC_BF16 ? launch_rope_typed<2, true>(P, stream) : launch_rope_typed<4, true>(P, stream);
  return dtype == SPEC_BF16 ? launch_rope_typed<2, false>(P, stream) : launch_rope_typed<4, false>(P, stream);
}

// One lane takes 8 elements of one (entry, head) row, keys and values, a cell;
// a workgroup takes P.per entries, and a lane has the loads of kReadCells
// cells on their way together.  Written past the caches (of 24000 tokens of 8
// heads of 128: 5 us less).
template <int ES>
__global__ __launch_bounds__(kWG) void kv4_read_kernel(KvReadParams P) {
  const CacheView& c = P.c;
  const uint32_t lpt = (uint32_t)c.dim >> 3, cells = (uint32_t)c.heads * lpt;  // of an entry, at most 2^15
  const int i0 = blockIdx.x * P.per;
  const uint32_t total = cells * (uint32_t)min(P.per, P.N - i0);
  for (uint32_t x0 = threadIdx.x; x0 < total; x0 += kWG * kReadCells) {
    uint32_t w[2][kReadCells];
    float f[2][kReadCells];
#pragma unroll
    for (int q = 0; q < kReadCells; ++q) {
      const uint32_t x = min(x0 + q * kWG, total - 1);  // (a lane past the end reads the last cell and stores nothing)
      const uint32_t e = x / cells, cell = x - e * cells;
      const uint32_t h = cell / lpt, col = (cell - h * lpt) * 8;
      const int64_t s = P.slots[i0 + e];
      const bool in = s >= 0 && s < ((int64_t)c.num_blocks << c.bs_shift);
      const int64_t blk = in ? s >> c.bs_shift : 0;
      const int t = in ? (int)(s & ((1 << c.bs_shift) - 1)) : 0;
      const int64_t at = blk * c.block + (int64_t)t * c.token + (int64_t)h * c.head + (col >> 1);
      const int64_t sat = blk * c.sblock + (int64_t)h * c.shead + ((int64_t)(col >> 5) << c.bs_shift) + t;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint32_t v = *reinterpret_cast<const uint32_t*>(c.codes[kv] + at);
        const uint32_t b = c.scales[kv][sat];
        w[kv][q] = in ? v : 0u;
        f[kv][q] = __uint_as_float(in ? b << 23 : 0u);  // (255, the exponent of NaN: NaN whatever the codes)
      }
    }
#pragma unroll
    for (int q = 0; q < kReadCells; ++q) {
      const uint32_t x = x0 + q * kWG;
      if (x >= total) break;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        char* dst = P.dst[kv] + ((int64_t)i0 * cells + x) * 8 * ES;
        if constexpr (ES == 2) {
          __builtin_nontemporal_store(
              u32x4{widen4<0>(w[kv][q], f[kv][q]), widen4<1>(w[kv][q], f[kv][q]), widen4<2>(w[kv][q], f[kv][q]),
                    widen4<3>(w[kv][q], f[kv][q])},
              reinterpret_cast<u32x4_any_out*>(dst));
        } else {
          const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[kv][q], f[kv][q], 0),
                      b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[kv][q], f[kv][q], 1),
                      d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[kv][q], f[kv][q], 2),
                      e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[kv][q], f[kv][q], 3);
          __builtin_nontemporal_store(f32x4{a.x, a.y, b.x, b.y}, reinterpret_cast<f32x4_any_out*>(dst));
          __builtin_nontemporal_store(f32x4{d.x, d.y, e.x, e.y}, reinterpret_cast<f32x4_any_out*>(dst + 16));
        }
      }
    }
  }
}

hipError_t launch_kv4_read(const KvReadParams& P, int dtype, hipStream_t stream) {
  const dim3 grid((unsigned)((P.N + P.per - 1) / P.per));
  if (dtype == SPEC_BF16)
    hipLaunchKernelGGL((kv4_read_kernel<2>), grid, dim3(kWG), 0, stream, P);
  else
    hipLaunchKernelGGL((kv4_read_kernel<4>), grid, dim3(kWG), 0, stream, P);
  return hipGetLastError();
}

}  // namespace specv
