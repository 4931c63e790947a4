// cache4.hip -- rotary positions, and the 4-bit paged KV cache: queries and keys
// rotated, keys and values quantised as they are written at the slots of a
// slot mapping, and read back, on gfx950.
//
// Rotation: pair i of a head, (x, y), at position p becomes
//   (x cos a - y sin a, y cos a + x sin a) * scale,  a = p * inv_freq[i],
// pairs (i, i + rot / 2), or (2 i, 2 i + 1) interleaved.  The angle, its cosine
// and sine and the products are taken in fp64 and rounded once: an angle of a
// far position has no correct fraction in fp32, and the codes of the cache are
// then those of the exact values (an fp32 product next to the border of two
// codes picks the wrong one about once in a million).  The cosines and sines
// are worked out once for all heads of a token; what is left is eight fp64
// instructions for 16 bytes, below memory's rate.
//
// Cache: 32 consecutive elements of a token's head share the scale 2^e, e the
// smallest exponent with |x| <= 6 * 2^e, and are held as e2m1 codes (0, 0.5, 1,
// 1.5, 2, 3, 4, 6 and a sign), the microscaled format that the widening
// instructions read.  A scale belongs to one token, so every token is written
// by itself: no order among the writers, nothing read back.
//
// One lane takes 8 elements of one head of a token; four lanes hold the 32
// elements of a scale.
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
// y itself would (inexact: to the neighbour whose last bit is 1).
__device__ __forceinline__ float to_odd(double y) {
  const float f = (float)y;
  const double d = y - (double)f;
  uint32_t u = __float_as_uint(f);
  if ((d > 0.0 || d < 0.0) && !(u & 1u)) u += (d > 0.0) == (y > 0.0) ? 1u : ~0u;
  return __uint_as_float(u);
}

// The largest of the four lanes of a quad, in each of them.
__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __int_as_float(dpp_i<0xb1, 0xf>(__float_as_int(x), 0)));
  return fmaxf(x, __int_as_float(dpp_i<0x4e, 0xf>(__float_as_int(x), 0)));
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

template <int ES>
__device__ __forceinline__ void store8(char* dst, const float x[8]) {
  if constexpr (ES == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = round_bf16x2(x[2 * i], x[2 * i + 1]);
    *reinterpret_cast<u32x4_any_out*>(dst) = u32x4{w[0], w[1], w[2], w[3]};
  } else {
    *reinterpret_cast<f32x4_any_out*>(dst) = f32x4{x[0], x[1], x[2], x[3]};
    *reinterpret_cast<f32x4_any_out*>(dst + 16) = f32x4{x[4], x[5], x[6], x[7]};
  }
}

// Grid: x sets of P.tokens tokens, y shares of a token's heads.  A round takes
// as many heads as the workgroup holds.  In place, with pairs half a head
// apart, two lanes write what both read: all of a round's reads are done
// before its writes (heads are never shared between workgroups).
template <int ES, bool WRITE, bool INTER>
__global__ __launch_bounds__(kWG) void rope_kernel(RopeParams P) {
  // cosine and sine of pair 8 j + q (interleaved: 4 j + q) of a token at
  // [token][q][j]: the lanes of a head read neighbouring places
  __shared__ double2 s_turn[kRopeAngles];
  const int tid = threadIdx.x;
  const int half = P.half, step = INTER ? 4 : 8, rows = half / step;
  const int n0 = blockIdx.x * P.tokens;
  const int tokens = min(P.tokens, P.N - n0);
  for (int i = tid; i < tokens * half; i += kWG) {
    const int t = i / half, f = i - t * half;
    double sn, cs;
    const double at = P.wide ? (double)static_cast<const int64_t*>(P.positions)[n0 + t]
                             : (double)static_cast<const int32_t*>(P.positions)[n0 + t];
    sin_cos(at * P.inv_freq[f], sn, cs);
    s_turn[t * half + (f % step) * rows + f / step] = double2{cs * P.scale, sn * P.scale};
  }
  __syncthreads();
  const int lanes = P.dim >> 3, per = kWG / lanes;
  const int heads = P.heads[0] + (WRITE ? 2 : 1) * P.heads[1];
  const int mine = tid / lanes, col = (tid - mine * lanes) * 8;
  const int rounds = (heads + per - 1) / per;
  for (int t = 0; t < tokens; ++t) {
    const int n = n0 + t;
    int64_t slot = -1;
    if constexpr (WRITE) {
      slot = P.slots[n];
      // of equal slots next to each other the last counts
      if (slot >= (int64_t)P.c.num_blocks << P.c.bs_shift || (n + 1 < P.N && P.slots[n + 1] == slot)) slot = -1;
    }
    for (int r = blockIdx.y; r < rounds; r += gridDim.y) {
      int h = r * per + mine;
      const bool on = mine < per && h < heads;
      const int what = !on ? 0 : h < P.heads[0] ? 0 : h < P.heads[0] + P.heads[1] ? 1 : 2;  // queries, keys, values
      h -= what == 0 ? 0 : what == 1 ? P.heads[0] : P.heads[0] + P.heads[1];
      const bool turn = on && what < 2 && col < 2 * half;
      RawGroup<ES, true> own = neg_inf_group<ES, true>(), other = own;
      if (on) {
        const char* src = P.src[what] + ((int64_t)n * P.tok[what] + (int64_t)h * P.hd[what]) * ES;
        own = load_any<ES>(src, col);
        if (!INTER && turn) other = load_any<ES>(src, col < half ? col + half : col - half);
      }
      if constexpr (!INTER) {
        // (here, so that what was loaded has arrived)
        opaque_group<ES, true>(own);
        opaque_group<ES, true>(other);
        __syncthreads();
      }
      if (!on) continue;
      float x[8];
      unpack_group<ES, true>(own, x);
      if (turn) {
        double y[8];
        const double2* cs = s_turn + t * half;
        if constexpr (INTER) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const double2 w = cs[q * rows + (col >> 3)];
            const double a = x[2 * q], b = x[2 * q + 1];
            y[2 * q] = __builtin_fma(a, w.x, -(b * w.y));
            y[2 * q + 1] = __builtin_fma(a, w.y, b * w.x);
          }
        } else {
          float z[8];
          unpack_group<ES, true>(other, z);
          const bool first = col < half;
          const int j = (first ? col : col - half) >> 3;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const double2 w = cs[q * rows + j];
            const double b = (double)z[q] * w.y;
            y[q] = __builtin_fma((double)x[q], w.x, first ? -b : b);
          }
        }
        if (WRITE && what == 1) {
#pragma unroll
          for (int q = 0; q < 8; ++q) x[q] = to_odd(y[q]);
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q) x[q] = (float)y[q];
        }
      }
      if (!WRITE || what == 0) {
        store8<ES>(P.dst[what] + ((int64_t)n * P.dtok[what] + (int64_t)h * P.dhd[what] + col) * ES, x);
        continue;
      }
      if constexpr (WRITE) {
        // (the four lanes of a scale are together in all of this)
        if (slot < 0) continue;
        float amax = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float a = fabsf(x[q]);
          amax = fmaxf(amax, a <= FLT_MAX ? a : INFINITY);
        }
        amax = quad_max(amax);
        const bool fine = amax <= FLT_MAX;
        const int e = fine ? exponent4(amax) : 0;
        const int64_t blk = slot >> P.c.bs_shift;
        const int in = (int)(slot & ((1 << P.c.bs_shift) - 1));
        const uint32_t w = encode8(x, two_to(e));
        *reinterpret_cast<uint32_t*>(P.c.codes[what - 1] + blk * P.c.block + (int64_t)in * P.c.token +
                                     (int64_t)h * P.c.head + (col >> 1)) = fine ? w : 0u;
        if ((tid & 3) == 0)
          P.c.scales[what - 1][blk * P.c.sblock + (int64_t)h * P.c.shead + ((col >> 5) << P.c.bs_shift) + in] =
              (uint8_t)(fine ? e + kScaleBias : 255);
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
// cells on their way together.
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
          *reinterpret_cast<u32x4_any_out*>(dst) =
              u32x4{widen4<0>(w[kv][q], f[kv][q]), widen4<1>(w[kv][q], f[kv][q]), widen4<2>(w[kv][q], f[kv][q]),
                    widen4<3>(w[kv][q], f[kv][q])};
        } else {
          const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[kv][q], f[kv][q], 0),
                      b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[kv][q], f[kv][q], 1),
                      d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[kv][q], f[kv][q], 2),
                      e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[kv][q], f[kv][q], 3);
          *reinterpret_cast<f32x4_any_out*>(dst) = f32x4{a.x, a.y, b.x, b.y};
          *reinterpret_cast<f32x4_any_out*>(dst + 16) = f32x4{d.x, d.y, e.x, e.y};
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
