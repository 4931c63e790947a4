// cache.hip -- the 8-bit paged KV cache: keys and values quantised as they are
// written at the slots of a slot mapping, and read back, on gfx950.
//
// A group of scale_tokens tokens of one block and head shares the scale 2^e,
// e the smallest exponent with |x| <= 448 * 2^e over what the group holds.  All of a
// group's entries of a call stand together in the list, so the first of them
// leads: the wave that meets it gathers the group's entries, reduces their
// largest magnitude, settles the exponent with the one the group has, moves
// the earlier tokens' codes if it grew, and writes the new codes.  No
// atomics, no second launch, and one owner for each group's bytes.
#include <limits.h>

#include "cache_device.hpp"

namespace specv {

__device__ __forceinline__ bool slot_in(const CacheView& c, int64_t s) {
  return s >= 0 && s < ((int64_t)c.num_blocks << c.bs_shift);
}

// The group (over the whole cache) of the last entry in front of entry i
// that lies in the cache, or -1; 64 entries a step.
__device__ __forceinline__ int64_t group_before(const KvWriteParams& P, int i, int lane) {
  for (int i0 = i; i0 > 0; i0 -= 64) {
    const int j = i0 - 1 - lane;
    const int64_t s = j >= 0 ? P.slots[j] : -1;
    const uint64_t on = __ballot(slot_in(P.c, s));
    if (on) {
      const int L = __builtin_ctzll(on);
      const int64_t g = s >> P.c.st_shift;
      return ((int64_t)lane_i((int)(g >> 32), L) << 32) | (uint32_t)lane_i((int)g, L);
    }
  }
  return -1;
}

// 8 elements of a source row widened to fp32.
template <int ES, bool VEC>
__device__ __forceinline__ void load8(const char* p, float x[8]) {
  load_group<ES, VEC>(p, 0, x);
}

// One group of one head, keys or values: entries idx[0, cnt) of the source
// go to the offsets off[0, cnt) of the group.  LPT lanes of 8 elements hold a
// token; 64 / LPT tokens are in a step.
template <int ES, bool VEC>
__device__ __forceinline__ void write_group(const KvWriteParams& P, int kv, int h, int64_t gid, const int* idx,
                                            const int* off, int cnt, int first, int lane) {
  const CacheView& c = P.c;
  const int lpt = c.dim >> 3, tps = 64 / lpt;
  const int tl = lane / lpt, col = (lane - tl * lpt) * 8;
  const bool on = tl < tps;
  const int64_t tok0 = gid << c.st_shift;
  const int64_t blk = tok0 >> c.bs_shift;
  const int in_blk = (int)(tok0 & ((1 << c.bs_shift) - 1));
  uint8_t* base = c.codes[kv] + blk * c.block + (int64_t)in_blk * c.token + (int64_t)h * c.head;
  uint8_t* sc = c.scales[kv] + blk * c.sblock + (int64_t)h * c.shead + (in_blk >> c.st_shift);
  const char* src = P.src[kv] + (int64_t)h * P.hd[kv] * ES;
  const int64_t ts = P.tok[kv];
  float amax = 0.f;
  for (int t0 = 0; t0 < cnt; t0 += tps) {
    const int t = t0 + tl;
    if (on && t < cnt) {
      float x[8];
      load8<ES, VEC>(src + ((int64_t)idx[t] * ts + col) * ES, x);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float a = fabsf(x[q]);
        amax = fmaxf(amax, a <= FLT_MAX ? a : 0.f);
      }
    }
  }
  int e = group_exponent(wave_max_f(amax));
  if (first > 0) {
    const int old = (int)*sc - kScaleBias;
    if (e > old) {
      // the tokens in front move to the larger scale
      const float f = two_to(max(old - e, -126));
      for (int t0 = 0; t0 < first; t0 += tps) {
        const int t = t0 + tl;
        if (on && t < first) {
          u32x2* p = reinterpret_cast<u32x2*>(base + (int64_t)t * c.token + col);
          u32x2 w = *p;
          float a[4], b[4];
          decode4(w.x, a);
          decode4(w.y, b);
          w.x = encode4(a[0] * f, a[1] * f, a[2] * f, a[3] * f);
          w.y = encode4(b[0] * f, b[1] * f, b[2] * f, b[3] * f);
          *p = w;
        }
      }
    } else {
      e = old;
    }
  }
  const float f = two_to(-e);
  for (int t0 = 0; t0 < cnt; t0 += tps) {
    const int t = t0 + tl;
    if (on && t < cnt) {
      float x[8];
      load8<ES, VEC>(src + ((int64_t)idx[t] * ts + col) * ES, x);
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] = finite_or_nan(x[q]) * f;
      u32x2 w;
      w.x = encode4(x[0], x[1], x[2], x[3]);
      w.y = encode4(x[4], x[5], x[6], x[7]);
      *reinterpret_cast<u32x2*>(base + (int64_t)off[t] * c.token + col) = w;
    }
  }
  if (lane == 0) *sc = (uint8_t)(e + kScaleBias);
}

// Grid: x the chunks of P.chunk (<= 64) entries, y the (head, keys or values)
// pairs, four to a workgroup: each wave owns one pair of its chunk and walks
// the groups that begin there.
template <int ES, bool VEC>
__global__ __launch_bounds__(kWG) void kv_write_kernel(KvWriteParams P) {
  __shared__ int s_at[kWaves][64], s_idx[kWaves][64], s_off[kWaves][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int pair = blockIdx.y * kWaves + wave;
  if (pair >= 2 * P.c.heads) return;
  const int kv = pair & 1, h = pair >> 1;
  int* at = s_at[wave];
  int* idx = s_idx[wave];
  int* off = s_off[wave];
  const int i0 = blockIdx.x * P.chunk;
  const int n = min(P.chunk, P.N - i0);
  const int64_t s = lane < n ? P.slots[i0 + lane] : -1;
  const uint64_t on = __ballot(slot_in(P.c, s));
  if (on == 0) return;
  const int64_t g = s >> P.c.st_shift;
  const int g_lo = (int)g, g_hi = (int)(g >> 32);
  int64_t prev = group_before(P, i0, lane);
  const int st = 1 << P.c.st_shift;
  for (uint64_t w = on; w; w &= w - 1) {
    const int L = __builtin_ctzll(w);
    const int64_t gid = ((int64_t)lane_i(g_hi, L) << 32) | (uint32_t)lane_i(g_lo, L);
    if (gid == prev) continue;
    prev = gid;
    // the group's entries: at[offset] = the last entry with it
    at[lane] = -1;
    __builtin_amdgcn_wave_barrier();
    for (int j0 = i0 + L; j0 < P.N; j0 += 64) {
      const int j = j0 + lane;
      const int64_t sj = j < P.N ? P.slots[j] : -1;
      const bool in = slot_in(P.c, sj);
      const uint64_t other = __ballot(in && (sj >> P.c.st_shift) != gid);
      const int end = other ? __builtin_ctzll(other) : 64;
      if (in && lane < end) atomicMax(&at[(int)sj & (st - 1)], j);
      if (other) break;
    }
    __builtin_amdgcn_wave_barrier();
    const int mine = at[lane];
    const uint64_t used = __ballot(lane < st && mine >= 0);
    const int place = __builtin_popcountll(used & (lane ? (~0ull >> (64 - lane)) : 0ull));
    if (lane < st && mine >= 0) {
      idx[place] = mine;
      off[place] = lane;
    }
    __builtin_amdgcn_wave_barrier();
    write_group<ES, VEC>(P, kv, h, gid, idx, off, __builtin_popcountll(used), __builtin_ctzll(used), lane);
    __builtin_amdgcn_wave_barrier();
  }
}

hipError_t launch_kv_write(const KvWriteParams& P, int dtype, bool vec, hipStream_t stream) {
  const dim3 grid((unsigned)((P.N + P.chunk - 1) / P.chunk), (unsigned)((2 * P.c.heads + kWaves - 1) / kWaves));
  if (dtype == SPEC_BF16) {
    if (vec)
      hipLaunchKernelGGL((kv_write_kernel<2, true>), grid, dim3(kWG), 0, stream, P);
    else
      hipLaunchKernelGGL((kv_write_kernel<2, false>), grid, dim3(kWG), 0, stream, P);
  } else {
    if (vec)
      hipLaunchKernelGGL((kv_write_kernel<4, true>), grid, dim3(kWG), 0, stream, P);
    else
      hipLaunchKernelGGL((kv_write_kernel<4, false>), grid, dim3(kWG), 0, stream, P);
  }
  return hipGetLastError();
}

// One lane takes 8 elements of one (entry, head) row, keys and values.
template <int ES, bool VEC>
__global__ __launch_bounds__(kWG) void kv_read_kernel(KvReadParams P) {
  const CacheView& c = P.c;
  const int lpt = c.dim >> 3;
  const int cells = c.heads * lpt;  // per entry, at most 2^15
  const int64_t total = (int64_t)P.N * cells;
  for (int64_t x = (int64_t)blockIdx.x * kWG + threadIdx.x; x < total; x += (int64_t)gridDim.x * kWG) {
    const int i = (int)(x / cells), cell = (int)(x - (int64_t)i * cells);
    const int h = cell / lpt, col = (cell - h * lpt) * 8;
    const int64_t s = P.slots[i];
    const bool in = slot_in(c, s);
    const int64_t blk = s >> c.bs_shift;
    const int t = (int)(s & ((1 << c.bs_shift) - 1));
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      float v[8];
      if (in) {
        const u32x2 w = *reinterpret_cast<const u32x2*>(c.codes[kv] + blk * c.block + (int64_t)t * c.token +
                                                        (int64_t)h * c.head + col);
        const float f = scale_of(c.scales[kv][blk * c.sblock + (int64_t)h * c.shead + (t >> c.st_shift)]);
        decode4(w.x, v);
        decode4(w.y, v + 4);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] *= f;
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = 0.f;
      }
      char* dst = P.dst[kv] + x * 8 * ES;
      if constexpr (ES == 2) {
        uint32_t w[4];  // exact in bf16: the upper halves
#pragma unroll
        for (int q = 0; q < 4; ++q)
          w[q] = (__float_as_uint(v[2 * q]) >> 16) | (__float_as_uint(v[2 * q + 1]) & 0xffff0000u);
        if constexpr (VEC) {
          __builtin_nontemporal_store(u32x4{w[0], w[1], w[2], w[3]}, reinterpret_cast<u32x4*>(dst));
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q) reinterpret_cast<uint16_t*>(dst)[q] = (uint16_t)(w[q >> 1] >> (16 * (q & 1)));
        }
      } else {
        if constexpr (VEC) {
          __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, reinterpret_cast<f32x4*>(dst));
          __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, reinterpret_cast<f32x4*>(dst + 16));
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q) reinterpret_cast<float*>(dst)[q] = v[q];
        }
      }
    }
  }
}

hipError_t launch_kv_read(const KvReadParams& P, int dtype, bool vec, hipStream_t stream) {
  const int64_t total = (int64_t)P.N * P.c.heads * (P.c.dim >> 3);
  const int64_t wgs = (total + kWG - 1) / kWG;
  const dim3 grid((unsigned)(wgs < 16384 ? wgs : 16384));
  if (dtype == SPEC_BF16) {
    if (vec)
      hipLaunchKernelGGL((kv_read_kernel<2, true>), grid, dim3(kWG), 0, stream, P);
    else
      hipLaunchKernelGGL((kv_read_kernel<2, false>), grid, dim3(kWG), 0, stream, P);
  } else {
    if (vec)
      hipLaunchKernelGGL((kv_read_kernel<4, true>), grid, dim3(kWG), 0, stream, P);
    else
      hipLaunchKernelGGL((kv_read_kernel<4, false>), grid, dim3(kWG), 0, stream, P);
  }
  return hipGetLastError();
}

}  // namespace specv
