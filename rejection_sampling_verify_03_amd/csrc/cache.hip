// cache.hip -- the 8-bit paged KV cache: keys and values quantised as they are
// written at the slots of a slot mapping, and read back, on gfx950.
//
// A group of scale_tokens tokens of one block and head shares the scale 2^e,
// e the smallest exponent with |x| <= 448 * 2^e over what the group holds.  All of a
// group's entries of a call stand together in the list, so the first of them
// leads: the wave that meets it gathers the group's entries, reduces their
// largest magnitude, settles the exponent with the one the group has, moves
// the earlier tokens' codes if it grew, and writes the new codes.  No
// global atomics, no second launch, and one owner for each group's bytes.
//
// Both are bound by memory.  Measured (MI355X): 32771 tokens of 8 heads of 128
// bf16 written in 36 us (143 MB read and written, 3.9 TB/s; a device copy
// reaches 4.7), 131072 tokens read back in 140 us (806 MB, 5.7 TB/s).  A write
// holds eight steps of a group in registers: four made it 20 % slower (groups
// of 32 tokens are then read twice), and heads that interleave keys and values
// over the waves cost a tenth (a wave's neighbours then read elsewhere).
#include <limits.h>

#include "cache_device.hpp"
#include "unaligned.hpp"

namespace specv {

__device__ __forceinline__ bool slot_in(const CacheView& c, int64_t s) {
  return s >= 0 && s < ((int64_t)c.num_blocks << c.bs_shift);
}

__device__ __forceinline__ int64_t lane_i64(int64_t x, int l) {
  return ((int64_t)lane_i((int)(x >> 32), l) << 32) | (uint32_t)lane_i((int)x, l);
}

// Past the first 64 entries beyond a chunk the list is read this many 64 at a
// time: a padded batch may end in many that are skipped (131072 of them behind
// one token: 250 us against 401 one at a time).
constexpr int kSkim = 8;

// The group (over the whole cache) of the last entry in front of entry i
// that lies in the cache, or -1; s holds the first 64 (lane l: entry
// i - 1 - l).
__device__ __forceinline__ int64_t group_before(const KvWriteParams& P, int i, int64_t s, int lane) {
  const uint64_t on = __ballot(slot_in(P.c, s));
  if (on) return lane_i64(s >> P.c.st_shift, __builtin_ctzll(on));
  for (int j0 = i - 65; j0 >= 0; j0 -= 64 * kSkim) {
    int64_t t[kSkim];
#pragma unroll
    for (int q = 0; q < kSkim; ++q) t[q] = j0 - 64 * q - lane >= 0 ? P.slots[j0 - 64 * q - lane] : -1;
#pragma unroll
    for (int q = 0; q < kSkim; ++q) {
      const uint64_t in = __ballot(slot_in(P.c, t[q]));
      if (in) return lane_i64(t[q] >> P.c.st_shift, __builtin_ctzll(in));
    }
  }
  return -1;
}

// One group of one head, keys or values: entries idx[0, cnt) of the source
// go to the offsets off[0, cnt) of the group.  dim / 8 lanes of 8 elements
// hold a token and 64 / (dim / 8) tokens are in a step; the loads of eight
// steps are on their way together, and up to eight steps stay in registers
// from the search for the maximum to the conversion (a longer group is read
// again, from L2).
constexpr int kWriteSteps = 8;
template <int ES>
__device__ __forceinline__ void write_group(const KvWriteParams& P, int kv, int h, int64_t gid, const int* idx,
                                            const int* off, int cnt, int first, int lane) {
  const CacheView& c = P.c;
  const int lpt = c.dim >> 3, tps = 64 / lpt;
  const int tl = lane / lpt, col = (lane - tl * lpt) * 8;
  const int64_t tok0 = gid << c.st_shift;
  const int64_t blk = tok0 >> c.bs_shift;
  const int in_blk = (int)(tok0 & ((1 << c.bs_shift) - 1));
  uint8_t* base = c.codes[kv] + blk * c.block + (int64_t)in_blk * c.token + (int64_t)h * c.head;
  uint8_t* sc = c.scales[kv] + blk * c.sblock + (int64_t)h * c.shead + (in_blk >> c.st_shift);
  const char* src = P.src[kv] + ((int64_t)h * P.hd[kv] + col) * ES;
  const int64_t ts = P.tok[kv];
  const int steps = (cnt + tps - 1) / tps;
  const int old = first > 0 ? (int)*sc - kScaleBias : 0;
  RawGroup<ES, true> rg[kWriteSteps];
  auto load_steps = [&](int s0) {  // a lane without a token takes the last one's elements
#pragma unroll
    for (int q = 0; q < kWriteSteps; ++q)
      if (s0 + q < steps) {
        const int t = min((s0 + q) * tps + min(tl, tps - 1), cnt - 1);
        rg[q] = load_any<ES>(src, (int64_t)idx[t] * ts);
      }
  };
  float amax = 0.f;
  for (int s0 = 0; s0 < steps; s0 += kWriteSteps) {
    load_steps(s0);
#pragma unroll
    for (int q = 0; q < kWriteSteps; ++q)
      if (s0 + q < steps) {
        float x[8];
        unpack_group<ES, true>(rg[q], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float a = fabsf(x[i]);
          amax = fmaxf(amax, a <= FLT_MAX ? a : 0.f);
        }
      }
  }
  int e = group_exponent(wave_max_f(amax));
  if (first > 0) {
    if (e > old) {
      // the tokens in front move to the larger scale; in front of a byte of 0
      // nothing was written, whatever codes stand there
      const bool none = old == -kScaleBias;
      const float f = two_to(max(old - e, -126));
      for (int t0 = 0; t0 < first; t0 += tps) {
        const int t = t0 + tl;
        if (tl < tps && t < first) {
          u32x2* p = reinterpret_cast<u32x2*>(base + (int64_t)t * c.token + col);
          u32x2 w = *p;
          float a[4], b[4];
          decode4(w.x, a);
          decode4(w.y, b);
          w.x = encode4(a[0] * f, a[1] * f, a[2] * f, a[3] * f);
          w.y = encode4(b[0] * f, b[1] * f, b[2] * f, b[3] * f);
          *p = none ? u32x2{0, 0} : w;
        }
      }
    } else {
      e = old;
    }
  }
  const float f = e < 127 ? two_to(-e) : 0x1p-127f;  // (127 only where the group had a byte of 254)
  for (int s0 = 0; s0 < steps; s0 += kWriteSteps) {
    if (steps > kWriteSteps) load_steps(s0);
#pragma unroll
    for (int q = 0; q < kWriteSteps; ++q) {
      const int t = (s0 + q) * tps + tl;
      if (tl < tps && t < cnt) {
        float x[8];
        unpack_group<ES, true>(rg[q], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = finite_or_nan(x[i]) * f;
        u32x2 w;
        w.x = encode4(x[0], x[1], x[2], x[3]);
        w.y = encode4(x[4], x[5], x[6], x[7]);
        *reinterpret_cast<u32x2*>(base + (int64_t)off[t] * c.token + col) = w;
      }
    }
  }
  if (lane == 0) *sc = (uint8_t)(e + kScaleBias);
}

// Grid: x the chunks of P.chunk (<= 64) entries, y the (head, keys or values)
// pairs, four to a workgroup: each wave owns one pair of its chunk and walks
// the groups that begin there.
template <int ES>
__global__ __launch_bounds__(kWG) void kv_write_kernel(KvWriteParams P) {
  __shared__ int s_at[kWaves][64], s_idx[kWaves][64], s_off[kWaves][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int pair = blockIdx.y * kWaves + wave;
  if (pair >= 2 * P.c.heads) return;
  const int kv = pair >= P.c.heads, h = pair - kv * P.c.heads;  // (neighbouring waves on neighbouring heads)
  int* at = s_at[wave];
  int* idx = s_idx[wave];
  int* off = s_off[wave];
  const int i0 = blockIdx.x * P.chunk;
  const int n = min(P.chunk, P.N - i0);
  const int64_t s = lane < n ? P.slots[i0 + lane] : -1;
  const int64_t s_before = i0 - 1 - lane >= 0 ? P.slots[i0 - 1 - lane] : -1;
  const bool in_s = slot_in(P.c, s);
  const uint64_t on = __ballot(in_s);
  if (on == 0) return;
  const int64_t g = s >> P.c.st_shift;
  int64_t prev = group_before(P, i0, s_before, lane);
  const int st = 1 << P.c.st_shift;
  for (uint64_t w = on; w; w &= w - 1) {
    const int L = __builtin_ctzll(w);
    const int64_t gid = lane_i64(g, L);
    if (gid == prev) continue;
    prev = gid;
    // the group's entries: at[offset] = the last entry with it.  Those of this
    // chunk are at hand; where no entry of another group ends them there, the
    // list is read on.
    at[lane] = -1;
    __builtin_amdgcn_wave_barrier();
    uint64_t other = __ballot(in_s && lane > L && g != gid);
    int end = other ? __builtin_ctzll(other) : 64;
    if (in_s && lane >= L && lane < end) atomicMax(&at[(int)s & (st - 1)], i0 + lane);
    auto take = [&](int64_t j, int64_t sj) {  // 64 more entries, lane l's: slots[j] = sj
      const bool in = slot_in(P.c, sj);
      other = __ballot(in && (sj >> P.c.st_shift) != gid);
      end = other ? __builtin_ctzll(other) : 64;
      if (in && lane < end) atomicMax(&at[(int)sj & (st - 1)], (int)j);
    };
    int64_t j = i0 + n + lane;
    if (!other && i0 + n < P.N) take(j, j < P.N ? P.slots[j] : -1);
    for (j += 64; !other && j - lane < P.N; j += 64 * kSkim) {
      int64_t sj[kSkim];
#pragma unroll
      for (int q = 0; q < kSkim; ++q) sj[q] = j + 64 * q < P.N ? P.slots[j + 64 * q] : -1;
#pragma unroll
      for (int q = 0; q < kSkim; ++q)
        if (!other) take(j + 64 * q, sj[q]);
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
    write_group<ES>(P, kv, h, gid, idx, off, __builtin_popcountll(used), __builtin_ctzll(used), lane);
    __builtin_amdgcn_wave_barrier();
  }
}

hipError_t launch_kv_write(const KvWriteParams& P, int dtype, hipStream_t stream) {
  const dim3 grid((unsigned)((P.N + P.chunk - 1) / P.chunk), (unsigned)((2 * P.c.heads + kWaves - 1) / kWaves));
  if (dtype == SPEC_BF16)
    hipLaunchKernelGGL((kv_write_kernel<2>), grid, dim3(kWG), 0, stream, P);
  else
    hipLaunchKernelGGL((kv_write_kernel<4>), grid, dim3(kWG), 0, stream, P);
  return hipGetLastError();
}

// One lane takes 8 elements of one (entry, head) row, keys and values, a cell;
// a workgroup takes P.per entries, and a lane has the loads of kReadCells
// cells on their way together.
template <int ES, bool VEC>
__global__ __launch_bounds__(kWG) void kv_read_kernel(KvReadParams P) {
  const CacheView& c = P.c;
  const uint32_t lpt = (uint32_t)c.dim >> 3, cells = (uint32_t)c.heads * lpt;  // of an entry, at most 2^15
  const int i0 = blockIdx.x * P.per;
  const uint32_t total = cells * (uint32_t)min(P.per, P.N - i0);
  for (uint32_t x0 = threadIdx.x; x0 < total; x0 += kWG * kReadCells) {
    u32x2 w[2][kReadCells];
    float f[2][kReadCells];
#pragma unroll
    for (int q = 0; q < kReadCells; ++q) {
      const uint32_t x = min(x0 + q * kWG, total - 1);  // (a lane past the end reads the last cell and stores nothing)
      const uint32_t e = x / cells, cell = x - e * cells;
      const uint32_t h = cell / lpt, col = (cell - h * lpt) * 8;
      const int64_t s = P.slots[i0 + e];
      const bool in = slot_in(c, s);
      const int64_t blk = in ? s >> c.bs_shift : 0;
      const int t = in ? (int)(s & ((1 << c.bs_shift) - 1)) : 0;
      const int64_t at = blk * c.block + (int64_t)t * c.token + (int64_t)h * c.head + col;
      const int64_t sat = blk * c.sblock + (int64_t)h * c.shead + (t >> c.st_shift);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(c.codes[kv] + at));
        const float sc = scale_of(c.scales[kv][sat]);
        const bool some = in && sc > 0.f;  // (0: never written, whatever the codes)
        w[kv][q] = some ? v : u32x2{0, 0};
        f[kv][q] = some ? sc : 0.f;
      }
    }
#pragma unroll
    for (int q = 0; q < kReadCells; ++q) {
      const uint32_t x = x0 + q * kWG;
      if (x >= total) break;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        float v[8];
        decode4(w[kv][q].x, v);
        decode4(w[kv][q].y, v + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= f[kv][q];
        char* dst = P.dst[kv] + ((int64_t)i0 * cells + x) * 8 * ES;
        if constexpr (ES == 2) {
          uint32_t o[4];  // exact in bf16: the upper halves
#pragma unroll
          for (int i = 0; i < 4; ++i)
            o[i] = (__float_as_uint(v[2 * i]) >> 16) | (__float_as_uint(v[2 * i + 1]) & 0xffff0000u);
          if constexpr (VEC) {
            __builtin_nontemporal_store(u32x4{o[0], o[1], o[2], o[3]}, reinterpret_cast<u32x4*>(dst));
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) reinterpret_cast<uint16_t*>(dst)[i] = (uint16_t)(o[i >> 1] >> (16 * (i & 1)));
          }
        } else {
          if constexpr (VEC) {
            __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, reinterpret_cast<f32x4*>(dst));
            __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, reinterpret_cast<f32x4*>(dst + 16));
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) reinterpret_cast<float*>(dst)[i] = v[i];
          }
        }
      }
    }
  }
}

hipError_t launch_kv_read(const KvReadParams& P, int dtype, bool vec, hipStream_t stream) {
  const dim3 grid((unsigned)((P.N + P.per - 1) / P.per));
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
