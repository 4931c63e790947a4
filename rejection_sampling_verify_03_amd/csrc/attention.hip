// attention.hip -- attention of each request's new tokens over its 8-bit paged
// context, on gfx950.
//
// For a row (new token i of request b, query head h of KV head kh) over the
// positions j that it sees:  s_j = scale * q . k_j,
//   out = sum_j exp(s_j) v_j / (sum_j exp(s_j) + exp(sink_h)),
// in one pass over the keys with a running reference in place of the maximum.
//
// The rows of one KV head, token-major (row m = token m / G, head m % G), are
// cut into blocks of 16 * RT; one 256-thread workgroup takes a block and a
// range of keys, each of its four waves every fourth tile of 32 keys, on its
// own: keys and values go from memory to the matrix units through registers
// alone, no barrier stands in the loop, and the waves' sums are joined once
// at the end.  Splits of the key range are joined by a second kernel.
//
// Both products run on v_mfma_f32_16x16x32_bf16 in the transposed order:
//   S^T (keys x rows) = K Q^T,   O^T (dims x rows) += V^T P^T,
// because lane l then holds row l % 16 of S^T for keys 4 (l / 16) + r, and
// with the 32 keys of a tile numbered
//   slot 8 g + j  =  key 4 g + j (j < 4),  key 16 + 4 g + j - 4 (j >= 4)
// that is where the second product wants P^T: the weights never leave their
// lanes.  The order of the sum over dims is free too: lane group g takes
// dims [g DP/4, (g+1) DP/4) of the keys, so a key is read in whole 16-byte
// loads.  The codes widen to bf16 exactly, scale included (one instruction
// for two); the values' bytes, which lie along dims, are first transposed
// four by four in registers.
//
// Weights are 2^(s_j log2(e) - ref) with a reference per row that moves only
// when a score passes it by 2^8: up to there the fp32 sums and the bf16
// weights lose nothing, and the sums are rarely rescaled.  The weights are
// rounded to bf16 for the second product (a relative error of at most 2^-8
// each, of no common sign, as the output's own rounding); their sum is kept
// in fp32 from the unrounded weights, so lse keeps fp32's accuracy.
#include <limits.h>

#include "cache_device.hpp"

namespace specv {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kTileKeys = 32;
constexpr float kNoRef = -FLT_MAX;   // the reference of a row that has seen nothing
constexpr float kRefSlack = 8.0f;   // how far (log2) a score may pass the reference

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// x with lanes l and l ^ 16 (l ^ 32) exchanged.
__device__ __forceinline__ float lane_xor16(float x) {
  return __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(x), 0x401f));
}
__device__ __forceinline__ float lane_xor32(float x) {
  const int i = __builtin_amdgcn_ds_bpermute(((int)(threadIdx.x & 63) ^ 32) << 2, __float_as_int(x));
  return __int_as_float(i);
}

// The keys that a block of rows sees, [kbeg, kend) with kbeg brought down to
// a whole tile, and the positions of its first and last token.
struct KeyRange {
  int lo, hi;      // tile-aligned first key, end
  int p_lo, p_hi;  // positions of the block's first and last token
  bool bad;        // the request's data cannot be used
};
__device__ __forceinline__ KeyRange key_range(const AttnParams& P, int n, int ctx, int tok_lo, int tok_hi) {
  KeyRange r;
  const int64_t cap = min((int64_t)P.max_ctx, (int64_t)P.max_blocks << P.c.bs_shift);
  r.bad = ctx < 0 || ctx > cap || n > P.max_q;
  r.p_lo = ctx - n + tok_lo;
  r.p_hi = ctx - n + tok_hi;
  const int beg = P.window > 0 ? max(0, r.p_lo - P.window + 1) : 0;
  r.lo = beg & ~(kTileKeys - 1);
  r.hi = max(r.p_hi + 1, r.lo);
  return r;
}

template <int DP>
struct TileRegs {
  u32x4 k[2][DP / 64];      // subtile u: key l % 16, dims [g DP/4, (g+1) DP/4)
  uint32_t v[8][DP / 64];   // slot j's key, dims [c DP/16, (c+1) DP/16), c = l % 16
  uint32_t ks[2];           // scale bytes of the keys' groups
  uint32_t vs[8];           // scale bytes of the values' groups (two used if !FINE)
  uint32_t ok;              // bit u: subtile u's block exists
};

// FINE: scale_tokens < 4, so that the four keys of a lane differ in scale.
template <int DP, bool FINE>
__device__ __forceinline__ void load_tile(const AttnParams& P, const int32_t* bt, int key0, int head, int lane,
                                          TileRegs<DP>& t) {
  const CacheView& c = P.c;
  const int r = lane & 15, g = lane >> 4;
  const int in_mask = (1 << c.bs_shift) - 1;
  t.ok = 0;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int k0 = key0 + 16 * u;
    const int lb = k0 >> c.bs_shift;
    int phys = lb < P.max_blocks ? bt[lb] : -1;
    if (phys >= 0 && phys < c.num_blocks)
      t.ok |= 1u << u;
    else
      phys = 0;
    const int in = k0 & in_mask;
    const uint8_t* kb = c.codes[0] + (int64_t)phys * c.block + (int64_t)head * c.head + (int64_t)in * c.token;
    const uint8_t* vb = c.codes[1] + (int64_t)phys * c.block + (int64_t)head * c.head + (int64_t)in * c.token;
    const int64_t so = (int64_t)phys * c.sblock + (int64_t)head * c.shead;
    const uint8_t* ksb = c.scales[0] + so;
    const uint8_t* vsb = c.scales[1] + so;
    t.ks[u] = ksb[(in + r) >> c.st_shift];
#pragma unroll
    for (int w = 0; w < DP / 64; ++w) {
      const int d = g * (DP / 4) + w * 16;
      t.k[u][w] = d < c.dim ? *reinterpret_cast<const u32x4*>(kb + (int64_t)r * c.token + d) : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int key = 4 * g + j;
      const uint8_t* p = vb + (int64_t)key * c.token;
      const int d = r * (DP / 16);
      if constexpr (DP == 64) {
        t.v[4 * u + j][0] = d < c.dim ? *reinterpret_cast<const uint32_t*>(p + d) : 0u;
      } else if constexpr (DP == 128) {
        const u32x2 w = d < c.dim ? *reinterpret_cast<const u32x2*>(p + d) : u32x2{0, 0};
        t.v[4 * u + j][0] = w.x;
        t.v[4 * u + j][1] = w.y;
      } else {
        const u32x4 w = d < c.dim ? *reinterpret_cast<const u32x4*>(p + d) : u32x4{0, 0, 0, 0};
        t.v[4 * u + j][0] = w.x;
        t.v[4 * u + j][1] = w.y;
        t.v[4 * u + j][2] = w.z;
        t.v[4 * u + j][3] = w.w;
      }
      if constexpr (FINE) t.vs[4 * u + j] = vsb[(in + key) >> c.st_shift];
    }
    if constexpr (!FINE) t.vs[u] = vsb[(in + 4 * g) >> c.st_shift];
  }
}

__device__ __forceinline__ bf16x8 pack8(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(bf16x8, u32x4{a, b, c, d});
}
template <bool HI>
__device__ __forceinline__ uint32_t widen2(uint32_t codes, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, HI));
}

// 4 x 4 bytes transposed: out[b] = byte b of a, b, c, d.
__device__ __forceinline__ void transpose4(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t out[4]) {
  const uint32_t ab0 = __builtin_amdgcn_perm(b, a, 0x05010400u), ab1 = __builtin_amdgcn_perm(b, a, 0x07030602u);
  const uint32_t cd0 = __builtin_amdgcn_perm(d, c, 0x05010400u), cd1 = __builtin_amdgcn_perm(d, c, 0x07030602u);
  out[0] = __builtin_amdgcn_perm(cd0, ab0, 0x05040100u);
  out[1] = __builtin_amdgcn_perm(cd0, ab0, 0x07060302u);
  out[2] = __builtin_amdgcn_perm(cd1, ab1, 0x05040100u);
  out[3] = __builtin_amdgcn_perm(cd1, ab1, 0x07060302u);
}

// Bit 7 of each byte that is an e4m3 NaN (0x7f or 0xff).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// Where a block's rows stop being computed here and go to memory.
template <int DP, int RT, bool FINE>
__global__ __launch_bounds__(kWG) void attn_kernel(AttnParams P) {
  constexpr int C = DP / 32;   // steps of the sum over dims
  constexpr int DT = DP / 16;  // 16-dim tiles of the output
  __shared__ __align__(16) char s_mem[(RT * C * 64 * 16 > kWaves * 16 * DP * 4) ? RT * C * 64 * 16
                                                                                : kWaves * 16 * DP * 4];
  __shared__ float s_ref[kWaves][RT * 16], s_sum[kWaves][RT * 16];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  int x = blockIdx.x;
  const int rb = x % P.nrb;
  x /= P.nrb;
  const int sp = x % P.nsplit;
  x /= P.nsplit;
  const int head = x % P.c.heads, b = x / P.c.heads;

  const int q0 = P.q_start[b], q1 = P.q_start[b + 1];
  if (q0 < 0 || q1 > P.N || q1 <= q0) return;
  const int n = q1 - q0, G = P.G;
  const int ctx = P.ctx_len[b];
  const int64_t rows = (int64_t)n * G;
  const int64_t m0 = (int64_t)rb * (RT * 16);
  // a request that cannot be used: NaN in all its rows (those of a request
  // with more than max_q tokens among them)
  {
    const KeyRange all = key_range(P, n, ctx, 0, n - 1);
    if (all.bad) {
      if (sp != 0) return;
      for (int64_t m = (int64_t)rb * kWG + tid; m < rows; m += (int64_t)P.nrb * kWG) {
        const int64_t row = (int64_t)(q0 + m / G) * P.Hq + head * G + m % G;
        for (int d = 0; d < P.c.dim; ++d) P.out[row * P.c.dim + d] = 0x7fc0;
        if (P.lse) P.lse[row] = __builtin_nanf("");
      }
      return;
    }
  }
  if (m0 >= rows) return;
  const int64_t m1 = min(rows, m0 + RT * 16);
  const KeyRange kr = key_range(P, n, ctx, (int)(m0 / G), (int)((m1 - 1) / G));
  const int64_t kb64 = (int64_t)kr.lo + (int64_t)sp * P.split_keys;
  if (sp > 0 && kb64 >= kr.hi) return;  // (the first split of an empty range still writes its zeros)
  const int k_beg = (int)kb64, k_end = (int)min((int64_t)kr.hi, kb64 + P.split_keys);

  // Q to LDS as the fragments of the first product: fragment (rt, c), lane l:
  // row 16 rt + l % 16, dims (l / 16) DP/4 + 8 c ..+ 8
  {
    u32x4* qf = reinterpret_cast<u32x4*>(s_mem);
    for (int f = tid; f < RT * C * 64; f += kWG) {
      const int l = f & 63, c = (f >> 6) % C, rt = (f >> 6) / C;
      const int64_t m = m0 + rt * 16 + (l & 15);
      const int d = (l >> 4) * (DP / 4) + 8 * c;
      u32x4 v{0, 0, 0, 0};
      if (m < m1 && d < P.c.dim) {
        const uint16_t* src = reinterpret_cast<const uint16_t*>(P.q) + (int64_t)(q0 + m / G) * P.q_tok +
                              (int64_t)(head * G + m % G) * P.q_head + d;
        if (P.qvec) {
          v = *reinterpret_cast<const u32x4*>(src);
        } else {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = (uint32_t)src[2 * i] | ((uint32_t)src[2 * i + 1] << 16);
          v = u32x4{w[0], w[1], w[2], w[3]};
        }
      }
      qf[f] = v;
    }
  }
  __syncthreads();

  int pos[RT];  // the position of this lane's row, -1 for rows past the block
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int64_t m = m0 + rt * 16 + r;
    pos[rt] = m < m1 ? ctx - n + (int)(m / G) : -1;
  }
  f32x4 acc[RT][DT];
  float ref[RT], sum[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    ref[rt] = kNoRef;
    sum[rt] = 0.f;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) acc[rt][dt] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  const int32_t* bt = P.bt + (int64_t)b * P.bt_stride;
  const u32x4* qf = reinterpret_cast<const u32x4*>(s_mem);
  TileRegs<DP> nx;
  int key0 = k_beg + wave * kTileKeys;
  if (key0 < k_end) load_tile<DP, FINE>(P, bt, key0, head, lane, nx);
  for (; key0 < k_end; key0 += kWaves * kTileKeys) {
    TileRegs<DP> t = nx;
    if (key0 + kWaves * kTileKeys < k_end) load_tile<DP, FINE>(P, bt, key0 + kWaves * kTileKeys, head, lane, nx);
    // every row of the block sees every key of the tile
    const bool whole = t.ok == 3u && key0 + kTileKeys - 1 <= kr.p_lo && (P.window == 0 || key0 > kr.p_hi - P.window);

    // S^T
    f32x4 s[RT][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float ksc = scale_of(t.ks[u]);
      bf16x8 ka[C];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const u32x4 w4 = t.k[u][c / 2];
        const uint32_t w0 = (c & 1) ? w4.z : w4.x, w1 = (c & 1) ? w4.w : w4.y;
        ka[c] = pack8(widen2<false>(w0, ksc), widen2<true>(w0, ksc), widen2<false>(w1, ksc), widen2<true>(w1, ksc));
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        f32x4 a{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < C; ++c)
          a = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ka[c], __builtin_bit_cast(bf16x8, qf[(rt * C + c) * 64 + lane]), a,
                                                      0, 0, 0);
        s[rt][u] = a;
      }
    }

    // a tile that some row sees only in part: nothing of the keys that no row
    // sees may enter (0 * NaN, 0 * inf), and a NaN among the others is kept
    // apart
    bool nans = false;
    if (!whole) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        bool some = false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int key = key0 + 16 * u + 4 * g + j;
          const bool any = ((t.ok >> u) & 1u) && key <= kr.p_hi && (P.window == 0 || key > kr.p_lo - P.window);
          some |= any;
#pragma unroll
          for (int w = 0; w < DP / 64; ++w) {
            t.v[4 * u + j][w] = any ? t.v[4 * u + j][w] : 0u;
            nans |= nan_bytes(t.v[4 * u + j][w]) != 0;
          }
          if constexpr (FINE) t.vs[4 * u + j] = any ? t.vs[4 * u + j] : (uint32_t)kScaleBias;
        }
        if constexpr (!FINE) t.vs[u] = some ? t.vs[u] : (uint32_t)kScaleBias;
      }
      nans = __ballot(nans) != 0;
    }

    // scores in units of log2, those not seen at -inf; the reference follows
    bf16x8 pb[RT];
    bool move = false;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      float mx = -INFINITY;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float v = s[rt][u][j] * P.scale2;
          if (!whole) {
            const int key = key0 + 16 * u + 4 * g + j;
            const bool see = ((t.ok >> u) & 1u) && key <= pos[rt] && (P.window == 0 || key > pos[rt] - P.window);
            v = see ? v : -INFINITY;
          }
          s[rt][u][j] = v;
          mx = fmaxf(mx, v);
        }
      move |= mx > ref[rt] + kRefSlack;
    }
    if (__ballot(move)) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        float mx = ref[rt];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int j = 0; j < 4; ++j) mx = fmaxf(mx, s[rt][u][j]);
        mx = fmaxf(mx, lane_xor16(mx));
        mx = fmaxf(mx, lane_xor32(mx));
        const float f = exp2_fast(ref[rt] - mx);
        ref[rt] = mx;
        sum[rt] *= f;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) acc[rt][dt] *= f;
      }
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      float p[8];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) p[4 * u + j] = exp2_fast(s[rt][u][j] - ref[rt]);
      sum[rt] += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
      if constexpr (FINE) {
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] *= scale_of(t.vs[j]);
      }
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{p[2 * j], p[2 * j + 1]}, bf16x2));
      pb[rt] = pack8(w[0], w[1], w[2], w[3]);
    }

    const float vsc0 = FINE ? 1.0f : scale_of(t.vs[0]), vsc1 = FINE ? 1.0f : scale_of(t.vs[1]);
    if (nans) {
      // rows that see a NaN value get NaN in that dim: visibility times
      // NaN-ness, then the NaNs leave the codes
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int ka = key0 + 16 * (j >> 1) + 4 * g + 2 * (j & 1);
          const bool ok = (t.ok >> (j >> 1)) & 1u;
          const bool a = ok && ka <= pos[rt] && (P.window == 0 || ka > pos[rt] - P.window);
          const bool c = ok && ka + 1 <= pos[rt] && (P.window == 0 || ka + 1 > pos[rt] - P.window);
          w[j] = (a ? 0x3f80u : 0u) | (c ? 0x3f800000u : 0u);
        }
        const bf16x8 see = pack8(w[0], w[1], w[2], w[3]);
#pragma unroll
        for (int dw = 0; dw < DP / 64; ++dw) {
          uint32_t lo[4], hi[4];
          transpose4(nan_bytes(t.v[0][dw]), nan_bytes(t.v[1][dw]), nan_bytes(t.v[2][dw]), nan_bytes(t.v[3][dw]), lo);
          transpose4(nan_bytes(t.v[4][dw]), nan_bytes(t.v[5][dw]), nan_bytes(t.v[6][dw]), nan_bytes(t.v[7][dw]), hi);
#pragma unroll
          for (int dd = 0; dd < 4; ++dd) {
            uint32_t a[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t y = (q < 2 ? lo[dd] : hi[dd]) >> (16 * (q & 1));
              a[q] = ((y & 0x80u) ? 0x3f80u : 0u) | ((y & 0x8000u) ? 0x3f800000u : 0u);
            }
            const f32x4 hit = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pack8(a[0], a[1], a[2], a[3]), see,
                                                                      f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (hit[q] > 0.f) acc[rt][4 * dw + dd][q] = __builtin_nanf("");
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int w = 0; w < DP / 64; ++w) {
          const uint32_t nb = nan_bytes(t.v[j][w]);
          t.v[j][w] &= ~((nb >> 7) * 0xffu);
        }
    }

    // O^T
#pragma unroll
    for (int dw = 0; dw < DP / 64; ++dw) {
      uint32_t lo[4], hi[4];
      transpose4(t.v[0][dw], t.v[1][dw], t.v[2][dw], t.v[3][dw], lo);
      transpose4(t.v[4][dw], t.v[5][dw], t.v[6][dw], t.v[7][dw], hi);
#pragma unroll
      for (int dd = 0; dd < 4; ++dd) {
        const bf16x8 va = pack8(widen2<false>(lo[dd], vsc0), widen2<true>(lo[dd], vsc0), widen2<false>(hi[dd], vsc1),
                                widen2<true>(hi[dd], vsc1));
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          acc[rt][4 * dw + dd] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(va, pb[rt], acc[rt][4 * dw + dd], 0, 0, 0);
      }
    }
  }

  // the four waves' sums joined: lane l holds of row l % 16 the dims
  // (4 g + q) DP/16 + dt
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    sum[rt] += lane_xor16(sum[rt]);
    sum[rt] += lane_xor32(sum[rt]);
    if (g == 0) {
      s_ref[wave][rt * 16 + r] = ref[rt];
      s_sum[wave][rt * 16 + r] = sum[rt];
    }
  }
  __syncthreads();  // (also: no wave reads Q any more)
  float* part = reinterpret_cast<float*>(s_mem);  // [wave][16][DP]
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    float top = kNoRef;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, s_ref[w][rt * 16 + r]);
    const float f = exp2_fast(ref[rt] - top);
    if (rt > 0) __syncthreads();
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int dt = 0; dt < DT; dt += 4)
        *reinterpret_cast<f32x4*>(part + (wave * 16 + r) * DP + (4 * g + q) * DT + dt) =
            f32x4{acc[rt][dt][q] * f, acc[rt][dt + 1][q] * f, acc[rt][dt + 2][q] * f, acc[rt][dt + 3][q] * f};
    __syncthreads();
    // 4 dims a thread
    for (int cell = tid; cell < 16 * (DP / 4); cell += kWG) {
      const int rr = cell / (DP / 4), d = (cell % (DP / 4)) * 4;
      const int64_t m = m0 + rt * 16 + rr;
      if (m >= m1 || d >= P.c.dim) continue;
      f32x4 o{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) o += *reinterpret_cast<const f32x4*>(part + (w * 16 + rr) * DP + d);
      float mx = kNoRef;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) mx = fmaxf(mx, s_ref[w][rt * 16 + rr]);
      float l = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) l += s_sum[w][rt * 16 + rr] * exp2_fast(s_ref[w][rt * 16 + rr] - mx);
      const int hq = head * G + (int)(m % G);
      const int64_t row = (int64_t)(q0 + m / G) * P.Hq + hq;
      if (P.nsplit > 1) {
        *reinterpret_cast<f32x4*>(P.po + (row * P.nsplit + sp) * P.c.dim + d) = o;
        if (d == 0) P.pm[row * P.nsplit + sp] = float2{mx, l};
      } else {
        if (P.sinks) {
          const float sk = P.sinks[hq] * 1.44269504088896341f;
          const float top2 = fmaxf(mx, sk);
          const float fa = exp2_fast(mx - top2);
          l = l * fa + exp2_fast(sk - top2);
          o *= fa;
          mx = top2;
        }
        // a row that sees nothing: l = 0
        const float inv = l == 0.f ? 0.f : 1.0f / l;
        uint32_t w[2];
#pragma unroll
        for (int q = 0; q < 2; ++q)
          w[q] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{o[2 * q] * inv, o[2 * q + 1] * inv}, bf16x2));
        *reinterpret_cast<u32x2*>(P.out + row * P.c.dim + d) = u32x2{w[0], w[1]};
        if (d == 0 && P.lse) P.lse[row] = l == 0.f ? -INFINITY : (mx + __builtin_amdgcn_logf(l)) * 0.693147180559945309f;
      }
    }
  }
}

// Joins the splits of a row: one wave per (token, query head).
__global__ __launch_bounds__(kWG) void attn_join_kernel(AttnParams P, int row_tiles) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (row >= (int64_t)P.N * P.Hq) return;
  const int tok = (int)(row / P.Hq), hq = (int)(row - (int64_t)tok * P.Hq);
  // the request that holds the token: the last b with q_start[b] <= tok
  int lo = 0, hi = P.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (P.q_start[mid] <= tok)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int q0 = P.q_start[lo], q1 = P.q_start[lo + 1];
  if (q0 < 0 || q1 > P.N || tok < q0 || tok >= q1) return;
  const int n = q1 - q0, ctx = P.ctx_len[lo];
  if (key_range(P, n, ctx, 0, n - 1).bad) return;  // its rows hold NaN already
  // the block of rows that held this one, and the splits that it has
  const int m = (tok - q0) * P.G + hq % P.G;
  const int rb = m / (16 * row_tiles);
  const int m1 = min(n * P.G, (rb + 1) * 16 * row_tiles);
  const KeyRange kr = key_range(P, n, ctx, rb * 16 * row_tiles / P.G, (m1 - 1) / P.G);
  const int ns = max(1, (int)(((int64_t)kr.hi - kr.lo + P.split_keys - 1) / P.split_keys));
  const float2* pm = P.pm + row * P.nsplit;
  float mx = P.sinks ? P.sinks[hq] * 1.44269504088896341f : kNoRef;
  for (int s = lane; s < ns; s += 64) mx = fmaxf(mx, pm[s].x);
  mx = wave_max_f(mx);
  float l = 0.f;
  for (int s = lane; s < ns; s += 64) l += pm[s].y * exp2_fast(pm[s].x - mx);
  l = (float)wave_total_d((double)l);
  if (P.sinks) l += exp2_fast(P.sinks[hq] * 1.44269504088896341f - mx);
  const float inv = l == 0.f ? 0.f : 1.0f / l;
  const float* po = P.po + row * P.nsplit * P.c.dim;
  for (int d = lane * 4; d < P.c.dim; d += 256) {
    f32x4 o{0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < ns; ++s) o += *reinterpret_cast<const f32x4*>(po + (int64_t)s * P.c.dim + d) * exp2_fast(pm[s].x - mx);
    uint32_t w[2];
#pragma unroll
    for (int q = 0; q < 2; ++q)
      w[q] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{o[2 * q] * inv, o[2 * q + 1] * inv}, bf16x2));
    *reinterpret_cast<u32x2*>(P.out + row * P.c.dim + d) = u32x2{w[0], w[1]};
  }
  if (lane == 0 && P.lse) P.lse[row] = l == 0.f ? -INFINITY : (mx + __builtin_amdgcn_logf(l)) * 0.693147180559945309f;
}

AttnPlan plan_attn(int32_t B, int32_t G, int32_t heads, int32_t dim, int32_t max_q, int32_t max_ctx, int32_t window) {
  AttnPlan p;
  const int64_t rows = (int64_t)max_q * G;
  const int64_t tiles = (rows + 15) / 16;
  const int rt_max = dim > 128 ? 2 : 4;
  p.rt = tiles <= 1 ? 1 : tiles <= 2 ? 2 : rt_max;
  p.nrb = (int32_t)((tiles + p.rt - 1) / p.rt);
  // keys that one block of rows can see, from a whole tile on
  int64_t keys = max_ctx;
  if (window > 0) {
    const int64_t toks = (p.rt * 16 + G - 1) / G + 1;
    const int64_t w = (int64_t)window + toks + kTileKeys;
    if (w < keys) keys = w;
  }
  const int64_t wgs = (int64_t)B * heads * p.nrb;
  int64_t ns = wgs > 0 ? 1024 / wgs : 1;
  const int64_t most = (keys + 511) / 512;  // at least 512 keys to a split
  if (ns > most) ns = most;
  if (ns < 1) ns = 1;
  const int64_t per = kWaves * kTileKeys;
  p.split_keys = (int32_t)(((keys + ns - 1) / ns + per - 1) / per * per);
  if (p.split_keys < per) p.split_keys = (int32_t)per;
  p.nsplit = (int32_t)((keys + p.split_keys - 1) / p.split_keys);
  if (p.nsplit < 1) p.nsplit = 1;
  return p;
}

template <int DP, int RT>
static hipError_t launch_attn_typed(const AttnParams& P, hipStream_t stream) {
  const int64_t grid = (int64_t)P.B * P.c.heads * P.nrb * P.nsplit;
  if (P.c.st_shift < 2)
    hipLaunchKernelGGL((attn_kernel<DP, RT, true>), dim3((unsigned)grid), dim3(kWG), 0, stream, P);
  else
    hipLaunchKernelGGL((attn_kernel<DP, RT, false>), dim3((unsigned)grid), dim3(kWG), 0, stream, P);
  return hipGetLastError();
}

template <int DP>
static hipError_t launch_attn_rows(const AttnParams& P, int rt, hipStream_t stream) {
  if (rt == 1) return launch_attn_typed<DP, 1>(P, stream);
  if (rt == 2) return launch_attn_typed<DP, 2>(P, stream);
  if constexpr (DP <= 128)
    return launch_attn_typed<DP, 4>(P, stream);
  else
    return hipErrorInvalidValue;
}

hipError_t launch_attn(const AttnParams& P, const AttnPlan& plan, hipStream_t stream) {
  hipError_t e;
  if (P.c.dim <= 64)
    e = launch_attn_rows<64>(P, plan.rt, stream);
  else if (P.c.dim <= 128)
    e = launch_attn_rows<128>(P, plan.rt, stream);
  else
    e = launch_attn_rows<256>(P, plan.rt, stream);
  if (e != hipSuccess || plan.nsplit <= 1) return e;
  const int64_t rows = (int64_t)P.N * P.Hq;
  hipLaunchKernelGGL(attn_join_kernel, dim3((unsigned)((rows + kWaves - 1) / kWaves)), dim3(kWG), 0, stream, P,
                     plan.rt);
  return hipGetLastError();
}

}  // namespace specv
