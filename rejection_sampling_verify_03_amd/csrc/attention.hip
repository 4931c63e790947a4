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
// range of keys, each of its four waves every fourth tile of 32 keys (or, for
// few rows, a KV head of its own), on its own: keys and values go from memory
// to the matrix units through registers alone, no barrier stands in the loop,
// and the waves' sums are joined once at the end.  Where there are few blocks
// with long contexts, the tiles of all blocks, end to end, are cut into equal
// runs, one to each workgroup that the card holds at once, whatever the lengths
// of the contexts; a second kernel joins the blocks that several runs hold
// (attention_plan.hpp).
//
// Both products run on v_mfma_f32_16x16x32_bf16 in the transposed order:
//   S^T (keys x rows) = K Q^T,   O^T (dims x rows) += V^T P^T,
// because lane l then holds row l % 16 of S^T for keys 4 (l / 16) + r, and
// with the 32 keys of a tile numbered
//   slot 8 g + j  =  key 4 g + j (j < 4),  key 16 + 4 g + j - 4 (j >= 4)
// that is where the second product wants P^T: the weights never leave their
// lanes.  The order of the sum over dims is free too: lane group g takes
// dims 64 w + 16 g ..+ 16 of the keys, so that keys are read in 16-byte loads
// of which four lanes' stand together.  The codes widen to bf16 exactly, scale
// included (one instruction for two); the values' bytes, which lie along dims,
// are first transposed four by four in registers.
//
// Weights are 2^(s_j log2(e) - ref) with a reference per row that moves only
// when a score passes it by 2^8: up to there the fp32 sums and the bf16
// weights lose nothing, and the sums are rarely rescaled.  The weights are
// rounded to bf16 for the second product (a relative error of at most 2^-8
// each, of no common sign, as the output's own rounding: the matrix units take
// both factors in one type, and the values are exact in bf16); where a scale
// covers fewer than 16 tokens it is multiplied into the weight before that,
// which is exact down to 2^-126.  Their sum is kept in fp32 from the unrounded
// weights, so lse keeps fp32's accuracy.
//
// Bounds, measured (MI355X).  Single tokens over long contexts: memory (three
// contexts of up to 131072 tokens, 691 MB, in 140 us; 131 us of it the main
// kernel, 5.3 TB/s; with all pages in L2 the call takes 84 us).  The
// verification batch, 72 rows to a KV head: instructions (128 us; 6 % less with
// all pages in L2; vector instructions in 55 % of the cycles, matrix
// instructions in 21 %).  A 2048-token chunk over 8192 tokens: the same (387 us,
// 0.8 PFLOP/s; vector 65 %, matrix 34 %: the two hardly overlap on two waves to
// a SIMD).  A prompt of 2048 tokens under a window of 128, where a wave has one
// or two tiles to a block: the fixed costs of a block (69 us, of 5 for bytes).
// RT is what 256 registers hold with few spilled: 5 row tiles at 64 dims (the 72
// rows of nine tokens and a group of eight in one block, 2 registers spilled
// with fine scales; 3 tiles: 175 us), 3 at 128 (7 spilled, 25 with fine scales;
// with 4 the chunk takes 992 us against 382), 1 at 256 (19, 27): there the
// verification batch is five units to a KV head, each of which reads the whole
// context (726 us with heads of 256, 251 with 128).  A second tile on
// its way in registers was no faster (133 against 133 us, long contexts 150
// against 141).
#include <limits.h>

#include "cache_device.hpp"

namespace specv {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

static_assert(kAttnWaves == kWaves, "waves of a workgroup");
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

// The kernels' parameters where the launch put them.  Values that only the
// start and the end of a unit need are read from there again (scalar loads of
// a cached line): kept in scalar registers through the loop over the keys they
// would not fit, and spill into vector registers.
typedef const AttnParams __attribute__((address_space(4)))* Params;
__device__ __forceinline__ Params params_again() {
  Params p = (Params)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return p;
}

// A unit of work: a block of 16 * RT rows of one request, for one KV head.
// Unit v is block v % nrb of request v / nrb; row k of it is token
// t0 + (h0 + k) / G of the request, head (h0 + k) % G of the group.
struct Unit {
  int b, q0, n, ctx;
  int t0, h0, rows;
  int lo, hi;      // the keys that its rows see lie in [lo, hi), lo a whole tile
  int p_lo, p_hi;  // positions of its first and last token
  int tiles;       // key tiles; 1 for a unit that only writes (nothing seen, or bad), 0 for no rows
  bool bad;        // the request's data cannot be used: its first unit writes NaN to all its rows
};

// x / G for the few rows of a block: a product and a shift, exact while
// x < 2^16 / G (x < 16 * RT + G here).
__device__ __forceinline__ int div_group(Params P, int x) { return (int)(((uint32_t)x * P->g_inv) >> 16); }

struct UnitData {
  int b, q0, q1, ctx;
};

__device__ __forceinline__ UnitData load_unit(Params P, int v) {
  const int b = v / P->nrb;
  return UnitData{b, P->q_start[b], P->q_start[b + 1], P->ctx_len[b]};
}

__device__ __forceinline__ Unit unit_from(Params P, int v, const UnitData& data, int block_rows) {
  Unit u;
  u.b = data.b;
  const int rb = v - u.b * P->nrb;
  u.q0 = data.q0;
  const int q1 = data.q1;
  u.ctx = data.ctx;
  u.n = q1 - u.q0;
  u.tiles = 0;
  u.t0 = u.h0 = u.rows = u.lo = u.hi = u.p_lo = u.p_hi = 0;
  u.bad = false;
  if (u.q0 < 0 || q1 > P->N || q1 <= u.q0) return u;
  const int64_t cap = min((int64_t)P->max_ctx, (int64_t)P->max_blocks << P->c.bs_shift);
  u.bad = u.ctx < 0 || u.ctx > cap || u.n > P->max_q;
  if (u.bad) {
    u.tiles = rb == 0;
    return u;
  }
  const int rows = u.n * P->G, m0 = rb * block_rows;  // at most 2^30 (max_q <= 2^24, G <= 64)
  if (m0 >= rows) return u;
  u.rows = min(rows - m0, block_rows);
  u.t0 = m0 / P->G;
  u.h0 = m0 - u.t0 * P->G;
  u.p_lo = u.ctx - u.n + u.t0;
  u.p_hi = u.p_lo + div_group(P, u.h0 + u.rows - 1);
  u.lo = (P->window > 0 ? max(0, u.p_lo - P->window + 1) : 0) & ~(kTileKeys - 1);
  u.hi = max(u.p_hi + 1, u.lo);
  u.tiles = max(1, (u.hi - u.lo + kTileKeys - 1) / kTileKeys);
  return u;
}

__device__ __forceinline__ Unit unit_of(Params P, int v, int block_rows) {
  return unit_from(P, v, load_unit(P, v), block_rows);
}

// A value that is the same in every lane, held in scalar registers.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform64(int64_t x) {
  return ((int64_t)uniform((int)(x >> 32)) << 32) | (uint32_t)uniform((int)x);
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

// Whether some byte is 0.
__device__ __forceinline__ bool zero_byte(uint32_t w) { return ((w - 0x01010101u) & ~w & 0x80808080u) != 0; }

// The largest of a lane's eight scores, three to an instruction.
__device__ __forceinline__ float max_of(const f32x4 (&s)[2]) {
  const float a = fmaxf(fmaxf(s[0][0], s[0][1]), s[0][2]), b = fmaxf(fmaxf(s[0][3], s[1][0]), s[1][1]);
  return fmaxf(fmaxf(fmaxf(s[1][2], s[1][3]), a), b);
}

// The lowest n bits, n clamped to 0..32.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// The keys of a tile that a row sees, a bit each: p is the row's position
// behind the tile's first key, ok the subtiles whose blocks exist.
__device__ __forceinline__ uint32_t seen_keys(int p, int window, uint32_t ok) {
  const uint32_t gone = window == 0 ? 0u : low_bits(p - window + 1);
  return low_bits(p + 1) & ~gone & ((ok & 1u) * 0xffffu | (ok >> 1) * 0xffff0000u);
}

// The place of row k of a run's partial sums: run j has two, for the unit that
// it begins with and for a later one (its last).
__device__ __forceinline__ int64_t part_row(Params P, int j, bool later, int head, int block_rows, int k) {
  return (((int64_t)j * 2 + later) * P->c.heads + head) * block_rows + k;
}

// What a row's sums of weights become: the factor of its sums of values, and
// its lse.  mx: their reference (log2); l: the sum of the weights, 0 if the row
// saw nothing.  Where the sink leads, or stands alone, lse is taken from the
// sink itself, so that it holds for sinks whose log2 is past fp32, and for
// infinite ones; where a score leads, such a sink adds nothing.
struct RowEnd {
  float f, lse;
};
__device__ __forceinline__ RowEnd row_end(Params P, int hq, float mx, float l) {
  constexpr float kLn2 = 0.693147180559945309f;
  if (P->sinks) {
    const float sink = P->sinks[hq], sk = sink * 1.44269504088896341f;
    if (l == 0.f || sk > mx) {
      const float f = l == 0.f ? 0.f : exp2_fast(mx - sk), sum = l * f + 1.0f;
      return RowEnd{f / sum, sink + __builtin_amdgcn_logf(sum) * kLn2};
    }
    l += exp2_fast(sk - mx);
  }
  return l == 0.f ? RowEnd{0.f, -INFINITY} : RowEnd{1.0f / l, (mx + __builtin_amdgcn_logf(l)) * kLn2};
}

// 4 dims of a row to the output, and with the first ones its lse.
__device__ __forceinline__ void store_row(Params P, int64_t row, int d, f32x4 o, RowEnd end) {
  uint32_t w[2];
#pragma unroll
  for (int q = 0; q < 2; ++q)
    w[q] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{o[2 * q] * end.f, o[2 * q + 1] * end.f}, bf16x2));
  *reinterpret_cast<u32x2*>(P->out + row * P->c.dim + d) = u32x2{w[0], w[1]};
  if (d == 0 && P->lse) P->lse[row] = end.lse;
}

// FINE: scale_tokens < 16, a scale for each key; otherwise one for each 16.
template <int DP, int RT, bool FINE>
__global__ __launch_bounds__(kWG, 2) void attn_kernel(AttnParams) {
  constexpr int C = DP / 32;   // steps of the sum over dims
  constexpr int DT = DP / 16;  // 16-dim tiles of the output
  constexpr int W = DP / 64;   // 16-byte loads of a lane's share of a key
  constexpr bool QREG = RT == 1 && C <= 4;  // Q's fragments stay in registers
  constexpr int kWindow = kAttnWindow;  // a subtile to a lane
  __shared__ __align__(16) char s_mem[(RT * C * 64 * 16 > kWaves * 16 * DP * 4) ? RT * C * 64 * 16
                                                                                : kWaves * 16 * DP * 4];
  __shared__ float s_ref[kWaves][RT * 16], s_sum[kWaves][RT * 16];
  __shared__ uint32_t s_nan[kWaves][DP];
  Params P = params_again();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // consecutive workgroups go to the 8 XCDs in turn; those that share lines
  // of the cache (P->items of them) stay on one
  int x = blockIdx.x >> 3;
  const int grp = (x / P->items) * 8 + (blockIdx.x & 7);
  if (grp >= P->groups) return;
  x = grp * P->items + x % P->items;
  const int units = P->B * P->nrb;

  // the waves share out hw heads and the tiles: wave w takes head w % hw and
  // every (kWaves / hw)-th tile
  const int hw = RT == 1 ? P->hw : 1, hs = wave & (hw - 1), ks = RT == 1 ? wave / hw : wave, kways = kAttnWaves / hw;
  const int hgroups = P->c.heads / hw;

  // the run of tiles [at, at + left) of unit v, v + 1, ... that this workgroup
  // takes for its heads: a whole unit, or (P->chunks > 0) one of the equal runs
  int v, at = 0, head0;
  int64_t left = INT64_MAX;
  if (P->chunks == 0) {
    const int rb = x % P->nrb;
    x /= P->nrb;
    head0 = x % hgroups * hw;
    v = (x / hgroups) * P->nrb + rb;
  } else {
    // the tiles of every 64 units, four of a wave's blocks on their way at a
    // time, then the block and the unit that hold the run's first tile
    // (one wave over all of them: 2000 contexts of 1500, two heads, 135 us against 106)
    const int lane = threadIdx.x & 63;
    head0 = x % hgroups * hw;
    double* s_tiles = reinterpret_cast<double*>(s_mem);
    static_assert(sizeof(s_mem) >= kMaxRunUnits / 64 * sizeof(double), "a place for each 64 units");
    const int blocks = (units + 63) / 64;
    auto tiles_of = [&](int v, const UnitData& data) {
      return v < units ? (double)unit_from(P, v, data, RT * 16).tiles : 0.0;
    };
    for (int k = wave; k < blocks; k += 4 * kWaves) {
      UnitData data[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) data[q] = load_unit(P, min((k + q * kWaves) * 64 + lane, units - 1));
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const double t = wave_total_d(tiles_of((k + q * kWaves) * 64 + lane, data[q]));
        if (lane == 0 && k + q * kWaves < blocks) s_tiles[k + q * kWaves] = t;
      }
    }
    __syncthreads();
    double sum = 0.0;
    for (int k = lane; k < blocks; k += 64) sum += s_tiles[k];
    const int64_t total = uniform64((int64_t)wave_total_d(sum));
    left = attn_run_tiles(total, P->chunks);
    const int64_t first = (int64_t)(x / hgroups) * left;
    if (first >= total) return;
    double base = 0.0;
    int k = 0;
    for (int k0 = 0;; k0 += 64) {  // (first < total: some block ends behind it)
      const double t = k0 + lane < blocks ? s_tiles[k0 + lane] : 0.0;
      const double end = wave_scan_d(t);
      const uint64_t past = __ballot(base + end > (double)first);
      if (past) {
        const int l = __builtin_ctzll(past);
        k = k0 + l;
        base += lane_d(end - t, l);
        break;
      }
      base += lane_d(end, 63);
    }
    const double t = tiles_of(k * 64 + lane, load_unit(P, min(k * 64 + lane, units - 1)));
    const double end = wave_scan_d(t);
    const int l = __builtin_ctzll(__ballot(base + end > (double)first));
    v = k * 64 + l;
    at = uniform((int)((double)first - (base + lane_d(end - t, l))));
    __syncthreads();  // (Q takes that memory next)
  }

  for (bool run_begin = true;; run_begin = false) {
  // the lane's number anew for each unit: what derives from it would
  // otherwise be kept in registers over the whole loop
  P = params_again();
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int lane = tid & 63, r = lane & 15, g = lane >> 4;
  const int G = P->G, dim = P->c.dim;
  const int tok_stride = (int)P->c.token;
  // a lane whose dims are past the head's takes the key's first ones instead:
  // Q is 0 there, and those dims of the output are not stored
  uint32_t koff[W];
#pragma unroll
  for (int w = 0; w < W; ++w)
    koff[w] = (uint32_t)(r * tok_stride + (w * 64 + g * 16 < dim ? w * 64 + g * 16 : 0));
  const uint32_t voff = (uint32_t)(4 * g * tok_stride + (r * (DP / 16) < dim ? r * (DP / 16) : 0));
  const Unit un = unit_of(P, v, RT * 16);
  const int len = (int)min(left, (int64_t)(un.tiles - at));  // of this unit
  if (un.bad && un.tiles > 0) {
    const int gw = G * hw;  // (query heads of the workgroup's heads stand together)
    for (int64_t m = tid; m < (int64_t)un.n * gw; m += kWG) {
      const int64_t row = (int64_t)(un.q0 + m / gw) * P->Hq + head0 * G + m % gw;
      for (int d = 0; d < P->c.dim; ++d) P->out[row * P->c.dim + d] = 0x7fc0;
      if (P->lse) P->lse[row] = __builtin_nanf("");
    }
  } else if (un.tiles > 0) {
  const int k_beg = un.lo + at * kTileKeys, k_end = min(un.hi, k_beg + len * kTileKeys);
  const bool joined = len < un.tiles;  // other runs hold more of this unit's keys
  const int head = head0 + hs;  // this wave's
  const int nt = (len - ks + kways - 1) / kways;

  // Q, to become the fragments of the first product in LDS: fragment (rt, c),
  // lane l: row 16 rt + l % 16, dims 64 (c / 2) + 16 (l / 16) + 8 (c % 2) ..+ 8
  // (RT = 1: a wave's own head's)
  constexpr int QF = RT == 1 ? C : (RT * C * 64 + kWG - 1) / kWG;
  u32x4 qreg[QF];
#pragma unroll
  for (int i = 0; i < QF; ++i) {
    const int f = RT == 1 ? i * 64 + lane : tid + i * kWG;
    const int l = f & 63, cc = (f >> 6) % C, rt = (f >> 6) / C;
    const int k = rt * 16 + (l & 15);
    const int d = (cc >> 1) * 64 + (l >> 4) * 16 + (cc & 1) * 8;
    qreg[i] = u32x4{0, 0, 0, 0};
    if (k < un.rows && d < P->c.dim) {
      const int t = div_group(P, un.h0 + k);
      const uint16_t* src = reinterpret_cast<const uint16_t*>(P->q) + (int64_t)(un.q0 + un.t0 + t) * P->q_tok +
                            (int64_t)(head * G + un.h0 + k - t * G) * P->q_head + d;
      if (P->qvec) {
        qreg[i] = *reinterpret_cast<const u32x4*>(src);
      } else {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = (uint32_t)src[2 * j] | ((uint32_t)src[2 * j + 1] << 16);
        qreg[i] = u32x4{w[0], w[1], w[2], w[3]};
      }
    }
  }

  int pos[RT];  // the position of this lane's row, -1 for rows past the block
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int k = rt * 16 + r;
    pos[rt] = k < un.rows ? un.p_lo + div_group(P, un.h0 + k) : -1;
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

  const float scale2 = P->scale2;
  const int window = P->window;
  const uint8_t *k_codes = P->c.codes[0], *v_codes = P->c.codes[1];
  const u32x4* qf = reinterpret_cast<const u32x4*>(s_mem) + (RT == 1 ? wave * C * 64 : 0) + lane;

  // Lane l knows subtile l % 2 of tile i0 + l / 2 of this wave: where its keys
  // begin, whether their block exists, and (!FINE) their scales.
  int pg_lo = 0, pg_hi = 0, sc_lo = 0, sc_hi = 0, ksv = 0, vsv = 0;
  uint64_t okv = 0, knone = 0, vnone = 0;  // (knone, vnone: !FINE, scale bytes of 0)
  auto look_up = [&](int i0) {
    const Params P = params_again();
    const int32_t* bt = P->bt + (int64_t)un.b * P->bt_stride;
    const int key = k_beg + ((i0 + (lane >> 1)) * kways + ks) * kTileKeys + (lane & 1) * 16;
    const int lb = key >> P->c.bs_shift, in = key & ((1 << P->c.bs_shift) - 1);
    int page = -1;
    if (key < k_end && lb < P->max_blocks) page = bt[lb];
    const bool ok = page >= 0 && page < P->c.num_blocks;
    page = ok ? page : 0;
    okv = __ballot(ok);
    const int64_t po = (int64_t)page * P->c.block + (int64_t)head * P->c.head + (int64_t)in * P->c.token;
    const int64_t so = (int64_t)page * P->c.sblock + (int64_t)head * P->c.shead + (in >> P->c.st_shift);
    pg_lo = (int)po;
    pg_hi = (int)(po >> 32);
    if constexpr (FINE) {
      sc_lo = (int)so;
      sc_hi = (int)(so >> 32);
    } else {
      ksv = P->c.scales[0][so];
      vsv = P->c.scales[1][so];
      knone = __ballot(ok && ksv == 0);
      vnone = __ballot(ok && vsv == 0);
    }
  };
  auto lane64 = [&](int lo, int hi, int l) { return ((int64_t)lane_i(hi, l) << 32) | (uint32_t)lane_i(lo, l); };

  // subtile u: key l % 16, dims 64 w + 16 g ..+ 16; slot j's key, dims
  // [r DP/16, (r+1) DP/16)
  struct Buffer {
    u32x4 k[2][W];
    uint32_t v[8][W];
    uint32_t kfine[2], vfine[2];  // (FINE) scale bytes of key r, and of keys 4 g ..+ 4
    float ksc[2], vsc[2];
    uint32_t ok;  // bits: 0, 1 the subtiles' blocks exist; 2, 3 their keys' scale is 0; 4, 5 their values'
  } buf;
  auto load_k = [&](int i) {
    Buffer& t = buf;
    if ((i & (kWindow - 1)) == 0) look_up(i);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int l = ((i & (kWindow - 1)) << 1) + u;
      const uint8_t* kb = k_codes + lane64(pg_lo, pg_hi, l);
#pragma unroll
      for (int w = 0; w < W; ++w) t.k[u][w] = *reinterpret_cast<const u32x4*>(kb + koff[w]);
      if constexpr (FINE) {
        const int64_t so = lane64(sc_lo, sc_hi, l);
        t.kfine[u] = P->c.scales[0][so + (uint32_t)(r >> P->c.st_shift)];
      } else {
        t.ksc[u] = scale_of((uint32_t)lane_i(ksv, l));
      }
    }
    const int l0 = (i & (kWindow - 1)) << 1;
    t.ok = (uint32_t)(okv >> l0) & 3u;
    if constexpr (!FINE) t.ok |= ((uint32_t)(knone >> l0) & 3u) << 2 | ((uint32_t)(vnone >> l0) & 3u) << 4;
  };
  auto load_v = [&](int i) {
    Buffer& t = buf;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int l = ((i & (kWindow - 1)) << 1) + u;
      const uint8_t* vb = v_codes + lane64(pg_lo, pg_hi, l);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint8_t* p = vb + (int64_t)j * tok_stride;
        if constexpr (W == 1) {
          t.v[4 * u + j][0] = *reinterpret_cast<const uint32_t*>(p + voff);
        } else if constexpr (W == 2) {
          const u32x2 w = *reinterpret_cast<const u32x2*>(p + voff);
          t.v[4 * u + j][0] = w.x;
          t.v[4 * u + j][1] = w.y;
        } else {
          const u32x4 w = *reinterpret_cast<const u32x4*>(p + voff);
          t.v[4 * u + j][0] = w.x;
          t.v[4 * u + j][1] = w.y;
          t.v[4 * u + j][2] = w.z;
          t.v[4 * u + j][3] = w.w;
        }
      }
      if constexpr (FINE) {
        const uint8_t* sb = P->c.scales[1] + lane64(sc_lo, sc_hi, l) + (uint32_t)((4 * g) >> P->c.st_shift);
        if (P->c.st_shift == 0) {
          uint32_t w;
          __builtin_memcpy(&w, sb, 4);
          t.vfine[u] = w;
        } else if (P->c.st_shift == 1) {
          t.vfine[u] = (uint32_t)sb[0] * 0x0101u | (uint32_t)sb[1] * 0x01010000u;
        } else {
          t.vfine[u] = (uint32_t)sb[0] * 0x01010101u;
        }
      } else {
        t.vsc[u] = scale_of((uint32_t)lane_i(vsv, l));
      }
    }
  };

  auto tile = [&](int i) {
    Buffer& t = buf;
    // more than a few fragments of Q are read from LDS for every tile rather
    // than kept in registers (the compiler would move the reads out of the loop)
    if constexpr (!QREG && RT * C > 4) asm volatile("" ::: "memory");
    const int key0 = k_beg + (i * kways + ks) * kTileKeys;
    const uint32_t okt = t.ok & 3u;
    // a scale byte of 0 (never written): values of 0, whatever the codes
    const uint32_t v_none = t.ok >> 4;
    if (FINE ? __ballot(t.kfine[0] == 0 || t.kfine[1] == 0) != 0 : (t.ok & 12u) != 0) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const bool none = FINE ? t.kfine[u] == 0 : ((t.ok >> (2 + u)) & 1u) != 0;
#pragma unroll
        for (int w = 0; w < W; ++w) t.k[u][w] = none ? u32x4{0, 0, 0, 0} : t.k[u][w];
      }
    }
    // every row of the block sees every key of the tile
    const bool whole = okt == 3u && key0 + kTileKeys - 1 <= un.p_lo && (window == 0 || key0 > un.p_hi - window);

    // S^T
    f32x4 s[RT][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float sc = FINE ? scale_of(t.kfine[u]) : t.ksc[u];
      bf16x8 ka[C];
#pragma unroll
      for (int cc = 0; cc < C; ++cc) {
        const u32x4 w4 = t.k[u][cc / 2];
        const uint32_t w0 = (cc & 1) ? w4.z : w4.x, w1 = (cc & 1) ? w4.w : w4.y;
        ka[cc] = pack8(widen2<false>(w0, sc), widen2<true>(w0, sc), widen2<false>(w1, sc), widen2<true>(w1, sc));
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) s[rt][u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int cc = 0; cc < C; ++cc)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          s[rt][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              ka[cc], __builtin_bit_cast(bf16x8, QREG ? qreg[QREG ? cc : 0] : qf[(rt * C + cc) * 64]), s[rt][u],
              0, 0, 0);
    }
    load_k(min(i + 1, nt - 1));
    if (FINE ? __ballot(zero_byte(t.vfine[0]) || zero_byte(t.vfine[1])) != 0 : v_none != 0) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool none = FINE ? ((t.vfine[u] >> (8 * j)) & 0xffu) == 0 : ((v_none >> u) & 1u) != 0;
#pragma unroll
          for (int w = 0; w < W; ++w) t.v[4 * u + j][w] = none ? 0u : t.v[4 * u + j][w];
        }
    }

    // a tile that some row sees only in part: scores not seen become -inf;
    // nothing of the keys that no row sees may enter (0 * NaN, 0 * inf), and a
    // NaN among the others is kept apart
    bool nans = false;
    if (!whole) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        bool some = false;
        uint32_t fine = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int key = key0 + 16 * u + 4 * g + j;
          const bool there = (okt >> u) & 1u;
          const bool any = there && key <= un.p_hi && (window == 0 || key > un.p_lo - window);
          some |= any;
#pragma unroll
          for (int w = 0; w < W; ++w) {
            t.v[4 * u + j][w] = any ? t.v[4 * u + j][w] : 0u;
            nans |= nan_bytes(t.v[4 * u + j][w]) != 0;
          }
          if constexpr (FINE) fine |= any ? t.vfine[u] & (0xffu << (8 * j)) : (uint32_t)kScaleBias << (8 * j);
        }
        if constexpr (FINE) t.vfine[u] = fine;
        if constexpr (!FINE) t.vsc[u] = __ballot(some) ? t.vsc[u] : 1.0f;
        __builtin_amdgcn_sched_barrier(0);  // (few conditions at a time: each is a pair of scalar registers)
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        // bit 16 u + 4 g + j of `see`: the row sees that key
        const uint32_t see = seen_keys(pos[rt] - key0, window, okt) >> (4 * g);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[rt][u][j] = (see >> (16 * u + j)) & 1u ? s[rt][u][j] : -INFINITY;
        __builtin_amdgcn_sched_barrier(0);
      }
      nans = __ballot(nans) != 0;
    }

    // the weights, against a reference that follows the scores
    bool move = false;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      move |= max_of(s[rt]) * scale2 > ref[rt] + kRefSlack;
    }
    if (__ballot(move)) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        float mx = fmaxf(ref[rt], max_of(s[rt]) * scale2);
        mx = fmaxf(mx, lane_xor16(mx));
        mx = fmaxf(mx, lane_xor32(mx));
        const float f = exp2_fast(ref[rt] - mx);
        ref[rt] = mx;
        sum[rt] *= f;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) acc[rt][dt] *= f;
      }
    }
    bf16x8 pb[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      float p[8];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) p[4 * u + j] = exp2_fast(__builtin_fmaf(s[rt][u][j], scale2, -ref[rt]));
      sum[rt] += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
      if constexpr (FINE) {
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] *= scale_of((t.vfine[j >> 2] >> (8 * (j & 3))) & 0xffu);
      }
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{p[2 * j], p[2 * j + 1]}, bf16x2));
      pb[rt] = pack8(w[0], w[1], w[2], w[3]);
    }

    if (nans) {
      // a row that sees a NaN value gets NaN in that dim: the keys with a NaN
      // in each dim as a mask in LDS, against the keys that a row sees; then
      // the NaNs leave the codes
      uint32_t* mask = s_nan[wave];
      for (int d = lane; d < DP; d += 64) mask[d] = 0;
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const uint32_t nb = nan_bytes(t.v[j][w]);
          for (uint32_t m = nb; m; m &= m - 1)
            atomicOr(&mask[r * DT + 4 * w + (__builtin_ctz(m) >> 3)], 1u << (16 * (j >> 2) + 4 * g + (j & 3)));
          t.v[j][w] &= ~((nb >> 7) * 0xffu);
        }
      __builtin_amdgcn_wave_barrier();
      uint32_t see[RT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) see[rt] = seen_keys(pos[rt] - key0, window, okt);
#pragma unroll
      for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t m = mask[(4 * g + q) * DT + dt];
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) acc[rt][dt][q] = m & see[rt] ? __builtin_nanf("") : acc[rt][dt][q];
          __builtin_amdgcn_sched_barrier(0);  // (one at a time: the path is rare and must not cost registers)
        }
    }

    // O^T
    const float v0 = FINE ? 1.0f : t.vsc[0], v1 = FINE ? 1.0f : t.vsc[1];
#pragma unroll
    for (int dw = 0; dw < W; ++dw) {
      uint32_t lo[4], hi[4];
      transpose4(t.v[0][dw], t.v[1][dw], t.v[2][dw], t.v[3][dw], lo);
      transpose4(t.v[4][dw], t.v[5][dw], t.v[6][dw], t.v[7][dw], hi);
#pragma unroll
      for (int dd = 0; dd < 4; ++dd) {
        const bf16x8 va = pack8(widen2<false>(lo[dd], v0), widen2<true>(lo[dd], v0), widen2<false>(hi[dd], v1),
                                widen2<true>(hi[dd], v1));
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          acc[rt][4 * dw + dd] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(va, pb[rt], acc[rt][4 * dw + dd], 0, 0, 0);
      }
    }
    load_v(min(i + 1, nt - 1));
  };
  // (in this order the first tile is on its way before Q is waited for)
  if (nt > 0) {
    load_k(0);
    load_v(0);
  }
#pragma unroll
  for (int i = 0; i < QF; ++i) {
    qreg[i] = (qreg[i] & P->q_keep) ^ P->q_flip;
    if (RT > 1 && tid + i * kWG < RT * C * 64) reinterpret_cast<u32x4*>(s_mem)[tid + i * kWG] = qreg[i];
    if (RT == 1 && !QREG) reinterpret_cast<u32x4*>(s_mem)[(wave * C + i) * 64 + lane] = qreg[i];
  }
  if (!QREG) __syncthreads();
  // every tile's loads are unconditional (the last ones' read a tile again):
  // behind a condition the compiler could not count the loads in flight, and
  // would wait for the values just asked for before it uses the keys
  for (int i = 0; i < nt; ++i) tile(i);

  P = params_again();
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
    for (int w = hs; w < kWaves; w += hw) top = fmaxf(top, s_ref[w][rt * 16 + r]);
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
    for (int cell = tid; cell < hw * 16 * (DP / 4); cell += kWG) {
      const int w0 = cell / (16 * (DP / 4)), rr = cell / (DP / 4) % 16, d = (cell % (DP / 4)) * 4;
      const int k = rt * 16 + rr;
      if (k >= un.rows || d >= P->c.dim) continue;
      f32x4 o{0.f, 0.f, 0.f, 0.f};
      float mx = kNoRef;
      for (int w = w0; w < kWaves; w += hw) {
        o += *reinterpret_cast<const f32x4*>(part + (w * 16 + rr) * DP + d);
        mx = fmaxf(mx, s_ref[w][rt * 16 + rr]);
      }
      float l = 0.f;
      for (int w = w0; w < kWaves; w += hw) l += s_sum[w][rt * 16 + rr] * exp2_fast(s_ref[w][rt * 16 + rr] - mx);
      const int t = div_group(P, un.h0 + k);
      const int hq = (head0 + w0) * G + un.h0 + k - t * G;
      const int64_t row = (int64_t)(un.q0 + un.t0 + t) * P->Hq + hq;
      if (joined) {
        const int64_t pr = part_row(P, grp, !run_begin, head0 + w0, RT * 16, k);
        *reinterpret_cast<f32x4*>(P->po + pr * P->c.dim + d) = o;
        if (d == 0) P->pm[pr] = float2{mx, l};
      } else {
        store_row(P, row, d, o, row_end(P, hq, mx, l));
      }
    }
  }
  }
  // which runs hold the unit, for the join (one workgroup of the heads tells it)
  if (P->chunks > 0 && head0 == 0 && threadIdx.x == 0 && un.tiles > 0) {
    if (at == 0) P->runs[v].x = grp * 2 + !run_begin;
    if (at + len == un.tiles) P->runs[v].y = grp;
  }
  // the next unit of the run
  left -= len;
  at = 0;
  if (P->chunks == 0 || left <= 0 || ++v >= units) break;
  __syncthreads();
  }
}

// Joins the runs of a unit that several hold: one workgroup per (unit, KV
// head, 16 rows), 4 dims a thread, the runs of a row shared out to what
// threads are left (a decode step of a few long contexts has few rows and many
// runs; there the workgroup is large).
template <int COLS, int NT>  // threads to a row, to a workgroup
__global__ __launch_bounds__(NT) void attn_join_kernel(AttnParams, int row_tiles) {
  constexpr int NS = NT / COLS;
  __shared__ float4 s_o[NT];
  __shared__ float2 s_ml[NT];
  const Params P = params_again();
  const int rt = blockIdx.x % row_tiles, x = blockIdx.x / row_tiles;
  const int v = x / P->c.heads, head = x % P->c.heads;
  const int2 runs = P->runs[v];  // (of a unit without rows: never written, and not used)
  const Unit u = unit_of(P, v, row_tiles * 16);
  const int j0 = runs.x >> 1, j1 = runs.y;
  const int rows = min(16, u.rows - rt * 16);
  if (u.bad || u.tiles <= 1 || rows <= 0 || j0 == j1) return;  // written whole
  const bool late = runs.x & 1;  // its first run began with another unit
  const int shift = rows > 8 ? 4 : rows > 4 ? 3 : rows > 2 ? 2 : rows > 1 ? 1 : 0;  // rows, rounded up to 2^shift
  const int tid = threadIdx.x, slot = tid / COLS, d = (tid % COLS) * 4;
  const bool wide = NS >= (1 << shift);  // (else the rows are taken in turn, each by one thread a column)
  const int ways = wide ? NS >> shift : 1, way = wide ? slot >> shift : 0;
  for (int r0 = 0; r0 < rows; r0 += NS) {
    const int k = rt * 16 + (wide ? slot & ((1 << shift) - 1) : r0 + slot);
    const bool on = k < u.rows && k < rt * 16 + 16 && d < P->c.dim;
    // eight runs' sums on their way at a time
    float mx = kNoRef, l = 0.f;
    f32x4 o{0.f, 0.f, 0.f, 0.f};
    for (int j = j0 + way; on && j <= j1; j += 8 * ways) {
      float2 p[8];
      f32x4 a[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int jj = min(j + q * ways, j1);
        const int64_t part = part_row(P, jj, late && jj == j0, head, row_tiles * 16, k);
        p[q] = P->pm[part];
        a[q] = *reinterpret_cast<const f32x4*>(P->po + part * P->c.dim + d);
      }
      float m = mx;
#pragma unroll
      for (int q = 0; q < 8; ++q) m = j + q * ways <= j1 ? fmaxf(m, p[q].x) : m;
      const float f = exp2_fast(mx - m);
      l *= f;
      o *= f;
      mx = m;
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (j + q * ways <= j1) {
          const float w = exp2_fast(p[q].x - m);
          l += p[q].y * w;
          o += a[q] * w;
        }
    }
    if (ways > 1) {
      s_o[tid] = float4{o.x, o.y, o.z, o.w};
      s_ml[tid] = float2{mx, l};
      __syncthreads();
      if (way == 0) {
        for (int w = 1; w < ways; ++w) {
          const int at = tid + (w << shift) * COLS;
          const float2 p = s_ml[at];
          const float4 q = s_o[at];
          const float m = fmaxf(mx, p.x);
          const float f = exp2_fast(mx - m), g = exp2_fast(p.x - m);
          l = l * f + p.y * g;
          o = o * f + f32x4{q.x, q.y, q.z, q.w} * g;
          mx = m;
        }
      }
    }
    if (!on || way != 0) continue;
    const int t = div_group(P, u.h0 + k);
    const int hq = head * P->G + u.h0 + k - t * P->G;
    const int64_t row = (int64_t)(u.q0 + u.t0 + t) * P->Hq + hq;
    store_row(P, row, d, o, row_end(P, hq, mx, l));
  }
}

template <int DP, int RT>
static hipError_t launch_attn_typed(const AttnParams& P, hipStream_t stream) {
  const dim3 grid((unsigned)(((int64_t)P.groups + 7) / 8 * 8 * P.items));
  if (P.c.st_shift < 4)
    hipLaunchKernelGGL((attn_kernel<DP, RT, true>), grid, dim3(kWG), 0, stream, P);
  else
    hipLaunchKernelGGL((attn_kernel<DP, RT, false>), grid, dim3(kWG), 0, stream, P);
  return hipGetLastError();
}

template <int DP>
static hipError_t launch_attn_rows(const AttnParams& P, int rt, hipStream_t stream) {
  if (rt == 1) return launch_attn_typed<DP, 1>(P, stream);
  if constexpr (DP <= 128) {
    if (rt == 2) return launch_attn_typed<DP, 2>(P, stream);
    if (rt == 3) return launch_attn_typed<DP, 3>(P, stream);
  }
  if constexpr (DP <= 64) {
    if (rt == 4) return launch_attn_typed<DP, 4>(P, stream);
    if (rt == 5) return launch_attn_typed<DP, 5>(P, stream);
  }
  return hipErrorInvalidValue;
}

template <int COLS>
static hipError_t launch_join(const AttnParams& P, const AttnPlan& plan, hipStream_t stream) {
  const dim3 grid((unsigned)(P.B * P.nrb * P.c.heads * plan.rt));
  // many runs to a unit: 10 us against 25 for three units of 85 runs; few runs
  // and many units: 10 us with small workgroups
  if (plan.chunks > 8 * P.B * P.nrb)
    hipLaunchKernelGGL((attn_join_kernel<COLS, 1024>), grid, dim3(1024), 0, stream, P, plan.rt);
  else
    hipLaunchKernelGGL((attn_join_kernel<COLS, kWG>), grid, dim3(kWG), 0, stream, P, plan.rt);
  return hipGetLastError();
}

hipError_t launch_attn(const AttnParams& P, const AttnPlan& plan, hipStream_t stream) {
  hipError_t e;
  if (P.c.dim <= 64)
    e = launch_attn_rows<64>(P, plan.rt, stream);
  else if (P.c.dim <= 128)
    e = launch_attn_rows<128>(P, plan.rt, stream);
  else
    e = launch_attn_rows<256>(P, plan.rt, stream);
  if (e != hipSuccess || plan.chunks == 0) return e;
  return P.c.dim <= 64 ? launch_join<16>(P, plan, stream)
                       : P.c.dim <= 128 ? launch_join<32>(P, plan, stream) : launch_join<64>(P, plan, stream);
}

}  // namespace specv
