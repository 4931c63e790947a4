// ops_kernels.hpp -- parameter blocks and launchers of the operators around
// a verification step: token log probabilities, the 8-bit paged cache and
// the attention over it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attention_plan.hpp"
#include "spec_verify.h"
#include "verify_layout.hpp"

namespace specv {

// ------------------------------------------------------ log probabilities --
struct LpRecord {  // one 4096-logit segment of a row
  float m;         // largest logit
  float s;         // sum of 2^((x - m) * log2(e) / T)
  float w;         // sum of the same times its exponent
  float pad;
};
static_assert(sizeof(LpRecord) == 16, "LpRecord layout");

constexpr int kLpCells = 64;     // cells of 64 consecutive logits in a segment
constexpr int kLpChunkSegs = 8;  // segments per workgroup of the statistics pass

// n / d for 0 <= n < 2^31 as a product and a shift (a scalar division is some
// forty vector instructions, in every wave): with 2^s the largest power of two
// below d, mul = ceil(2^(32+s) / d) < 2^32 is off by less than d from exact,
// which stays below one quotient for n < 2^31.
struct FastDiv {
  uint32_t mul, shift;  // mul 0: d = 1
  __host__ __device__ static FastDiv by(uint32_t d) {
    uint32_t s = 0;
    while (d > 1 && (2u << s) < d) ++s;
    return d > 1 ? FastDiv{(uint32_t)(((1ull << (32 + s)) + d - 1) / d), s} : FastDiv{0, 0};
  }
  __host__ __device__ uint32_t of(uint32_t n) const {
    return mul ? (uint32_t)(((uint64_t)n * mul) >> 32) >> shift : n;
  }
};

struct LogprobsParams {
  int32_t B, R, V, nseg, C, top;  // C: chunks of kLpChunkSegs segments per row
  FastDiv by_C, by_R;
  const char* logits;
  int64_t req, row;
  const int32_t* tokens;
  const float* temperature;  // or null
  float* logprobs;
  float* entropy;  // or null
  int32_t* top_ids;
  float* top_lp;
  LpRecord* rec;   // [B * R, nseg]
  float* cells;    // [B * R, nseg, kLpCells] largest logit of each cell (top > 0)
};

hipError_t launch_logprobs(const LogprobsParams& P, int dtype, hipStream_t stream);

// ------------------------------------------------------------ paged cache --
struct CacheView {
  int32_t num_blocks, heads, dim;
  int32_t bs_shift, st_shift;  // log2 of block_size and scale_tokens
  uint8_t* codes[2];           // keys, values
  uint8_t* scales[2];
  int64_t block, token, head;  // strides of the codes, bytes
  int64_t sblock, shead;       // strides of the scales, bytes
};

struct KvWriteParams {
  CacheView c;
  int32_t N, chunk;  // entries per workgroup
  const char* src[2];
  int64_t tok[2], hd[2];  // strides in elements
  const int64_t* slots;
};

struct KvReadParams {
  CacheView c;
  int32_t N, per;  // per: entries per workgroup
  char* dst[2];
  const int64_t* slots;
};

constexpr int kReadCells = 4;  // cells of 8 elements that a lane of the read has on their way
// Entries to a workgroup of the read: one round of kReadCells cells a lane,
// whole entries, but few of them where the card would not be filled.
inline int32_t kv_read_per(int32_t N, int32_t heads, int32_t dim) {
  const int64_t most = 256 * kReadCells / ((int64_t)heads * (dim >> 3)), spread = ((int64_t)N + 1023) / 1024;
  return (int32_t)(most < 1 ? 1 : most < spread ? most : spread);
}
// Entries to a workgroup of the write: few where there are few, so that they
// spread over the card (32 for a prompt: 38 us against 41 with 64 and 47 with
// 16 on 32771 tokens of 8 heads of 128).
inline int32_t kv_write_chunk(int32_t N) { return N >= 8192 ? 32 : N >= 1024 ? 16 : 4; }
hipError_t launch_kv_write(const KvWriteParams& P, int dtype, hipStream_t stream);
hipError_t launch_kv_read(const KvReadParams& P, int dtype, bool vec, hipStream_t stream);

// -------------------------------------------------------------- attention --
struct AttnParams {
  CacheView c;
  int32_t B, N, Hq, G;  // G: query heads per KV head
  uint32_t g_inv;       // 65535 / G + 1
  int32_t max_q, max_ctx, window, max_blocks;
  int32_t nrb, chunks;              // row blocks per (request, KV head); equal runs of tiles (0: a unit each)
  int32_t hw;                       // KV heads of a workgroup (1, 2 or 4)
  int32_t items, groups;            // workgroups kept on one XCD, and how many such sets
  // the scores are scale2 * q . k with scale2 = |scale| * log2(e) > 0: a
  // negative scale is the sign of q (q_flip: the sign bits of two bf16), a
  // scale of 0 a q of 0 (q_keep = 0, else all bits)
  uint32_t q_flip, q_keep;
  float scale2;
  const char* q;
  int64_t q_tok, q_head;  // elements
  const int32_t* q_start;
  const int32_t* ctx_len;
  const int32_t* bt;
  int64_t bt_stride;
  const float* sinks;
  uint16_t* out;
  float* lse;
  float* po;   // [chunks, 2, heads, 16 * rt, dim] partial sums (chunks > 0)
  float2* pm;  // [chunks, 2, heads, 16 * rt] their reference exponents and sums of weights
  int2* runs;  // [B * nrb] the runs that hold each unit: (first * 2 + whether it began with another unit, last)
  int32_t qvec;
};

hipError_t launch_attn(const AttnParams& P, const AttnPlan& plan, hipStream_t stream);

}  // namespace specv
