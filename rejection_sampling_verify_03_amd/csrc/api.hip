// api.hip -- the C ABI: host-side argument validation, workspace sizing and
// kernel launches.  Every check here runs before anything is enqueued, and no
// launch entry point synchronises the stream or allocates memory (the host
// query spec_workspace_error waits for the stream it is given).
#include <float.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

#include "spec_verify.h"
#include "ops_kernels.hpp"
#include "overlap.hpp"
#include "verify_kernels.hpp"
#include "verify_layout.hpp"

using namespace specv;

// The workspace of spec_verify_launch_noalloc: one copy of this array per GPU
// the library runs on, held until the process ends.  Host code never passes
// its name to a kernel (on the host it is only a stand-in for the symbol): it
// uses the device address hipGetSymbolAddress gives for the current device.
static __device__ __align__(256) unsigned char scratch[SPEC_NOALLOC_SCRATCH_BYTES];

namespace {

constexpr int64_t kExpandRowsPerWG = 4;
constexpr int64_t kThreads = 256;  // per workgroup of the statistics, cache and attention kernels

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// [n, m, len] elements of es bytes by their strides.
MemRows mem_rows(const void* base, int32_t n, int64_t outer, int32_t m, int64_t inner, int64_t len, int64_t es) {
  constexpr int64_t kMost = INT64_MAX / 4;  // (in bytes within 64 bits; no memory is so large)
  auto bytes = [&](int32_t rows, int64_t stride) { return rows > 1 ? (stride < kMost ? stride : kMost) * es : 0; };
  return MemRows{(uintptr_t)base, n, bytes(n, outer), m, bytes(m, inner), len * es};
}

// Device address of `scratch` per device, looked up on the first call made
// with that device current (a lookup, not an allocation).
constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch[kMaxDevices] = {};

int scratch_address(hipStream_t stream, void** out) {
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return SPEC_ELAUNCH;
  if (stream != nullptr) {  // the lookup is for the current device: the stream must be on it
    hipDevice_t sdev = -1;
    if (hipStreamGetDevice(stream, &sdev) != hipSuccess) return SPEC_ELAUNCH;
    if (sdev != dev) return SPEC_EINVAL;
  }
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (g_scratch[dev] == nullptr) {
    void* ptr = nullptr;
    if (hipGetSymbolAddress((void**)&ptr, HIP_SYMBOL(scratch)) != hipSuccess || ptr == nullptr)
      return SPEC_ELAUNCH;
    g_scratch[dev] = ptr;
  }
  *out = g_scratch[dev];
  return SPEC_OK;
}

// Whether a grid of `blocks` workgroups of `threads` fits one dispatch
// (2^32 work-items).
static bool fits_dispatch(int64_t blocks, int64_t threads) { return blocks * threads <= (int64_t)UINT32_MAX; }

int verify_check(const spec_verify_args* a) {
  if (!a) return SPEC_EINVAL;
  if (a->B < 0 || a->K < 1 || a->K > SPEC_MAX_K || a->V < 1 || a->V > SPEC_MAX_V) return SPEC_EINVAL;
  if (a->dtype != SPEC_F32 && a->dtype != SPEC_BF16) return SPEC_EDTYPE;
  if (a->B == 0) return SPEC_OK;
  if (!a->target_logits || !a->draft_logits || !a->draft_tokens || !a->temperature ||
      !a->accepted_counts || !a->output_tokens || !a->workspace)
    return SPEC_EINVAL;
  if (a->t_row_stride < a->V || a->d_row_stride < a->V) return SPEC_EINVAL;
  if (a->t_req_stride != 0 && a->t_req_stride < (int64_t)(a->K + 1) * a->t_row_stride) return SPEC_EINVAL;
  if (!a->draft_row_index && a->d_req_stride != 0 && a->d_req_stride < (int64_t)a->K * a->d_row_stride)
    return SPEC_EINVAL;
  if (a->draft_row_index && a->draft_rows < 0) return SPEC_EINVAL;
  const Layout L = make_layout(a->B, a->K, a->V);
  if ((int64_t)a->B * L.R * L.C1 > INT32_MAX || (int64_t)a->B * L.nseg > INT32_MAX) return SPEC_EINVAL;
  if (!aligned16(a->workspace) || (a->draft_stats && !aligned16(a->draft_stats))) return SPEC_EALIGN;
  // position 0 always starts the first phase; bit 0 alone: dynamic early exit
  if ((a->phase_starts & 1u) && a->phase_starts != SPEC_PHASES_DYNAMIC) return SPEC_EINVAL;
  if (a->K < 63 && (a->phase_starts >> (a->K + 1)) != 0) return SPEC_EINVAL;
  if ((int64_t)a->B * (L.R * L.C1 + a->K + 1) > INT32_MAX) return SPEC_EINVAL;  // the dynamic pass's grid
  if (!verify_grids_fit(a->B, a->K, L.C1, L.nseg, a->phase_starts == SPEC_PHASES_DYNAMIC, a->draft_stats != nullptr,
                        0))
    return SPEC_EINVAL;
  if (a->workspace_bytes < L.total) return SPEC_EWORKSPACE;
  return SPEC_OK;
}

int expand_check(const spec_expand_args* a) {
  if (!a) return SPEC_EINVAL;
  if (a->B < 0 || a->K < 1 || a->H < 0 || a->N_in < 0) return SPEC_EINVAL;
  if ((int64_t)a->N_in + (int64_t)a->B * (a->K - 1) > INT32_MAX) return SPEC_EINVAL;
  if (a->B == 0) return SPEC_OK;
  if (!fits_dispatch(a->B, 256)) return SPEC_EINVAL;  // one 256-thread workgroup per request at least
  if (!a->bonus_tokens == !a->verify_output_tokens) return SPEC_EINVAL;  // exactly one bonus source
  if (!a->in_start || !a->accepted_counts || !a->out_token_ids ||
      !a->out_positions || !a->rejected_mask || !a->masked_mask || !a->new_token_indices || !a->out_start)
    return SPEC_EINVAL;
  if (a->N_in > 0 && (!a->in_token_ids || !a->in_positions || !a->hidden_map)) return SPEC_EINVAL;
  if (a->out_hidden) {
    if (a->H > 0 && (!a->mask_hidden || (a->N_in > 0 && !a->target_hidden))) return SPEC_EINVAL;
    if (a->hidden_row_stride < a->H) return SPEC_EINVAL;
  }
  if (a->slot_mapping) {
    if (a->block_size < 1 || a->max_blocks < 0 || a->bt_row_stride < a->max_blocks) return SPEC_EINVAL;
    if (a->max_blocks > 0 && !a->block_table) return SPEC_EINVAL;
  }
  return SPEC_OK;
}

size_t draft_ws_bytes(int32_t B, int32_t K, int32_t V) {
  const int64_t nseg = ((int64_t)V + kSeg - 1) / kSeg;
  return align256((size_t)B * K * nseg * sizeof(RowPartial));
}

int draft_check(const spec_draft_args* a) {
  if (!a) return SPEC_EINVAL;
  if (a->B < 0 || a->K < 1 || a->V < 1 || a->V > SPEC_MAX_V || a->N < 0) return SPEC_EINVAL;
  if (a->dtype != SPEC_F32 && a->dtype != SPEC_BF16) return SPEC_EDTYPE;
  if (a->B == 0) return SPEC_OK;
  if (!a->row_index || !a->temperature || !a->tokens || !a->workspace) return SPEC_EINVAL;
  if (a->N > 0 && !a->logits) return SPEC_EINVAL;
  if (a->row_stride < a->V) return SPEC_EINVAL;
  const int64_t nseg = ((int64_t)a->V + kSeg - 1) / kSeg;
  const int64_t C = (nseg + kDraftChunkSegs - 1) / kDraftChunkSegs;
  if ((int64_t)a->B * a->K * C > INT32_MAX) return SPEC_EINVAL;
  if (!fits_dispatch((int64_t)a->B * a->K * C, 256) || !fits_dispatch((int64_t)a->B * a->K, 64)) return SPEC_EINVAL;
  if (!aligned16(a->workspace) || (a->stats_out && !aligned16(a->stats_out))) return SPEC_EALIGN;
  if (a->workspace_bytes < draft_ws_bytes(a->B, a->K, a->V)) return SPEC_EWORKSPACE;
  return SPEC_OK;
}

size_t shard_ws_bytes(int32_t B, int32_t Vs) {
  const int64_t nseg = ((int64_t)Vs + kSeg - 1) / kSeg;
  return align256((size_t)B * sizeof(ReqDesc)) + align256((size_t)B * nseg * 2 * sizeof(double)) +
         align256((size_t)B * sizeof(int32_t));
}

// Phase p of a cut (bit k of `starts` starts a phase at position k; 0 = one
// phase): positions [lo, hi) with hi = K + 1 for the last; the number of
// phases and the start of the last.
struct PhaseRange {
  int lo, hi, count, last_lo;
};

PhaseRange phase_range(uint64_t starts, int K, int p) {
  PhaseRange r{0, K + 1, 0, 0};
  int lo = 0;
  for (int j = 0; lo <= K; ++j) {
    int hi = lo + 1;
    while (hi <= K && !((starts >> hi) & 1u)) ++hi;
    if (j == p) {
      r.lo = lo;
      r.hi = hi;
    }
    r.count = j + 1;
    r.last_lo = lo;
    lo = hi;
  }
  return r;
}

int shard_check(const spec_shard_args* a) {
  if (!a) return SPEC_EINVAL;
  if (a->B < 0 || a->K < 1 || a->K > SPEC_MAX_K || a->V < 1 || a->V > SPEC_MAX_V) return SPEC_EINVAL;
  if (a->dtype != SPEC_F32 && a->dtype != SPEC_BF16) return SPEC_EDTYPE;
  if (a->G < 1 || a->g < 0 || a->g >= a->G) return SPEC_EINVAL;
  if (a->Vs < 1 || a->v0 < 0 || (int64_t)a->v0 + a->Vs > a->V) return SPEC_EINVAL;
  if (a->B == 0) return SPEC_OK;
  if (!a->target_logits || !a->draft_logits || !a->draft_tokens || !a->temperature || !a->records ||
      !a->masses || !a->accepted_counts || !a->output_tokens || !a->workspace)
    return SPEC_EINVAL;
  if (a->t_row_stride < a->Vs || a->d_row_stride < a->Vs) return SPEC_EINVAL;
  if (a->t_req_stride != 0 && a->t_req_stride < (int64_t)(a->K + 1) * a->t_row_stride) return SPEC_EINVAL;
  if (!a->draft_row_index && a->d_req_stride != 0 && a->d_req_stride < (int64_t)a->K * a->d_row_stride)
    return SPEC_EINVAL;
  if (a->draft_row_index && a->draft_rows < 0) return SPEC_EINVAL;
  if ((int64_t)a->B * (2 * a->K + 1) > INT32_MAX) return SPEC_EINVAL;
  if (!fits_dispatch((int64_t)a->B * (2 * a->K + 1), 256) || !fits_dispatch(a->B, 1024)) return SPEC_EINVAL;
  if (a->phase_starts & 1u) return SPEC_EINVAL;  // position 0 always starts the first phase
  if (a->K < 63 && (a->phase_starts >> (a->K + 1)) != 0) return SPEC_EINVAL;
  if (a->phase < 0 || a->phase >= phase_range(a->phase_starts, a->K, 0).count) return SPEC_EINVAL;
  if (!aligned16(a->workspace)) return SPEC_EALIGN;
  if (a->workspace_bytes < shard_ws_bytes(a->B, a->Vs)) return SPEC_EWORKSPACE;
  return SPEC_OK;
}

ShardParams shard_params(const spec_shard_args* a) {
  ShardParams P;
  P.B = a->B;
  P.K = a->K;
  P.V = a->V;
  P.R = 2 * a->K + 1;
  P.G = a->G;
  P.g = a->g;
  P.v0 = a->v0;
  P.Vs = a->Vs;
  P.nseg = (int32_t)(((int64_t)a->Vs + kSeg - 1) / kSeg);
  P.target = static_cast<const char*>(a->target_logits);
  P.t_req = a->t_req_stride;
  P.t_row = a->t_row_stride;
  P.draft = static_cast<const char*>(a->draft_logits);
  P.d_req = a->d_req_stride;
  P.d_row = a->d_row_stride;
  P.tokens = a->draft_tokens;
  P.temperature = a->temperature;
  P.seed = a->seed;
  P.step = a->step;
  P.request_base = a->request_base;
  P.recs = static_cast<ShardRec*>(a->records);
  P.masses = a->masses;
  P.accepted = a->accepted_counts;
  P.out_tokens = a->output_tokens;
  char* ws = static_cast<char*>(a->workspace);
  P.desc = reinterpret_cast<ReqDesc*>(ws);
  const size_t off_seg = align256((size_t)a->B * sizeof(ReqDesc));
  P.seg = reinterpret_cast<double*>(ws + off_seg);
  P.state = reinterpret_cast<int32_t*>(ws + off_seg + align256((size_t)a->B * P.nseg * 2 * sizeof(double)));
  P.dridx = a->draft_row_index;
  P.draft_rows = a->draft_row_index ? a->draft_rows : 0;
  P.num_drafts = a->num_drafts;
  const PhaseRange ph = phase_range(a->phase_starts, a->K, a->phase);
  P.ph_lo = ph.lo;
  P.ph_nt = ph.hi - ph.lo;
  P.ph_nd = (ph.hi < a->K ? ph.hi : a->K) - ph.lo;
  P.ph_check = a->phase > 0;
  P.phased = ph.count > 1;
  P.last_lo = ph.last_lo;
  return P;
}

bool shard_vec(const spec_shard_args* a) {
  const int es = a->dtype == SPEC_BF16 ? 2 : 4;
  return aligned16(a->target_logits) && aligned16(a->draft_logits) && (a->t_row_stride * es) % 16 == 0 &&
         (a->t_req_stride * es) % 16 == 0 && (a->d_row_stride * es) % 16 == 0 &&
         (a->draft_row_index || (a->d_req_stride * es) % 16 == 0);
}

// ------------------------------------------- log probabilities, paged cache
size_t logprobs_ws_bytes(int32_t B, int32_t R, int32_t V, int32_t top) {
  const size_t segs = (size_t)B * R * (((size_t)V + kSeg - 1) / kSeg);
  return align256(segs * sizeof(LpRecord)) + (top > 0 ? align256(segs * kLpCells * sizeof(float)) : 0);
}

bool logprobs_shape_ok(int32_t B, int32_t R, int32_t V, int32_t top) {
  if (B < 0 || R < 0 || V < 1 || V > SPEC_MAX_V || top < 0 || top > SPEC_MAX_TOP) return false;
  const int64_t rows = (int64_t)B * R, nseg = ((int64_t)V + kSeg - 1) / kSeg;
  const int64_t C = (nseg + kLpChunkSegs - 1) / kLpChunkSegs;
  return rows <= INT32_MAX && rows * C <= INT32_MAX && fits_dispatch(rows * C, kThreads) && fits_dispatch(rows, 64);
}

int logprobs_check(const spec_logprobs_args* a) {
  if (!a) return SPEC_EINVAL;
  if (!logprobs_shape_ok(a->B, a->R, a->V, a->top)) return SPEC_EINVAL;
  if (a->dtype != SPEC_F32 && a->dtype != SPEC_BF16) return SPEC_EDTYPE;
  if (a->B == 0 || a->R == 0) return SPEC_OK;
  if (!a->logits || !a->tokens || !a->logprobs || !a->workspace) return SPEC_EINVAL;
  if (a->top > 0 && (!a->top_ids || !a->top_logprobs)) return SPEC_EINVAL;
  if (a->row_stride < a->V) return SPEC_EINVAL;
  if (a->req_stride != 0 && a->req_stride / a->R < a->row_stride) return SPEC_EINVAL;
  if (!aligned16(a->workspace)) return SPEC_EALIGN;
  if (a->workspace_bytes < logprobs_ws_bytes(a->B, a->R, a->V, a->top)) return SPEC_EWORKSPACE;
  return SPEC_OK;
}

bool power_of_two(int32_t x, int32_t lo, int32_t hi) { return x >= lo && x <= hi && (x & (x - 1)) == 0; }

int log2_of(int32_t x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

bool cache_shape_ok(const spec_kv_cache& c) {
  return c.num_blocks >= 1 && power_of_two(c.block_size, 16, 1024) && power_of_two(c.scale_tokens, 1, 64) &&
         c.scale_tokens <= c.block_size && c.heads >= 1 && c.heads <= 1024 && c.head_dim >= 16 && c.head_dim <= 256 &&
         c.head_dim % 16 == 0;
}

int cache_check(const spec_kv_cache& c) {
  if (!cache_shape_ok(c)) return SPEC_EINVAL;
  if (!c.k_codes || !c.v_codes || !c.k_scales || !c.v_scales) return SPEC_EINVAL;
  if (!aligned16(c.k_codes) || !aligned16(c.v_codes)) return SPEC_EALIGN;
  if (c.block_stride % 16 || c.token_stride % 16 || c.head_stride % 16) return SPEC_EALIGN;
  if (c.token_stride < c.head_dim || c.head_stride < c.head_dim) return SPEC_EINVAL;
  // 16 tokens within 32 bits for the kernels' offsets; heads within what keeps
  // the sums below far from 2^63
  constexpr int64_t kMost = (int64_t)1 << 42;
  if (c.token_stride > ((int64_t)1 << 26) || c.head_stride > kMost) return SPEC_EINVAL;
  const int64_t tokens = (int64_t)(c.block_size - 1) * c.token_stride, heads = (int64_t)(c.heads - 1) * c.head_stride;
  // heads inside a token or tokens inside a head, and a block's extent apart
  const bool heads_in = c.token_stride >= heads + c.head_dim, tokens_in = c.head_stride >= tokens + c.head_dim;
  if (!(heads_in || tokens_in || c.heads == 1)) return SPEC_EINVAL;
  if (c.num_blocks > 1 && c.block_stride < tokens + heads + c.head_dim) return SPEC_EINVAL;
  if (c.scale_head_stride < c.block_size / c.scale_tokens || c.scale_head_stride > kMost) return SPEC_EINVAL;
  if (c.scale_block_stride < c.heads * c.scale_head_stride && c.num_blocks > 1) return SPEC_EINVAL;
  return SPEC_OK;
}

CacheView cache_view(const spec_kv_cache& c) {
  CacheView v;
  v.num_blocks = c.num_blocks;
  v.heads = c.heads;
  v.dim = c.head_dim;
  v.bs_shift = log2_of(c.block_size);
  v.st_shift = log2_of(c.scale_tokens);
  v.codes[0] = c.k_codes;
  v.codes[1] = c.v_codes;
  v.scales[0] = c.k_scales;
  v.scales[1] = c.v_scales;
  v.block = c.block_stride;
  v.token = c.token_stride;
  v.head = c.head_stride;
  v.sblock = c.scale_block_stride;
  v.shead = c.scale_head_stride;
  return v;
}

int kv_write_check(const spec_kv_write_args* a) {
  if (!a || a->N < 0) return SPEC_EINVAL;
  if (a->dtype != SPEC_F32 && a->dtype != SPEC_BF16) return SPEC_EDTYPE;
  const int rc = cache_check(a->cache);
  if (rc != SPEC_OK) return rc;
  if (a->N == 0) return SPEC_OK;
  if (!a->key || !a->value || !a->slots) return SPEC_EINVAL;
  if (a->k_token_stride < 0 || a->k_head_stride < 0 || a->v_token_stride < 0 || a->v_head_stride < 0)
    return SPEC_EINVAL;
  const int64_t chunk = kv_write_chunk(a->N);
  if (!fits_dispatch(((int64_t)a->N + chunk - 1) / chunk * ((2 * a->cache.heads + 3) / 4), kThreads))
    return SPEC_EINVAL;
  // keys and values are written by different waves
  if (a->cache.k_codes == a->cache.v_codes || a->cache.k_scales == a->cache.v_scales) return SPEC_EINVAL;
  return SPEC_OK;
}

int kv_read_check(const spec_kv_read_args* a) {
  if (!a || a->N < 0) return SPEC_EINVAL;
  if (a->dtype != SPEC_F32 && a->dtype != SPEC_BF16) return SPEC_EDTYPE;
  const int rc = cache_check(a->cache);
  if (rc != SPEC_OK) return rc;
  if (a->N == 0) return SPEC_OK;
  if (!a->key || !a->value || !a->slots) return SPEC_EINVAL;
  const int64_t per = kv_read_per(a->N, a->cache.heads, a->cache.head_dim);
  if (!fits_dispatch(((int64_t)a->N + per - 1) / per, kThreads)) return SPEC_EINVAL;
  return SPEC_OK;
}

// ------------------------------------------------ sampling, 4-bit cache, rotation
size_t cut_ws_bytes(int32_t B, int32_t R, int32_t V) {
  const size_t rows = (size_t)B * R;
  return align256(rows * sizeof(uint64_t)) + rows * cut_split_row(cut_parts((int64_t)rows, V, 4));
}

bool cut_shape_ok(int32_t B, int32_t R, int32_t V) {
  if (B < 0 || R < 0 || V < 1 || V > SPEC_MAX_V) return false;
  const int64_t rows = (int64_t)B * R;
  if (rows > INT32_MAX) return false;
  const int64_t chunk = cut_chunk(rows, V), C = ((int64_t)V + chunk - 1) / chunk;
  return rows * C <= INT32_MAX && fits_dispatch(rows * C, kThreads) && fits_dispatch(rows, 1024);
}

// The sizes, settings and workspace that a sampling and a truncation share.
// rowless: the logits have no rows (every entry of the row table is outside them).
template <class Args>
int cut_check(const Args* a, bool rowless) {
  if (!a || !cut_shape_ok(a->B, a->R, a->V)) return SPEC_EINVAL;
  if (a->dtype != SPEC_F32 && a->dtype != SPEC_BF16) return SPEC_EDTYPE;
  if (a->B == 0 || a->R == 0) return SPEC_OK;
  if ((!a->logits && !rowless) || !a->temperature || !a->workspace) return SPEC_EINVAL;
  if (a->row_stride < a->V) return SPEC_EINVAL;
  if (!aligned16(a->workspace)) return SPEC_EALIGN;
  if (a->workspace_bytes < cut_ws_bytes(a->B, a->R, a->V)) return SPEC_EWORKSPACE;
  return SPEC_OK;
}

template <class Args>
CutParams cut_params(const Args* a) {
  CutParams P = {};
  P.B = a->B;
  P.R = a->R;
  P.V = a->V;
  P.chunk = cut_chunk((int64_t)a->B * a->R, a->V);
  P.C = (int32_t)(((int64_t)a->V + P.chunk - 1) / P.chunk);
  while (((int64_t)1 << P.ibits) < a->V) ++P.ibits;
  // V weights of at most 2^frac within 63 bits, eight within the 52 of a double
  int bits = P.ibits;
  if (((int64_t)1 << bits) == a->V) ++bits;
  P.frac = 63 - bits < 48 ? 63 - bits : 48;
  P.by_C = FastDiv::by((uint32_t)P.C);
  P.by_R = FastDiv::by((uint32_t)P.R);
  P.logits = static_cast<const char*>(a->logits);
  P.req = a->req_stride;
  P.row = a->row_stride;
  P.temperature = a->temperature;
  P.top_k = a->top_k;
  P.top_p = a->top_p;
  P.min_p = a->min_p;
  P.last = static_cast<uint64_t*>(a->workspace);
  const size_t rows = (size_t)a->B * a->R;
  P.parts = cut_parts((int64_t)rows, a->V, a->dtype == SPEC_BF16 ? 2 : 4);
  if (P.parts > 1) {  // (whole ranges of indices to a part)
    const int64_t range = (int64_t)1 << (P.ibits > kCutRangeBits ? P.ibits - kCutRangeBits : 0);
    const int64_t ranges = (a->V + range - 1) / range;
    P.seg = (int32_t)((ranges + P.parts - 1) / P.parts * range);
    P.split_row = (int64_t)cut_split_row(P.parts);
    P.parts = (int32_t)(((int64_t)a->V + P.seg - 1) / P.seg);
    P.split = static_cast<char*>(a->workspace) + align256(rows * sizeof(uint64_t));
  }
  return P;
}

int cache4_check(const spec_kv4_cache& c) {
  if (c.num_blocks < 1 || !power_of_two(c.block_size, 16, 1024) || c.heads < 1 || c.heads > 1024 || c.head_dim < 32 ||
      c.head_dim > 256 || c.head_dim % 32)
    return SPEC_EINVAL;
  if (!c.k_codes || !c.v_codes || !c.k_scales || !c.v_scales) return SPEC_EINVAL;
  if (!aligned16(c.k_codes) || !aligned16(c.v_codes)) return SPEC_EALIGN;
  if (c.block_stride % 16 || c.token_stride % 16 || c.head_stride % 16) return SPEC_EALIGN;
  const int64_t bytes = c.head_dim / 2;
  constexpr int64_t kMost = (int64_t)1 << 42;  // (as for 8 bits)
  if (c.token_stride < bytes || c.head_stride < bytes) return SPEC_EINVAL;
  if (c.token_stride > ((int64_t)1 << 26) || c.head_stride > kMost) return SPEC_EINVAL;
  const int64_t tokens = (int64_t)(c.block_size - 1) * c.token_stride, heads = (int64_t)(c.heads - 1) * c.head_stride;
  const bool heads_in = c.token_stride >= heads + bytes, tokens_in = c.head_stride >= tokens + bytes;
  if (!(heads_in || tokens_in || c.heads == 1)) return SPEC_EINVAL;
  if (c.num_blocks > 1 && c.block_stride < tokens + heads + bytes) return SPEC_EINVAL;
  if (c.scale_head_stride < (int64_t)(c.head_dim / 32) * c.block_size || c.scale_head_stride > kMost) return SPEC_EINVAL;
  if (c.scale_block_stride < c.heads * c.scale_head_stride && c.num_blocks > 1) return SPEC_EINVAL;
  return SPEC_OK;
}

CacheView cache4_view(const spec_kv4_cache& c) {
  CacheView v;
  v.num_blocks = c.num_blocks;
  v.heads = c.heads;
  v.dim = c.head_dim;
  v.bs_shift = log2_of(c.block_size);
  v.st_shift = 0;
  v.codes[0] = c.k_codes;
  v.codes[1] = c.v_codes;
  v.scales[0] = c.k_scales;
  v.scales[1] = c.v_scales;
  v.block = c.block_stride;
  v.token = c.token_stride;
  v.head = c.head_stride;
  v.sblock = c.scale_block_stride;
  v.shead = c.scale_head_stride;
  return v;
}

// One rotated tensor: its input and output.  Lanes write the output in no order,
// and others read.
bool turned_ok(const void* in, int64_t tok, int64_t head, const void* out, int64_t out_tok, int64_t out_head, int32_t N,
               int32_t heads, int32_t dim, int64_t es) {
  if (!in || !out || tok < 0 || head < 0 || out_tok < 0 || out_head < 0) return false;
  const MemRows to = mem_rows(out, N, out_tok, heads, out_head, dim, es);
  if (rows_share(to)) return false;
  return in == out ? tok == out_tok && head == out_head : !rows_meet(mem_rows(in, N, tok, heads, head, dim, es), to);
}

// How the tokens and heads of a rotation are shared out; false: too many.
bool rope_split(RopeParams& P) {
  const int64_t per = kThreads / ((P.dim + 15) / 16), heads = (int64_t)P.heads[0] + (P.write ? 2 : 1) * (int64_t)P.heads[1];
  const int64_t rounds = (heads + per - 1) / per;
  P.by_heads = FastDiv::by((uint32_t)heads);
  // many tokens: as many to a workgroup as its lanes work out angles for; few:
  // one, its heads shared out.  Few against many, us, on both sides of the border
  // (72 = 64 + 8 heads, 40 = 32 + 8):
  //   bf16, 4000, 8000, 16000 tokens  72 heads of 64    19.5 17.1   33.9 28.7   63.7 58.6
  //                                   40 heads of 128   18.4 16.5   32.9 30.8   62.3 52.4
  //                                   32 heads of 96    13.6 13.9   20.2 22.8   37.2 40.5
  //   fp32                            72 heads of 64    29.2 27.6   55.2 52.4   111 115
  //                                   40 heads of 128   32.0 31.9   61.5 61.5   119 132
  // A small rotated part makes few workgroups of many tokens (72 heads of 192 of which
  // 32 dims are rotated, bf16: 40.5 62.5 for 4000 tokens, 76.9 79.1 for 8000), and large
  // fp32 batches lose as well: no border on the tokens alone suits all.
  const bool many = (int64_t)P.N * rounds >= 16384;
  P.tokens = !many ? 1 : P.half > 0 ? kRopeAngles / P.half : 8;
  P.shares = many ? 1 : (int32_t)rounds;
  return fits_dispatch((((int64_t)P.N + P.tokens - 1) / P.tokens) * P.shares, kThreads);
}

int rope_check(const spec_rope_args* a, RopeParams& P) {
  if (!a || a->N < 0 || a->q_heads < 0 || a->q_heads > 1024 || a->k_heads < 0 || a->k_heads > 1024) return SPEC_EINVAL;
  if (a->head_dim < 8 || a->head_dim > 256 || a->head_dim % 8) return SPEC_EINVAL;
  if (a->rot_dim < 16 || a->rot_dim > a->head_dim || a->rot_dim % 16) return SPEC_EINVAL;
  if (a->dtype != SPEC_F32 && a->dtype != SPEC_BF16) return SPEC_EDTYPE;
  if (!(fabs(a->scale) <= DBL_MAX)) return SPEC_EINVAL;
  if (a->N == 0 || a->q_heads + a->k_heads == 0) return SPEC_OK;
  if (!a->inv_freq || !a->positions) return SPEC_EINVAL;
  const int64_t es = a->dtype == SPEC_BF16 ? 2 : 4;
  const bool q = a->q_heads > 0, k = a->k_heads > 0;
  if (q && !turned_ok(a->q, a->q_token_stride, a->q_head_stride, a->q_out, a->q_out_token_stride, a->q_out_head_stride,
                      a->N, a->q_heads, a->head_dim, es))
    return SPEC_EINVAL;
  if (k && !turned_ok(a->k, a->k_token_stride, a->k_head_stride, a->k_out, a->k_out_token_stride, a->k_out_head_stride,
                      a->N, a->k_heads, a->head_dim, es))
    return SPEC_EINVAL;
  if (q && k) {
    const MemRows qo = mem_rows(a->q_out, a->N, a->q_out_token_stride, a->q_heads, a->q_out_head_stride, a->head_dim, es),
                  ko = mem_rows(a->k_out, a->N, a->k_out_token_stride, a->k_heads, a->k_out_head_stride, a->head_dim, es);
    if (rows_meet(qo, ko) ||
        (a->k != a->k_out &&
         rows_meet(mem_rows(a->k, a->N, a->k_token_stride, a->k_heads, a->k_head_stride, a->head_dim, es), qo)) ||
        (a->q != a->q_out &&
         rows_meet(mem_rows(a->q, a->N, a->q_token_stride, a->q_heads, a->q_head_stride, a->head_dim, es), ko)))
      return SPEC_EINVAL;
  }
  P = {};
  P.N = a->N;
  P.heads[0] = a->q_heads;
  P.heads[1] = a->k_heads;
  P.dim = a->head_dim;
  P.half = a->rot_dim / 2;
  P.inter = a->interleaved != 0;
  P.positions = a->positions;
  P.wide = a->wide_positions != 0;
  P.inv_freq = a->inv_freq;
  P.scale = a->scale;
  P.src[0] = static_cast<const char*>(a->q);
  P.tok[0] = a->q_token_stride;
  P.hd[0] = a->q_head_stride;
  P.src[1] = static_cast<const char*>(a->k);
  P.tok[1] = a->k_token_stride;
  P.hd[1] = a->k_head_stride;
  P.dst[0] = static_cast<char*>(a->q_out);
  P.dtok[0] = a->q_out_token_stride;
  P.dhd[0] = a->q_out_head_stride;
  P.dst[1] = static_cast<char*>(a->k_out);
  P.dtok[1] = a->k_out_token_stride;
  P.dhd[1] = a->k_out_head_stride;
  return rope_split(P) ? SPEC_OK : SPEC_EINVAL;
}

int kv4_write_check(const spec_kv4_write_args* a, RopeParams& P) {
  if (!a || a->N < 0) return SPEC_EINVAL;
  if (a->dtype != SPEC_F32 && a->dtype != SPEC_BF16) return SPEC_EDTYPE;
  const int rc = cache4_check(a->cache);
  if (rc != SPEC_OK) return rc;
  if (a->rot_dim < 0 || a->rot_dim > a->cache.head_dim || a->rot_dim % 16) return SPEC_EINVAL;
  if (a->q_heads < 0 || a->q_heads > 1024 || (a->q_heads > 0 && a->rot_dim == 0)) return SPEC_EINVAL;
  if (a->rot_dim > 0 && !(fabs(a->scale) <= DBL_MAX)) return SPEC_EINVAL;
  // keys and values are written by different lanes
  if (a->cache.k_codes == a->cache.v_codes || a->cache.k_scales == a->cache.v_scales) return SPEC_EINVAL;
  if (a->N == 0) return SPEC_OK;
  if (!a->key || !a->value || !a->slots) return SPEC_EINVAL;
  if (a->k_token_stride < 0 || a->k_head_stride < 0 || a->v_token_stride < 0 || a->v_head_stride < 0)
    return SPEC_EINVAL;
  if (a->rot_dim > 0 && (!a->inv_freq || !a->positions)) return SPEC_EINVAL;
  if (a->q_heads > 0) {
    const int64_t es = a->dtype == SPEC_BF16 ? 2 : 4;
    const int32_t heads = a->cache.heads, dim = a->cache.head_dim;
    if (!turned_ok(a->q, a->q_token_stride, a->q_head_stride, a->q_out, a->q_out_token_stride, a->q_out_head_stride,
                   a->N, a->q_heads, dim, es))
      return SPEC_EINVAL;
    const MemRows qo = mem_rows(a->q_out, a->N, a->q_out_token_stride, a->q_heads, a->q_out_head_stride, dim, es);
    if (rows_meet(mem_rows(a->key, a->N, a->k_token_stride, heads, a->k_head_stride, dim, es), qo) ||
        rows_meet(mem_rows(a->value, a->N, a->v_token_stride, heads, a->v_head_stride, dim, es), qo))
      return SPEC_EINVAL;
  }
  P = {};
  P.c = cache4_view(a->cache);
  P.N = a->N;
  P.heads[0] = a->q_heads;
  P.heads[1] = a->cache.heads;
  P.dim = a->cache.head_dim;
  P.half = a->rot_dim / 2;
  P.inter = a->interleaved != 0;
  P.write = 1;
  P.positions = a->positions;
  P.wide = a->wide_positions != 0;
  P.inv_freq = a->inv_freq;
  P.scale = a->scale;
  P.src[0] = static_cast<const char*>(a->q);
  P.tok[0] = a->q_token_stride;
  P.hd[0] = a->q_head_stride;
  P.src[1] = static_cast<const char*>(a->key);
  P.tok[1] = a->k_token_stride;
  P.hd[1] = a->k_head_stride;
  P.src[2] = static_cast<const char*>(a->value);
  P.tok[2] = a->v_token_stride;
  P.hd[2] = a->v_head_stride;
  P.dst[0] = static_cast<char*>(a->q_out);
  P.dtok[0] = a->q_out_token_stride;
  P.dhd[0] = a->q_out_head_stride;
  P.slots = a->slots;
  return rope_split(P) ? SPEC_OK : SPEC_EINVAL;
}

int kv4_read_check(const spec_kv4_read_args* a) {
  if (!a || a->N < 0) return SPEC_EINVAL;
  if (a->dtype != SPEC_F32 && a->dtype != SPEC_BF16) return SPEC_EDTYPE;
  const int rc = cache4_check(a->cache);
  if (rc != SPEC_OK) return rc;
  if (a->N == 0) return SPEC_OK;
  if (!a->key || !a->value || !a->slots) return SPEC_EINVAL;
  const int64_t per = kv_read_per(a->N, a->cache.heads, a->cache.head_dim);
  if (!fits_dispatch(((int64_t)a->N + per - 1) / per, kThreads)) return SPEC_EINVAL;
  return SPEC_OK;
}

bool attn_sizes_ok(const spec_attn_args* a) {
  if (a->B < 0 || a->N < 0 || a->max_q < 1 || a->max_q > (1 << 24) || a->max_ctx < 0 || a->max_ctx > (1 << 30) ||
      a->window < 0)
    return false;
  const spec_kv_cache& c = a->cache;
  if (c.heads < 1 || c.heads > 1024 || c.head_dim < 16 || c.head_dim > 256 || c.head_dim % 16) return false;
  if (a->q_heads < c.heads || a->q_heads % c.heads || a->q_heads / c.heads > 64) return false;
  return (int64_t)a->B * c.heads <= INT32_MAX;  // (times the blocks of rows, at most 2^26, within 64 bits)
}

AttnPlan attn_plan(const spec_attn_args* a, bool four) {
  return plan_attn(a->B, a->q_heads / a->cache.heads, a->cache.heads, a->cache.head_dim, a->max_q, a->max_ctx,
                   a->window, a->cache.head_stride < a->cache.token_stride, four);
}

size_t attn_ws_bytes(const spec_attn_args* a, const AttnPlan& p) {
  if (p.chunks == 0 || a->B == 0) return 0;
  const size_t parts = (size_t)p.chunks * 2 * a->cache.heads * 16 * p.rt;
  return align256(parts * a->cache.head_dim * sizeof(float)) + align256(parts * sizeof(float2)) +
         align256((size_t)a->B * p.nrb * sizeof(int2));
}

// cache_rc: what the check of the cache says.
int attn_check(const spec_attn_args* a, int cache_rc, bool four, AttnPlan& plan) {
  if (!attn_sizes_ok(a)) return SPEC_EINVAL;
  if (a->dtype != SPEC_BF16) return SPEC_EDTYPE;
  if (cache_rc != SPEC_OK) return cache_rc;
  if (!(fabsf(a->scale) <= FLT_MAX / 1.4427f)) return SPEC_EINVAL;  // (the kernel takes scale * log2(e))
  if (a->max_blocks < 0 || a->bt_row_stride < a->max_blocks) return SPEC_EINVAL;
  if (a->B == 0 || a->N == 0) return SPEC_OK;
  if (!a->q || !a->q_start || !a->ctx_len || !a->out) return SPEC_EINVAL;
  if (a->max_blocks > 0 && !a->block_table) return SPEC_EINVAL;
  if (a->q_token_stride < 0 || a->q_head_stride < 0) return SPEC_EINVAL;
  if (!aligned16(a->out)) return SPEC_EALIGN;
  plan = attn_plan(a, four);
  const int64_t grid = (int64_t)a->B * a->cache.heads * plan.nrb;
  if (grid > INT32_MAX || !fits_dispatch((plan.groups + 7) / 8 * 8 * plan.items, kThreads) ||
      (plan.chunks > 0 && !fits_dispatch(grid * plan.rt, kThreads)))
    return SPEC_EINVAL;
  const size_t need = attn_ws_bytes(a, plan);
  if (need > 0) {
    if (!a->workspace) return SPEC_EINVAL;
    if (!aligned16(a->workspace)) return SPEC_EALIGN;
    if (a->workspace_bytes < need) return SPEC_EWORKSPACE;
  }
  return SPEC_OK;
}

int attn_launch(const spec_attn_args* a, const AttnPlan& plan, const CacheView& view, bool four, hipStream_t stream);

// An attention over the 4-bit cache as one over a cache of 8 bits: what is not
// the cache, and of the cache what its plan reads.
spec_attn_args attn_of(const spec_attn4_args* a) {
  spec_attn_args b = {};
  b.cache.num_blocks = a->cache.num_blocks;
  b.cache.block_size = a->cache.block_size;
  b.cache.scale_tokens = 1;
  b.cache.heads = a->cache.heads;
  b.cache.head_dim = a->cache.head_dim;
  b.cache.token_stride = a->cache.token_stride;
  b.cache.head_stride = a->cache.head_stride;
  b.B = a->B;
  b.N = a->N;
  b.q_heads = a->q_heads;
  b.max_q = a->max_q;
  b.max_ctx = a->max_ctx;
  b.window = a->window;
  b.dtype = a->dtype;
  b.scale = a->scale;
  b.q = a->q;
  b.q_token_stride = a->q_token_stride;
  b.q_head_stride = a->q_head_stride;
  b.q_start = a->q_start;
  b.ctx_len = a->ctx_len;
  b.block_table = a->block_table;
  b.bt_row_stride = a->bt_row_stride;
  b.max_blocks = a->max_blocks;
  b.sinks = a->sinks;
  b.out = a->out;
  b.lse = a->lse;
  b.workspace = a->workspace;
  b.workspace_bytes = a->workspace_bytes;
  return b;
}

}  // namespace

extern "C" {

size_t spec_shard_workspace_bytes(int32_t B, int32_t K, int32_t Vs) {
  if (B < 0 || K < 1 || K > SPEC_MAX_K || Vs < 1 || Vs > SPEC_MAX_V) return 0;
  return shard_ws_bytes(B, Vs);
}

int spec_shard_stats_launch(const spec_shard_args* a, hipStream_t stream) {
  const int rc = shard_check(a);
  if (rc != SPEC_OK || a->B == 0) return rc;
  return launch_shard_stats(shard_params(a), a->dtype, shard_vec(a), stream) == hipSuccess ? SPEC_OK : SPEC_ELAUNCH;
}

int spec_shard_phase_launch(const spec_shard_args* a, hipStream_t stream) {
  if (!a || a->K < 1 || a->K > SPEC_MAX_K) return SPEC_EINVAL;
  if (a->phase >= phase_range(a->phase_starts, a->K, 0).count - 1) return SPEC_EINVAL;  // not the last phase
  const int rc = shard_check(a);
  if (rc != SPEC_OK) return rc;
  if (a->B == 0) return SPEC_OK;
  return launch_shard_phase(shard_params(a), a->dtype, shard_vec(a), stream) == hipSuccess ? SPEC_OK : SPEC_ELAUNCH;
}

int spec_shard_decide_launch(const spec_shard_args* a, hipStream_t stream) {
  const int rc = shard_check(a);
  if (rc != SPEC_OK || a->B == 0) return rc;
  return launch_shard_decide(shard_params(a), a->dtype, shard_vec(a), stream) == hipSuccess ? SPEC_OK
                                                                                            : SPEC_ELAUNCH;
}

int spec_shard_draw_launch(const spec_shard_args* a, hipStream_t stream) {
  const int rc = shard_check(a);
  if (rc != SPEC_OK || a->B == 0) return rc;
  return launch_shard_draw(shard_params(a), a->dtype, shard_vec(a), stream) == hipSuccess ? SPEC_OK : SPEC_ELAUNCH;
}

size_t spec_draft_workspace_bytes(int32_t B, int32_t K, int32_t V) {
  if (B < 0 || K < 1 || V < 1 || V > SPEC_MAX_V) return 0;
  return draft_ws_bytes(B, K, V);
}

int spec_draft_sample_launch(const spec_draft_args* a, hipStream_t stream) {
  const int rc = draft_check(a);
  if (rc != SPEC_OK || a->B == 0) return rc;
  const int es = a->dtype == SPEC_BF16 ? 2 : 4;
  DraftParams P;
  P.B = a->B;
  P.K = a->K;
  P.V = a->V;
  P.N = a->N;
  P.nseg = (int32_t)(((int64_t)a->V + kSeg - 1) / kSeg);
  P.C = (P.nseg + kDraftChunkSegs - 1) / kDraftChunkSegs;
  P.logits = static_cast<const char*>(a->logits);
  P.row_stride = a->row_stride;
  P.row_index = a->row_index;
  P.temperature = a->temperature;
  P.seed = a->seed;
  P.step = a->step;
  P.request_base = a->request_base;
  P.tokens = a->tokens;
  P.segp = static_cast<RowPartial*>(a->workspace);
  P.stats = static_cast<RowPartial*>(a->stats_out);
  const bool vec = aligned16(a->logits) && (a->row_stride * es) % 16 == 0;
  return launch_draft(P, a->dtype, vec, stream) == hipSuccess ? SPEC_OK : SPEC_ELAUNCH;
}

uint64_t spec_verify_plan_phases(int32_t K, const double* survival, double sampled_fraction, double phase_cost) {
  if (K < 1 || K > SPEC_MAX_K || !survival) return 0;
  if (!(sampled_fraction >= 0.0 && sampled_fraction <= 1.0) || !(phase_cost >= 0.0 && phase_cost < 1e300)) return 0;
  for (int k = 0; k <= K; ++k)
    if (!(survival[k] >= 0.0 && survival[k] <= 1.0)) return 0;
  // best[s]: least expected cost of positions s..K when a phase starts at s
  double best[SPEC_MAX_K + 2];
  int next[SPEC_MAX_K + 2];
  best[K + 1] = 0.0;
  for (int s = K; s >= 0; --s) {
    best[s] = -1.0;
    for (int e = K + 1; e > s; --e) {
      const double rows = (double)(e - s) + sampled_fraction * (double)((e < K ? e : K) - s);
      const double c = survival[s] * rows + (e <= K ? phase_cost : 0.0) + best[e];
      if (best[s] < 0.0 || c < best[s]) {  // ties keep the longer phase, found first
        best[s] = c;
        next[s] = e;
      }
    }
  }
  uint64_t mask = 0;
  for (int s = next[0]; s <= K; s = next[s]) mask |= (uint64_t)1 << s;
  return mask;
}

double spec_verify_phase_cost(int32_t B, int32_t K, int32_t V, int32_t dtype) {
  if (B < 1 || K < 1 || K > SPEC_MAX_K || V < 1 || V > SPEC_MAX_V) return -1.0;
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return -1.0;
  // measured on MI355X (see the header): the boundary's fixed cost, the extra
  // when a phase's rows cannot fill the chip, the slots of the row pass
  // (256 compute units x 5 resident 256-thread workgroups) and its rate
  constexpr double kBoundaryUs = 12.0, kUnderfillUs = 7.7, kSlots = 256.0 * 5.0, kRowBytesPerUs = 6.8e6;
  const Layout L = make_layout(1, K, V);
  const double per_row_unit = (double)B * (double)L.C1;  // workgroups reading one row of every request
  const double fill = per_row_unit < kSlots ? 1.0 - per_row_unit / kSlots : 0.0;
  const double boundary_us = kBoundaryUs + kUnderfillUs * fill;
  const double row_us = (double)B * (double)V * (dtype == SPEC_BF16 ? 2.0 : 4.0) / kRowBytesPerUs;
  return boundary_us / row_us;
}

size_t spec_verify_workspace_bytes(int32_t B, int32_t K, int32_t V) {
  if (B < 0 || K < 1 || K > SPEC_MAX_K || V < 1 || V > SPEC_MAX_V) return 0;
  return make_layout(B, K, V).total;
}

// The kernel parameters of a checked verification (B >= 1); vec: 16-byte
// row loads are possible.
static VerifyParams verify_params(const spec_verify_args* a, bool& vec) {
  const Layout L = make_layout(a->B, a->K, a->V);
  const int es = a->dtype == SPEC_BF16 ? 2 : 4;
  VerifyParams P;
  P.B = a->B;
  P.K = a->K;
  P.V = a->V;
  P.R = L.R;
  P.C1 = L.C1;
  P.chunk1 = L.chunk1;
  P.nseg = L.nseg;
  P.target = static_cast<const char*>(a->target_logits);
  P.t_req = a->t_req_stride;
  P.t_row = a->t_row_stride;
  P.draft = static_cast<const char*>(a->draft_logits);
  P.d_req = a->d_req_stride;
  P.d_row = a->d_row_stride;
  P.dridx = a->draft_row_index;
  P.num_drafts = a->num_drafts;
  P.dstats = static_cast<const RowPartial*>(a->draft_stats);
  P.draft_rows = a->draft_row_index ? a->draft_rows : 0;
  P.tokens = a->draft_tokens;
  P.temperature = a->temperature;
  P.seed = a->seed;
  P.step = a->step;
  P.request_base = a->request_base;
  P.accepted = a->accepted_counts;
  P.out_tokens = a->output_tokens;
  P.debug = a->debug_probs;
  char* ws = static_cast<char*>(a->workspace);
  P.rowp = reinterpret_cast<RowPartial*>(ws + L.off_rowp);
  P.desc = reinterpret_cast<ReqDesc*>(ws + L.off_desc);
  P.seg = reinterpret_cast<double*>(ws + L.off_seg);
  vec = aligned16(a->target_logits) && aligned16(a->draft_logits) && (a->t_row_stride * es) % 16 == 0 &&
        (a->t_req_stride * es) % 16 == 0 && (a->d_row_stride * es) % 16 == 0 &&
        (a->draft_row_index || (a->d_req_stride * es) % 16 == 0);
  P.err = reinterpret_cast<int32_t*>(ws + L.off_err);
  P.state = reinterpret_cast<int32_t*>(ws + L.off_state);
  P.epoch = reinterpret_cast<uint64_t*>(ws + L.off_epoch);
  // A workspace's launches are tagged by its counter plus this salt, from the
  // workspace's address and the number of this call in the process, which no
  // leftover memory can repeat: of a workspace allocated again at the same
  // address the counter may hold a value that an earlier launch ran at, whose
  // records still stand (in a test of that, 110 of 192 requests invalid without
  // the call's number).  Replays of a captured call share its number and differ
  // in the counter.  2^64 over the golden ratio and over the root of two: d
  // times either stays 2^64 / (3 d) away from 0, so that small differences of
  // the address or the number do not cancel against the counter's.
  static std::atomic<uint64_t> calls{0};
  P.salt = (uint64_t)(uintptr_t)a->workspace * 0x9E3779B97F4A7C15ull +
           (calls.fetch_add(1, std::memory_order_relaxed) + 1) * 0xB504F333F9DE6485ull;
  P.dstate = reinterpret_cast<uint64_t*>(ws + L.off_dstate);
  P.trec = reinterpret_cast<TaggedPartial*>(ws + L.off_trec);
  P.dyn = a->phase_starts == SPEC_PHASES_DYNAMIC;
  // a request's decider slot sits this many request groups after its chunks
  P.dyn_shift = (int32_t)min((int64_t)a->B - 1, (int64_t)a->B * kDynShiftNum / kDynShiftDen);
  P.ph_lo = P.ph_nt = P.ph_nd = P.ph_rd = P.ph_check = 0;
  P.last_lo = P.phased = 0;
  P.ex_on = 0;
  P.ex_G = 1;
  return P;
}

static int verify_enqueue(const VerifyParams& P, const spec_verify_args* a, bool vec, hipStream_t stream) {
  return launch_verify(P, a->dtype, vec, a->phase_starts, static_cast<hipEvent_t>(a->phase_event), stream) ==
                 hipSuccess
             ? SPEC_OK
             : SPEC_ELAUNCH;
}

int spec_verify_launch(const spec_verify_args* a, hipStream_t stream) {
  const int rc = verify_check(a);
  if (rc != SPEC_OK || a->B == 0) return rc;
  bool vec;
  const VerifyParams P = verify_params(a, vec);
  return verify_enqueue(P, a, vec, stream);
}

int spec_verify_launch_noalloc(const spec_verify_args* a, hipStream_t stream) {
  if (!a) return SPEC_EINVAL;
  if (a->B < 0 || a->K < 1 || a->K > SPEC_MAX_K || a->V < 1 || a->V > SPEC_MAX_V) return SPEC_EINVAL;
  if (a->B == 0) return verify_check(a);  // nothing to enqueue (a bad dtype is still reported)
  if (make_layout(a->B, a->K, a->V).total > (size_t)SPEC_NOALLOC_SCRATCH_BYTES) return SPEC_EWORKSPACE;
  void* ws = nullptr;
  const int rs = scratch_address(stream, &ws);
  if (rs != SPEC_OK) return rs;
  // the same checks and kernels as spec_verify_launch, with this device's
  // scratch array as the workspace
  spec_verify_args b = *a;
  b.workspace = ws;
  b.workspace_bytes = SPEC_NOALLOC_SCRATCH_BYTES;
  const int rc = verify_check(&b);
  if (rc != SPEC_OK) return rc;
  bool vec;
  const VerifyParams P = verify_params(&b, vec);
  return verify_enqueue(P, &b, vec, stream);
}

// The kernel parameters of a checked expansion (B >= 1), G workgroups per
// request window.
static ExpandParams expand_params(const spec_expand_args* a, bool hidden_only, int64_t rows_per_wg) {
  ExpandParams P;
  P.hidden_only = hidden_only ? 1 : 0;
  P.B = a->B;
  P.K = a->K;
  P.H = a->H;
  P.N_in = a->N_in;
  P.mask_id = a->mask_token_id;
  // about rows_per_wg output rows per workgroup on average; a request's
  // window is shared by G workgroups row-interleaved
  const int64_t n_out = (int64_t)a->N_in + (int64_t)a->B * (a->K - 1);
  const int64_t avg_window = (n_out + a->B - 1) / a->B;
  int64_t G = (avg_window + rows_per_wg - 1) / rows_per_wg;
  if (G < 1) G = 1;
  if (G > 64) G = 64;
  if ((int64_t)a->B * G > INT32_MAX || !fits_dispatch((int64_t)a->B * G, 256)) G = 1;
  P.G = (int32_t)G;
  P.ids = a->in_token_ids;
  P.pos = a->in_positions;
  P.in_start = a->in_start;
  P.acc = a->accepted_counts;
  P.bonus = a->bonus_tokens;
  P.vtok = a->verify_output_tokens;
  P.th = a->target_hidden;
  P.th_stride = a->hidden_row_stride;
  P.mh = a->mask_hidden;
  P.out_ids = a->out_token_ids;
  P.out_pos = a->out_positions;
  P.rej = a->rejected_mask;
  P.msk = a->masked_mask;
  P.nti = a->new_token_indices;
  P.hmap = a->hidden_map;
  P.out_start = a->out_start;
  P.out_h = (a->H > 0) ? a->out_hidden : nullptr;
  P.slots = a->slot_mapping;
  P.bt = a->block_table;
  P.bt_stride = a->bt_row_stride;
  P.max_blocks = a->slot_mapping ? a->max_blocks : 0;
  P.block_size = a->slot_mapping ? a->block_size : 1;
  P.vec = (a->H % 8) == 0 && (a->hidden_row_stride % 8) == 0 && aligned16(a->target_hidden) &&
          aligned16(a->mask_hidden) && aligned16(a->out_hidden);
  return P;
}

static int expand_launch(const spec_expand_args* a, bool hidden_only, hipStream_t stream) {
  const ExpandParams P = expand_params(a, hidden_only, kExpandRowsPerWG);
  return launch_expand(P, P.vec != 0, stream) == hipSuccess ? SPEC_OK : SPEC_ELAUNCH;
}

int spec_expand_launch(const spec_expand_args* a, hipStream_t stream) {
  const int rc = expand_check(a);
  if (rc != SPEC_OK || a->B == 0) return rc;
  return expand_launch(a, false, stream);
}

int spec_expand_hidden_launch(const spec_expand_args* a, hipStream_t stream) {
  if (!a) return SPEC_EINVAL;
  if (a->B < 0 || a->K < 1 || a->H < 0 || a->N_in < 0) return SPEC_EINVAL;
  if ((int64_t)a->N_in + (int64_t)a->B * (a->K - 1) > INT32_MAX) return SPEC_EINVAL;
  if (a->B == 0 || a->H == 0) return SPEC_OK;
  if (!a->in_start || !a->out_hidden || !a->mask_hidden || (a->N_in > 0 && !a->target_hidden))
    return SPEC_EINVAL;
  if (a->hidden_row_stride < a->H) return SPEC_EINVAL;
  return expand_launch(a, true, stream);
}

int spec_verify_expand_launch(const spec_verify_args* v, const spec_expand_args* e, hipStream_t stream) {
  int rc = verify_check(v);
  if (rc != SPEC_OK) return rc;
  rc = expand_check(e);
  if (rc != SPEC_OK) return rc;
  // the expansion reads this verification's outputs: same batch, the counts
  // and the bonus source are the verification's own output arrays
  if (e->B != v->B || e->K != v->K) return SPEC_EINVAL;
  if (v->B == 0) return SPEC_OK;
  if (e->accepted_counts != v->accepted_counts || e->verify_output_tokens != v->output_tokens) return SPEC_EINVAL;
  bool vec;
  VerifyParams P = verify_params(v, vec);
  P.ex = expand_params(e, false, 1);  // one output row per wave on average
  P.ex_on = 1;
  P.ex_G = P.ex.G;
  if ((int64_t)P.B * P.nseg + (int64_t)P.B * P.ex_G > INT32_MAX) return SPEC_EINVAL;
  if (!verify_grids_fit(P.B, P.K, P.C1, P.nseg, P.dyn != 0, P.dstats != nullptr, (int64_t)P.B * P.ex_G))
    return SPEC_EINVAL;
  return verify_enqueue(P, v, vec, stream);
}

size_t spec_logprobs_workspace_bytes(int32_t B, int32_t R, int32_t V, int32_t top) {
  return logprobs_shape_ok(B, R, V, top) ? logprobs_ws_bytes(B, R, V, top) : 0;
}

int spec_logprobs_launch(const spec_logprobs_args* a, hipStream_t stream) {
  const int rc = logprobs_check(a);
  if (rc != SPEC_OK || a->B == 0 || a->R == 0) return rc;
  LogprobsParams P;
  P.B = a->B;
  P.R = a->R;
  P.V = a->V;
  P.nseg = (int32_t)(((int64_t)a->V + kSeg - 1) / kSeg);
  P.C = (P.nseg + kLpChunkSegs - 1) / kLpChunkSegs;
  P.by_C = FastDiv::by((uint32_t)P.C);
  P.by_R = FastDiv::by((uint32_t)P.R);
  P.top = a->top;
  P.logits = static_cast<const char*>(a->logits);
  P.req = a->req_stride;
  P.row = a->row_stride;
  P.tokens = a->tokens;
  P.temperature = a->temperature;
  P.logprobs = a->logprobs;
  P.entropy = a->entropy;
  P.top_ids = a->top_ids;
  P.top_lp = a->top_logprobs;
  char* ws = static_cast<char*>(a->workspace);
  P.rec = reinterpret_cast<LpRecord*>(ws);
  P.cells = reinterpret_cast<float*>(ws + align256((size_t)a->B * a->R * P.nseg * sizeof(LpRecord)));
  return launch_logprobs(P, a->dtype, stream) == hipSuccess ? SPEC_OK : SPEC_ELAUNCH;
}

int spec_kv_write_launch(const spec_kv_write_args* a, hipStream_t stream) {
  const int rc = kv_write_check(a);
  if (rc != SPEC_OK || a->N == 0) return rc;
  KvWriteParams P;
  P.c = cache_view(a->cache);
  P.N = a->N;
  P.chunk = kv_write_chunk(a->N);
  P.src[0] = static_cast<const char*>(a->key);
  P.src[1] = static_cast<const char*>(a->value);
  P.tok[0] = a->k_token_stride;
  P.hd[0] = a->k_head_stride;
  P.tok[1] = a->v_token_stride;
  P.hd[1] = a->v_head_stride;
  P.slots = a->slots;
  return launch_kv_write(P, a->dtype, stream) == hipSuccess ? SPEC_OK : SPEC_ELAUNCH;
}

int spec_kv_read_launch(const spec_kv_read_args* a, hipStream_t stream) {
  const int rc = kv_read_check(a);
  if (rc != SPEC_OK || a->N == 0) return rc;
  KvReadParams P;
  P.c = cache_view(a->cache);
  P.N = a->N;
  P.per = kv_read_per(a->N, a->cache.heads, a->cache.head_dim);
  P.dst[0] = static_cast<char*>(a->key);
  P.dst[1] = static_cast<char*>(a->value);
  P.slots = a->slots;
  return launch_kv_read(P, a->dtype, aligned16(a->key) && aligned16(a->value), stream) == hipSuccess ? SPEC_OK
                                                                                                     : SPEC_ELAUNCH;
}

size_t spec_attn_workspace_bytes(const spec_attn_args* a) {
  if (!a || !attn_sizes_ok(a)) return 0;
  return attn_ws_bytes(a, attn_plan(a, false));
}

int spec_attn_launch(const spec_attn_args* a, hipStream_t stream) {
  if (!a) return SPEC_EINVAL;
  AttnPlan plan;
  const int rc = attn_check(a, cache_check(a->cache), false, plan);
  if (rc != SPEC_OK || a->B == 0 || a->N == 0) return rc;
  return attn_launch(a, plan, cache_view(a->cache), false, stream);
}

size_t spec_attn4_workspace_bytes(const spec_attn4_args* a) {
  if (!a || a->cache.head_dim % 32) return 0;
  const spec_attn_args b = attn_of(a);
  return attn_sizes_ok(&b) ? attn_ws_bytes(&b, attn_plan(&b, true)) : 0;
}

int spec_attn4_launch(const spec_attn4_args* a, hipStream_t stream) {
  if (!a) return SPEC_EINVAL;
  const spec_attn_args b = attn_of(a);
  AttnPlan plan;
  const int rc = attn_check(&b, cache4_check(a->cache), true, plan);
  if (rc != SPEC_OK || a->B == 0 || a->N == 0) return rc;
  return attn_launch(&b, plan, cache4_view(a->cache), true, stream);
}

int spec_sample_launch(const spec_sample_args* a, hipStream_t stream) {
  const int rc = cut_check(a, a && a->row_index && a->rows == 0);
  if (rc != SPEC_OK || a->B == 0 || a->R == 0) return rc;
  if (!a->uniforms || !a->tokens) return SPEC_EINVAL;
  if (a->row_index ? a->rows < 0 : a->req_stride != 0 && a->req_stride / a->R < a->row_stride) return SPEC_EINVAL;
  CutParams P = cut_params(a);
  P.row_index = a->row_index;
  P.rows = a->rows;
  P.uniforms = a->uniforms;
  P.tokens = a->tokens;
  return launch_cut(P, a->dtype, stream) == hipSuccess ? SPEC_OK : SPEC_ELAUNCH;
}

size_t spec_sample_workspace_bytes(int32_t B, int32_t R, int32_t V) {
  return cut_shape_ok(B, R, V) ? cut_ws_bytes(B, R, V) : 0;
}

int spec_truncate_launch(const spec_truncate_args* a, hipStream_t stream) {
  const int rc = cut_check(a, false);
  if (rc != SPEC_OK || a->B == 0 || a->R == 0) return rc;
  if (!a->out) return SPEC_EINVAL;
  if (a->req_stride != 0 && a->req_stride / a->R < a->row_stride) return SPEC_EINVAL;
  if (a->out_row_stride < a->V || (a->B > 1 && a->out_req_stride / a->R < a->out_row_stride)) return SPEC_EINVAL;
  if (a->out == a->logits) {
    if (a->out_row_stride != a->row_stride || (a->B > 1 && a->out_req_stride != a->req_stride)) return SPEC_EINVAL;
  } else {  // (one workgroup's writes would change what another still reads)
    const int64_t es = a->dtype == SPEC_BF16 ? 2 : 4;
    if (rows_meet(mem_rows(a->logits, a->B, a->req_stride, a->R, a->row_stride, a->V, es),
                  mem_rows(a->out, a->B, a->out_req_stride, a->R, a->out_row_stride, a->V, es)))
      return SPEC_EINVAL;
  }
  CutParams P = cut_params(a);
  P.out = static_cast<char*>(a->out);
  P.out_req = a->out_req_stride;
  P.out_row = a->out_row_stride;
  return launch_cut(P, a->dtype, stream) == hipSuccess ? SPEC_OK : SPEC_ELAUNCH;
}

int spec_rope_launch(const spec_rope_args* a, hipStream_t stream) {
  RopeParams P;
  const int rc = rope_check(a, P);
  if (rc != SPEC_OK || a->N == 0 || a->q_heads + a->k_heads == 0) return rc;
  return launch_rope(P, a->dtype, stream) == hipSuccess ? SPEC_OK : SPEC_ELAUNCH;
}

int spec_kv4_write_launch(const spec_kv4_write_args* a, hipStream_t stream) {
  RopeParams P;
  const int rc = kv4_write_check(a, P);
  if (rc != SPEC_OK || a->N == 0) return rc;
  return launch_rope(P, a->dtype, stream) == hipSuccess ? SPEC_OK : SPEC_ELAUNCH;
}

int spec_kv4_read_launch(const spec_kv4_read_args* a, hipStream_t stream) {
  const int rc = kv4_read_check(a);
  if (rc != SPEC_OK || a->N == 0) return rc;
  KvReadParams P;
  P.c = cache4_view(a->cache);
  P.N = a->N;
  P.per = kv_read_per(a->N, a->cache.heads, a->cache.head_dim);
  P.dst[0] = static_cast<char*>(a->key);
  P.dst[1] = static_cast<char*>(a->value);
  P.slots = a->slots;
  return launch_kv4_read(P, a->dtype, stream) == hipSuccess ? SPEC_OK : SPEC_ELAUNCH;
}

}  // extern "C"

// The kernel parameters of a checked attention (B, N >= 1), and its launch.
namespace {
int attn_launch(const spec_attn_args* a, const AttnPlan& plan, const CacheView& view, bool four, hipStream_t stream) {
  AttnParams P;
  P.c = view;
  P.four = four;
  P.B = a->B;
  P.N = a->N;
  P.Hq = a->q_heads;
  P.G = a->q_heads / a->cache.heads;
  P.g_inv = 65535u / (uint32_t)P.G + 1u;
  P.max_q = a->max_q;
  P.max_ctx = a->max_ctx;
  P.window = a->window < (1 << 30) ? a->window : 1 << 30;  // (no context is longer)
  P.max_blocks = a->max_blocks;
  P.nrb = plan.nrb;
  P.chunks = plan.chunks;
  P.hw = plan.hw;
  P.items = (int32_t)plan.items;
  P.groups = (int32_t)plan.groups;
  P.q_flip = a->scale < 0.f ? 0x80008000u : 0u;
  P.scale2 = (a->scale < 0.f ? -a->scale : a->scale) * 1.44269504088896341f;
  P.q_keep = P.scale2 > 0.f ? ~0u : 0u;
  if (!(P.scale2 > 0.f)) P.scale2 = 1.f;
  P.q = static_cast<const char*>(a->q);
  P.q_tok = a->q_token_stride;
  P.q_head = a->q_head_stride;
  P.q_start = a->q_start;
  P.ctx_len = a->ctx_len;
  P.bt = a->block_table;
  P.bt_stride = a->bt_row_stride;
  P.sinks = a->sinks;
  P.out = static_cast<uint16_t*>(a->out);
  P.lse = a->lse;
  P.po = static_cast<float*>(a->workspace);
  P.pm = nullptr;
  P.runs = nullptr;
  if (plan.chunks > 0) {
    const size_t parts = (size_t)plan.chunks * 2 * a->cache.heads * 16 * plan.rt;
    char* ws = static_cast<char*>(a->workspace) + align256(parts * a->cache.head_dim * sizeof(float));
    P.pm = reinterpret_cast<float2*>(ws);
    P.runs = reinterpret_cast<int2*>(ws + align256(parts * sizeof(float2)));
  }
  P.qvec = aligned16(a->q) && a->q_token_stride % 8 == 0 && a->q_head_stride % 8 == 0;
  return launch_attn(P, plan, stream) == hipSuccess ? SPEC_OK : SPEC_ELAUNCH;
}
}  // namespace

extern "C" {

int spec_workspace_error(const void* workspace, hipStream_t stream) {
  if (workspace == nullptr) return SPEC_EINVAL;
  if (hipStreamSynchronize(stream) != hipSuccess) return SPEC_ELAUNCH;
  int32_t n = 0;
  if (hipMemcpy(&n, workspace, sizeof(n), hipMemcpyDeviceToHost) != hipSuccess) return SPEC_ELAUNCH;
  return n;
}

const char* spec_status_string(int status) {
  switch (status) {
    case SPEC_OK: return "SPEC_OK";
    case SPEC_EINVAL: return "SPEC_EINVAL: invalid argument (null pointer, size or stride out of range)";
    case SPEC_EDTYPE: return "SPEC_EDTYPE: unknown logits dtype";
    case SPEC_EALIGN: return "SPEC_EALIGN: workspace or statistics records not 16-byte aligned";
    case SPEC_EWORKSPACE: return "SPEC_EWORKSPACE: workspace too small";
    case SPEC_ELAUNCH: return "SPEC_ELAUNCH: kernel launch failed";
    default: return "unknown spec_status";
  }
}

}  // extern "C"
