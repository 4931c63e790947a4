// attention_plan.hpp -- how an attention's rows and keys are cut into
// workgroups (host code; the kernels read the result from their parameters).
#pragma once

#include <stdint.h>

namespace specv {

constexpr int kTileKeys = 32;     // keys of a tile
constexpr int kAttnWaves = 4;     // waves of a workgroup
constexpr int kAttnWindow = 32;   // tiles whose pages a wave holds at a time: it looks them up anew after as many

// All units' tiles, end to end, are cut into `chunks` equal runs, none shorter
// than kMinChunk (32: 94 us against 82 for 64 contexts of 4096 tokens; 8: no
// faster).
constexpr int kMinChunk = 16;
constexpr int kMaxRunUnits = 65536;  // a workgroup's room for their tiles, 64 units to a place
constexpr int64_t attn_run_tiles(int64_t total, int32_t chunks) {
  return (total + chunks - 1) / chunks > kMinChunk ? (total + chunks - 1) / chunks : kMinChunk;
}

struct AttnPlan {
  int32_t rt;      // row tiles (of 16) to a block of rows
  int32_t nrb;     // blocks of rows per (request, KV head)
  int32_t chunks;  // equal runs of tiles (0: a unit to a workgroup)
  int32_t hw;      // KV heads of a workgroup
  int64_t items, groups;
};

// Workgroups that a CU holds at once: the plan counts on so many, and the kernels'
// launch bounds keep their registers low enough for them.  8 bits at 64 dims and
// one row tile: 4 would fit in part, 118 us against 107 for 256 contexts of 2048
// tokens.  4 bits, one row tile: 4 at 64 dims, 31 us against 46 with 3 for 256
// contexts of 2048 tokens with four heads; 3 at 128, 81 us against 87 with 2 for
// three contexts of up to 131072, 46 against 52 for 64 of 4096.
constexpr int attn_resident(int dim, int rt, bool four) {
  return four && rt == 1 && dim <= 128 ? (dim <= 64 ? 4 : 3) : dim <= 64 && rt <= 2 ? 3 : 2;
}

// heads_in: the heads of a token stand together in the cache; four: it holds 4 bits.
inline AttnPlan plan_attn(int32_t B, int32_t G, int32_t heads, int32_t dim, int32_t max_q, int32_t max_ctx, int32_t window,
                   bool heads_in, bool four = false) {
  AttnPlan p;
  const int64_t rows = (int64_t)max_q * G;
  const int64_t tiles = (rows + 15) / 16;
  const int rt_max = dim > 128 ? 1 : dim > 64 ? 3 : 5;
  p.nrb = (int32_t)((tiles + rt_max - 1) / rt_max);
  p.rt = (int32_t)((tiles + p.nrb - 1) / p.nrb);
  p.nrb = (int32_t)((tiles + p.rt - 1) / p.rt);
  // keys that one block of rows can see
  int64_t keys = max_ctx;
  if (window > 0 && (int64_t)window + p.rt * 16 < keys) keys = (int64_t)window + p.rt * 16;
  const int64_t units = (int64_t)B * p.nrb;
  const int slots = 256 * attn_resident(dim, p.rt, four);  // workgroups that the card holds at once
  // heads that stand side by side in a token, to a wave each: a workgroup reads
  // them together
  const int hw = p.rt > 1 || !heads_in ? 1 : heads % 4 == 0 ? 4 : heads % 2 == 0 ? 2 : 1;
  p.hw = 1;
  if (keys <= 1024 || (keys <= 2048 && units * heads <= slots) ||
      (keys <= 4096 && units * (heads / hw) >= 2 * slots) || units > kMaxRunUnits ||
      (p.nrb > 1 && units * heads >= 2 * slots)) {
    // a unit to a workgroup, the blocks of one head on one XCD, for its keys:
    // short contexts (8 of 1500 tokens: 19 us against 24 in runs, but 256 of
    // 2048: 117 against 107), so many units that the card is full of them (2000
    // with two heads of up to 1500 tokens: 82 us against 103, 8000 with one: 144
    // against 207; a few long ones among many would be its last), more units
    // than the runs' beginnings are searched for in, or many blocks of long
    // prompts (two chunks of 2048 tokens in contexts of 8192: 391 us against 530)
    p.chunks = 0;
    // (512 requests of up to 1000 tokens, 8 heads of 64, which half fill a line
    // each: 77 us against 108; where it leaves workgroups idle, fewer heads)
    p.hw = hw;
    while (p.hw > 1 && units * (heads / p.hw) < slots) p.hw /= 2;
    p.items = p.nrb;
    p.groups = (int64_t)B * (heads / p.hw);
  } else {
    // equal runs, as many as are resident at once; a run's heads on one XCD.
    // With few rows (small partial sums), long runs and a token's heads side
    // by side a wave takes a head of its own, so that a workgroup reads them
    // together (three contexts of 131072 tokens: 141 us against 167; where
    // tokens stand inside heads it is the other way, 150 against 133).
    if (units * keys / kTileKeys * heads >= (int64_t)slots * kAttnWaves * 32)
      p.hw = hw;
    const int hgroups = heads / p.hw;
    p.chunks = slots / hgroups > 8 ? slots / hgroups / 8 * 8 : 8;
    p.items = hgroups;
    p.groups = p.chunks;
  }
  return p;
}

}  // namespace specv
