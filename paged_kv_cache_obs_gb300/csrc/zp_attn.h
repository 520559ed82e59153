// zp_attn.h — host-side plans that the attention entry points share.
#pragma once

#include "zp_internal.h"

namespace zp {

constexpr uint64_t kWaitNs = 2000000000ull;  // a wait inside a kernel gives up after this

// What the split and the tiled attention kernels take.
struct AttnArgs {
  const uint8_t* pool;     // bf16 or E4M3 tiles
  const float* scales;     // E4M3 only
  int64_t num_blocks;
  const uint16_t* q;
  uint16_t* out;
  int64_t q_ts, q_hs, o_ts, o_hs;
  const int32_t* q_start;  // NULL: one query per request
  const int32_t *tables, *seq_lens;
  int32_t* err;
  float* part;             // [B][Hkv][parts][rows][d + 4]: sums, maximum, sum of weights
  int T, B, layer, layers, max_blocks, Hkv, G, b, max_q, window, sinks;
  int splits;              // CTAs that share a row's tokens
  bool ordered;            // split kernel: long requests first
  float sl2;               // scale * log2(e)
  uint64_t limit_ns;       // of a wait: kWaitNs, or the test hooks' limit
  bool stall;              // test hooks: a wait goes to a barrier that nothing completes
};

// The most rows (queries times heads of a group) that the split kernel takes.
constexpr int kMaxSplitRows = 16;

// The SMs that plans are made for: the current device's, or a GB300's where there is none (workspace sizes).
inline int plan_sms() {
  const int n = num_sms();
  return n > 0 ? n : 152;
}

// How a call is cut: CTAs of a (request, kv head), how many of them form a cluster, and what the
// partial sums of the clusters take.
struct SplitPlan {
  int rows;             // query rows that a CTA holds: 8 or 16
  int splits, cluster;
  bool ordered;  // long requests first
  size_t bytes;
};
// `room`: bytes of the workspace; what does not fit it is split among fewer CTAs.
constexpr size_t kHeader = 256;  // of a workspace: the error word
SplitPlan split_plan(const zp_params* p, int B, int max_q, int max_blocks, int window, int sinks, size_t room = SIZE_MAX);

// Launches the split kernel (and the one that joins its parts).
zp_status split_launch(AttnArgs a, const zp_params* p, bool fp8, const SplitPlan& plan, void* workspace, cudaStream_t st);

// How a call of the tiled kernel is cut: items (2 x 128 rows) of a request and kv head, CTAs that
// share an item's tiles, CTAs that are launched, items in all.
struct TilePlan {
  int nx, splits, ctas;
  int64_t items;
  size_t bytes;
};
TilePlan tile_plan(const zp_params* p, int T, int B, int max_q, int max_blocks, int window, int sinks, size_t room = SIZE_MAX);

// Launches the tiled kernel (rows above kMaxSplitRows), and the one that joins the parts.
zp_status tile_launch(AttnArgs a, const zp_kv_pool* pool, const zp_params* p, const TilePlan& plan, void* workspace, cudaStream_t st);

}  // namespace zp
