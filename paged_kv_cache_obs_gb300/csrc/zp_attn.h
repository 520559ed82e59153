// zp_attn.h — host-side plans that the attention entry points share.
#pragma once

#include "zp_internal.h"

namespace zp {

constexpr uint64_t kWaitNs = 2000000000ull;  // a wait inside a kernel gives up after this

// What the split and the tiled attention kernels take.
struct AttnArgs {
  const uint8_t* pool;     // bf16 or E4M3 tiles
  const float* scales;     // E4M3 only
  const uint16_t *k, *v;   // rows of packed prompts, in place of a pool
  int64_t k_ts, k_hs, v_ts, v_hs;
  bool kv_tma;             // they are aligned, and come by TMA
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
// `many8`: codes, and requests of several queries.
SplitPlan split_plan(const zp_params* p, int B, int max_q, int max_blocks, int window, int sinks, size_t room = SIZE_MAX, bool many8 = false);

// Launches the split kernel (and the one that joins its parts).
zp_status split_launch(AttnArgs a, const zp_params* p, bool fp8, const SplitPlan& plan, void* workspace, cudaStream_t st);

// How a call of the tiled kernel is cut: items (2 x 128 rows) of a request and kv head, CTAs that
// share an item's tiles, CTAs that are launched, items in all.
struct TilePlan {
  int nx, splits, ctas;
  int64_t items;
  size_t bytes;
};
// `rounds`: a CTA may take several parts one after another (over the bf16 pool it takes one, so that rows keep the sums that
// they had).
TilePlan tile_plan(const zp_params* p, int T, int B, int max_q, int max_blocks, int window, int sinks, size_t room = SIZE_MAX,
                   bool rounds = false);

// Launch the tiled kernel (rows above kMaxSplitRows, and prompts), and the one that joins the parts: over the bf16 pool, the
// 8-bit pool, or rows of packed prompts (whose a.b is the run of tokens that a copy brings: 16 or 128).
zp_status tile_launch(const AttnArgs& a, const zp_params* p, const TilePlan& plan, void* workspace, cudaStream_t st);
zp_status tile8_launch(const AttnArgs& a, const zp_params* p, const TilePlan& plan, void* workspace, cudaStream_t st);
// Packed prompts of up to 128 tokens (256 with 64-wide heads), in small CTAs.
bool short_prompts(const zp_params* p, int T, int B, int max_len);
zp_status short_launch(AttnArgs a, const zp_params* p, int max_len, void* workspace, cudaStream_t st);
zp_status tile_rows_launch(const AttnArgs& a, const zp_params* p, const TilePlan& plan, void* workspace, cudaStream_t st);

}  // namespace zp
