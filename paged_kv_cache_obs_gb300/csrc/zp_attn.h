// zp_attn.h — host-side plans that the attention entry points share.
#pragma once

#include "zp_internal.h"

namespace zp {

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
  uint32_t* done;          // [B][Hkv] splits of the row finished so far; zero between calls
  float* part;             // [B][Hkv][max_splits][rows][d + 2]
  int T, B, layer, max_blocks, Hkv, G, b, max_q, window, sinks;
  int tps, max_splits;     // 16-token tiles per split; splits of the longest request
  float sl2;               // scale * log2(e)
};

struct SplitPlan {
  int rows;         // query rows of a (request, kv head) that a CTA holds: 8 or 16
  int tps, splits;
};

// The most rows (queries times heads of a group) that the split kernel takes.
constexpr int kMaxSplitRows = 16;

SplitPlan split_plan(const zp_params* p, int B, int max_q, int64_t max_tokens, int window, int sinks);

// Workspace that no call of these sizes exceeds, whatever its window.
size_t split_bytes(const zp_params* p, int B, int max_q, int64_t max_tokens);

// Launches the split kernel; `a.tps`, `a.max_splits`, `a.done` and `a.part` are set from the plan
// and the workspace.
zp_status split_launch(AttnArgs a, bool fp8, int head_dim, const SplitPlan& plan, void* workspace, cudaStream_t st);

// Launches the tiled kernel (rows above kMaxSplitRows); of the workspace it uses the error word.
zp_status tile_launch(AttnArgs a, const zp_kv_pool* pool, const zp_params* p, void* workspace, cudaStream_t st);

}  // namespace zp
