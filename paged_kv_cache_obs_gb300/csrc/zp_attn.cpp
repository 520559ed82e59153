// zp_attn.cpp — the entry points of decode attention over the 8-bit pool and of attention with a
// sliding window: argument checks, workspace, and the choice of the kernel.
#include <algorithm>
#include <climits>
#include <cmath>

#include "zp_attn.h"

namespace zp {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

zp_status check(const zp_params* p, int32_t layer, int64_t num_blocks, const zp_rows* q, const zp_rows* out,
                const int32_t* tables, const int32_t* seq_lens, int32_t T, int32_t B, int32_t max_blocks, int32_t window,
                int32_t sinks) {
  if (!p || B < 0 || max_blocks < 1 || window < 0 || sinks < 0 || num_blocks <= 0) return ZP_ERR_INVALID_ARG;
  if (layer < 0 || layer >= p->num_layers) return ZP_ERR_INVALID_ARG;
  // (layer, block) is one 32-bit coordinate of the tensor map
  if (num_blocks >= INT_MAX / p->num_layers) return ZP_ERR_UNSUPPORTED;
  if (p->num_kv_heads <= 0 || p->num_q_heads <= 0 || p->num_q_heads % p->num_kv_heads != 0) return ZP_ERR_INVALID_ARG;
  if (!(p->scale > 0.0f) || !std::isfinite(p->scale * kLog2e)) return ZP_ERR_INVALID_ARG;
  if (p->head_dim != 64 && p->head_dim != 128) return ZP_ERR_UNSUPPORTED;
  if (p->block_size != 16 && p->block_size != 32) return ZP_ERR_UNSUPPORTED;
  if (p->num_q_heads / p->num_kv_heads > 16 || B > 65535 || p->num_kv_heads > 65535) return ZP_ERR_UNSUPPORTED;
  // differences of three positions fit 32 bits
  if (static_cast<int64_t>(max_blocks) * p->block_size > (1 << 30)) return ZP_ERR_UNSUPPORTED;
  if (B == 0) return ZP_OK;
  if (!q || !out || !q->data || !out->data || !aligned(q->data, 2) || !aligned(out->data, 2)) return ZP_ERR_INVALID_ARG;
  if (rows_overlap(*out, T, p->num_q_heads, p->head_dim)) return ZP_ERR_INVALID_ARG;
  if (!tables || !seq_lens) return ZP_ERR_INVALID_ARG;
  return ZP_OK;
}

AttnArgs args_of(const zp_params* p, int32_t layer, int64_t num_blocks, const zp_rows* q, const zp_rows* out,
                 const int32_t* tables, const int32_t* seq_lens, int32_t B, int32_t max_blocks, int32_t window,
                 int32_t sinks) {
  AttnArgs a{};
  a.num_blocks = num_blocks;
  a.q = static_cast<const uint16_t*>(q->data);
  a.out = static_cast<uint16_t*>(out->data);
  a.q_ts = q->token_stride, a.q_hs = q->head_stride;
  a.o_ts = out->token_stride, a.o_hs = out->head_stride;
  a.tables = tables;
  a.seq_lens = seq_lens;
  a.B = B;
  a.layer = layer;
  a.layers = p->num_layers;
  a.max_blocks = max_blocks;
  a.Hkv = p->num_kv_heads;
  a.G = p->num_q_heads / p->num_kv_heads;
  a.b = p->block_size;
  // a window or first tokens past the longest cache see what all of it would
  const int most = max_blocks * p->block_size;
  a.window = window >= most ? 0 : window;
  a.sinks = sinks < most ? sinks : most;
  a.sl2 = p->scale * kLog2e;
  return a;
}

// A workspace of a call that asks for `need` bytes.  Fewer are taken if they are a multiple of 256 bytes,
// as the sizes of other batches and of other operators are: a batch that has shrunk asks for more than it
// did when it was large, since it is split further.  Any other number is not a workspace's size.
bool workspace_ok(const void* workspace, size_t bytes, size_t need) {
  return workspace && aligned(workspace, 256) && bytes >= kHeader && (bytes >= need || bytes % 256 == 0);
}

bool sizes_ok(const zp_params* p, int32_t B, int32_t max_blocks) {
  return p && B >= 0 && max_blocks >= 1 && p->num_kv_heads > 0 && p->num_q_heads > 0 &&
         p->num_q_heads % p->num_kv_heads == 0 && p->num_q_heads / p->num_kv_heads <= 16 && p->head_dim > 0 && p->block_size > 0;
}

// The two calls; stall_ns != 0 only from the test hooks.
zp_status kv8_decode(const zp_kv8_pool* pool, int32_t layer, const zp_rows* q, const int32_t* block_tables, const int32_t* seq_lens,
                     int32_t B, int32_t max_blocks, int32_t window, int32_t sinks, const zp_rows* out, const zp_params* p,
                     void* workspace, size_t workspace_bytes, zp_stream stream, uint64_t stall_ns) {
  if (!pool || !pool->codes || !pool->scales) return ZP_ERR_INVALID_ARG;
  const zp_status s = check(p, layer, pool->num_blocks, q, out, block_tables, seq_lens, B, B, max_blocks, window, sinks);
  if (s != ZP_OK) return s;
  if (!aligned(pool->codes, 16) || !aligned(pool->scales, 4)) return ZP_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes, zp_kv8_decode_workspace_size(p, B, max_blocks))) return ZP_ERR_INVALID_ARG;
  if (B == 0) return ZP_OK;
  AttnArgs a = args_of(p, layer, pool->num_blocks, q, out, block_tables, seq_lens, B, max_blocks, window, sinks);
  a.pool = static_cast<const uint8_t*>(pool->codes);
  a.scales = pool->scales;
  a.T = B;
  a.max_q = 1;
  a.stall = stall_ns != 0;
  a.limit_ns = a.stall ? stall_ns : kWaitNs;
  return split_launch(a, p, true, split_plan(p, B, 1, max_blocks, window, sinks, workspace_bytes), workspace,
                      reinterpret_cast<cudaStream_t>(stream));
}

zp_status paged_window(const zp_kv_pool* pool, int32_t layer, const zp_rows* q, const int32_t* q_start, int32_t T, int32_t max_q,
                       const int32_t* block_tables, const int32_t* seq_lens, int32_t B, int32_t max_blocks, int32_t window,
                       int32_t sinks, const zp_rows* out, const zp_params* p, void* workspace, size_t workspace_bytes,
                       zp_stream stream, uint64_t stall_ns) {
  if (!pool || !pool->base || T < 0 || max_q < 1) return ZP_ERR_INVALID_ARG;
  if (T == 0) B = 0;  // nothing to do, and q and out may be empty
  const zp_status s = check(p, layer, pool->num_blocks, q, out, block_tables, seq_lens, T, B, max_blocks, window, sinks);
  if (s != ZP_OK) return s;
  if (!aligned(pool->base, 16) || (B > 0 && !q_start)) return ZP_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes, zp_paged_window_workspace_size(p, T, B, max_q, max_blocks, window, sinks)))
    return ZP_ERR_INVALID_ARG;
  if (B == 0) return ZP_OK;
  AttnArgs a = args_of(p, layer, pool->num_blocks, q, out, block_tables, seq_lens, B, max_blocks, window, sinks);
  a.pool = static_cast<const uint8_t*>(pool->base);
  a.q_start = q_start;
  a.T = T;
  // a request of more tokens than its blocks hold is refused by its length in any case
  a.max_q = std::min(max_q, max_blocks * p->block_size);
  a.stall = stall_ns != 0;
  a.limit_ns = a.stall ? stall_ns : kWaitNs;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (static_cast<int64_t>(a.G) * max_q <= kMaxSplitRows) {
    return split_launch(a, p, false, split_plan(p, B, max_q, max_blocks, window, sinks, workspace_bytes), workspace, st);
  }
  return tile_launch(a, pool, p, tile_plan(p, T, B, max_q, max_blocks, window, sinks, workspace_bytes), workspace, st);
}

bool stall_ok(int64_t ns) { return ns >= 1 && ns <= 1000000000; }

}  // namespace
}  // namespace zp

using namespace zp;

extern "C" size_t zp_kv8_decode_workspace_size(const zp_params* p, int32_t B, int32_t max_blocks) {
  if (!sizes_ok(p, B, max_blocks)) return 0;
  return split_plan(p, B, 1, max_blocks, 0, 0).bytes;
}

extern "C" size_t zp_paged_window_workspace_size(const zp_params* p, int32_t T, int32_t B, int32_t max_q,
                                                 int32_t max_blocks, int32_t window, int32_t sinks) {
  if (!sizes_ok(p, B, max_blocks) || T < 0 || max_q < 1 || window < 0 || sinks < 0) return 0;
  if (static_cast<int64_t>(p->num_q_heads / p->num_kv_heads) * max_q > kMaxSplitRows)
    return tile_plan(p, T, B, max_q, max_blocks, window, sinks).bytes;
  return split_plan(p, B, max_q, max_blocks, window, sinks).bytes;
}

extern "C" zp_status zp_kv8_decode_attn(const zp_kv8_pool* pool, int32_t layer, const zp_rows* q,
                                        const int32_t* block_tables, const int32_t* seq_lens, int32_t B,
                                        int32_t max_blocks, int32_t window, int32_t sinks, const zp_rows* out,
                                        const zp_params* p, void* workspace, size_t workspace_bytes, zp_stream stream) {
  zp::NvtxRange nvtx_range("zp_kv8_decode_attn");
  return kv8_decode(pool, layer, q, block_tables, seq_lens, B, max_blocks, window, sinks, out, p, workspace, workspace_bytes, stream, 0);
}

extern "C" zp_status zp_paged_window_attn(const zp_kv_pool* pool, int32_t layer, const zp_rows* q, const int32_t* q_start,
                                          int32_t T, int32_t max_q, const int32_t* block_tables, const int32_t* seq_lens,
                                          int32_t B, int32_t max_blocks, int32_t window, int32_t sinks, const zp_rows* out,
                                          const zp_params* p, void* workspace, size_t workspace_bytes, zp_stream stream) {
  zp::NvtxRange nvtx_range("zp_paged_window_attn");
  return paged_window(pool, layer, q, q_start, T, max_q, block_tables, seq_lens, B, max_blocks, window, sinks, out, p, workspace,
                      workspace_bytes, stream, 0);
}

extern "C" zp_status zp_test_kv8_decode_stalled(const zp_kv8_pool* pool, int32_t layer, const zp_rows* q,
                                                const int32_t* block_tables, const int32_t* seq_lens, int32_t B,
                                                int32_t max_blocks, int32_t window, int32_t sinks, const zp_rows* out,
                                                const zp_params* p, void* workspace, size_t workspace_bytes,
                                                int64_t stall_limit_ns, zp_stream stream) {
  if (!stall_ok(stall_limit_ns)) return ZP_ERR_INVALID_ARG;
  return kv8_decode(pool, layer, q, block_tables, seq_lens, B, max_blocks, window, sinks, out, p, workspace, workspace_bytes, stream,
                    static_cast<uint64_t>(stall_limit_ns));
}

extern "C" zp_status zp_test_paged_window_stalled(const zp_kv_pool* pool, int32_t layer, const zp_rows* q, const int32_t* q_start,
                                                  int32_t T, int32_t max_q, const int32_t* block_tables,
                                                  const int32_t* seq_lens, int32_t B, int32_t max_blocks, int32_t window,
                                                  int32_t sinks, const zp_rows* out, const zp_params* p, void* workspace,
                                                  size_t workspace_bytes, int64_t stall_limit_ns, zp_stream stream) {
  if (!stall_ok(stall_limit_ns)) return ZP_ERR_INVALID_ARG;
  return paged_window(pool, layer, q, q_start, T, max_q, block_tables, seq_lens, B, max_blocks, window, sinks, out, p, workspace,
                      workspace_bytes, stream, static_cast<uint64_t>(stall_limit_ns));
}
