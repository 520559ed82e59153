// zp_append.cu — new keys and values into the bf16 pool, by slot; sm_103a.
//
// Row t of k and v goes to token slots[t] % b of block slots[t] / b: a copy, bound by HBM (every value is read
// once and written once).  A thread keeps its 16 bytes of a row and walks the CTA's rows (token, K or V, head) without
// divisions, the slot and the values of several rows on their way together: 8200 tokens of 8 heads of 128 take 12.4 us, 5.4 TB/s
// (13.5 with a division for each row).
#include <algorithm>
#include <climits>

#include "zp_internal.h"
#include "zp_launch.h"

namespace zp {
namespace {

constexpr int kThreadsA = 128;
constexpr int kRowsA = 4;  // of a thread, whose loads are in flight together
constexpr int kCtaRows = 32;  // of a CTA at least: whole tokens

struct AppendArgs {
  const uint16_t *k, *v;
  int64_t k_ts, k_hs, v_ts, v_hs;
  const int32_t* slots;
  uint16_t* pool;  // of the layer
  int32_t* err;
  int64_t num_slots;
  int T, tokens, Hkv, bshift;  // tokens: of a CTA
};

// D: head size; WIDE: rows are 16-byte aligned.
template <int D, bool WIDE>
__global__ void __launch_bounds__(kThreadsA) append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int kVecs = D / 8, kWalk = kThreadsA / kVecs;  // 16-byte pieces of a row, rows of a pass
  after_previous();
  next_may_start();
  const int c = threadIdx.x % kVecs, per = 2 * a.Hkv;  // place in the row; rows of a token
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tokens;
  const int end = static_cast<int>(min(static_cast<int64_t>(a.tokens), a.T - t0)) * per;
  int row = threadIdx.x / kVecs, tk = row / per, kvh = row - tk * per;
  bool bad = false;
  while (row < end) {
    uint4 x[kRowsA];
    uint16_t* to[kRowsA];
#pragma unroll
    for (int u = 0; u < kRowsA; ++u) {
      to[u] = nullptr;
      if (row >= end) continue;
      const int64_t t = t0 + tk, slot = a.slots[t];
      const bool is_v = kvh >= a.Hkv;
      const int64_t h = is_v ? kvh - a.Hkv : kvh;
      const uint16_t* const from = (is_v ? a.v + t * a.v_ts + h * a.v_hs : a.k + t * a.k_ts + h * a.k_hs) + c * 8;
      if (WIDE) {
        x[u] = *reinterpret_cast<const uint4*>(from);
      } else {
        uint32_t y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = static_cast<uint32_t>(from[2 * e]) | static_cast<uint32_t>(from[2 * e + 1]) << 16;
        x[u] = make_uint4(y[0], y[1], y[2], y[3]);
      }
      bad |= slot >= a.num_slots;
      if (slot >= 0 && slot < a.num_slots) {
        const int64_t tile = (slot >> a.bshift) * per + kvh;
        to[u] = a.pool + (((tile << a.bshift) + (slot & ((1 << a.bshift) - 1))) * D + c * 8);
      }
      row += kWalk;
      kvh += kWalk;
      while (kvh >= per) kvh -= per, ++tk;
    }
#pragma unroll
    for (int u = 0; u < kRowsA; ++u)
      if (to[u]) *reinterpret_cast<uint4*>(to[u]) = x[u];
  }
  if (bad) atomicCAS(a.err, 0, ZP_ERR_BAD_TABLE);
}

}  // namespace
}  // namespace zp

using namespace zp;

extern "C" zp_status zp_kv_append(const zp_kv_pool* pool, int32_t layer, const zp_rows* k, const zp_rows* v, const int32_t* slots,
                                  int32_t T, const zp_params* p, void* workspace, size_t workspace_bytes, zp_stream stream) {
  zp::NvtxRange nvtx_range("zp_kv_append");
  if (!pool || !pool->base || !p || pool->num_blocks <= 0 || T < 0) return ZP_ERR_INVALID_ARG;
  if (!aligned(pool->base, 16) || layer < 0 || layer >= p->num_layers || p->num_kv_heads <= 0) return ZP_ERR_INVALID_ARG;
  if ((p->head_dim != 64 && p->head_dim != 128) || (p->block_size != 16 && p->block_size != 32) || p->num_kv_heads > 65535)
    return ZP_ERR_UNSUPPORTED;
  if (pool->num_blocks > INT_MAX / p->block_size) return ZP_ERR_UNSUPPORTED;  // slots are 32-bit numbers
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < 256) return ZP_ERR_INVALID_ARG;
  if (T == 0) return ZP_OK;
  if (!slots || !k || !v || !k->data || !v->data || !aligned(k->data, 2) || !aligned(v->data, 2)) return ZP_ERR_INVALID_ARG;
  AppendArgs a{};
  a.k = static_cast<const uint16_t*>(k->data);
  a.v = static_cast<const uint16_t*>(v->data);
  a.k_ts = k->token_stride, a.k_hs = k->head_stride, a.v_ts = v->token_stride, a.v_hs = v->head_stride;
  a.slots = slots;
  const int64_t values = pool->num_blocks * 2 * p->num_kv_heads * p->block_size * p->head_dim;  // of a layer
  a.pool = static_cast<uint16_t*>(pool->base) + layer * values;
  a.err = static_cast<int32_t*>(workspace);
  a.num_slots = pool->num_blocks * p->block_size;
  a.T = T;
  a.tokens = std::max(1, kCtaRows / (2 * p->num_kv_heads));
  a.Hkv = p->num_kv_heads;
  a.bshift = p->block_size == 16 ? 4 : 5;
  const bool vec = wide(k) && wide(v);
  const int grid = static_cast<int>((static_cast<int64_t>(T) + a.tokens - 1) / a.tokens);
  auto* const kernel = p->head_dim == 128 ? (vec ? append_kernel<128, true> : append_kernel<128, false>)
                                          : (vec ? append_kernel<64, true> : append_kernel<64, false>);
  return launch_in_order(kernel, dim3(static_cast<unsigned>(grid)), kThreadsA, 0, reinterpret_cast<cudaStream_t>(stream), 1, a) ==
                 cudaSuccess
             ? ZP_OK
             : ZP_ERR_CUDA;
}
