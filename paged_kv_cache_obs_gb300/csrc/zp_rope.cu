// zp_rope.cu — rotary positions of queries and keys, sm_103a.
//
// Pair i of a token at position p is turned by the angle p * f_i:
//   (y_a, y_b) = m * (x_a cos - x_b sin, x_b cos + x_a sin).
// f_i is held as turns per position in units of 2^-64, so p * f_i modulo one turn is one 64-bit
// integer product, exact for every int32 position (its only error is the table's own, which is fp64's
// rounding of f_i / 2 pi: |p| 2^-56 turns for the fastest pair); in fp32 the angle of position 10^6 would be off by 0.06 rad.  The top 32 bits
// are the signed fraction of a turn that sincospif takes.
//
// The kernel is bound by HBM: every value is read once and written once (out of place).  A CTA
// takes a few tokens: its threads first issue the loads of their first values, then compute the
// tokens' cos and sin (one pair per thread, shared by all heads through shared memory) while
// those are on their way.
#include <cmath>

#include "zp_internal.h"
#include "zp_launch.h"
#include "zp_ptx.cuh"

namespace zp {
namespace {

// Small CTAs with few loads a thread, so that an SM holds many of them at different stages: 8192 tokens
// of 32 heads of 128 take 21.9 us (6.1 TB/s) so, 24.3 with 256 threads, 25.1 with 4 rows a thread too.
constexpr int kThreadsR = 128;
// Rows of a thread whose loads are in flight together: 3 in CTAs of one token, which have few (256 tokens of 40 heads
// of 128 take 3.45 us so and 3.6 with 2, one token 2.8 and 3.2), 2 in those of two (see above).
constexpr int kRowsOne = 3, kRowsR = 2;
// Tokens per CTA: two where there are CTAs enough (2047 tokens of 40 heads take 10.6 us so and 11.3 with one),
// one below 1024 tokens (1000 take 5.8 us with one, 6.6 with two).
constexpr int kMaxTokensR = 2;

struct RopeArgs {
  const uint16_t *q, *k;
  uint16_t *qo, *ko;
  int64_t q_ts, q_hs, k_ts, k_hs, qo_ts, qo_hs, ko_ts, ko_hs;
  const int32_t* positions;
  int T, Hq, Hkv, d, rd, inplace_q, inplace_k, tokens;  // tokens: per CTA
  float mscale;
};

// One pair; the roundings are written out so that every form of the kernel gives the same bits.
__device__ __forceinline__ float turn_a(float a, float b, float c, float s) { return fmaf(a, c, -__fmul_rn(b, s)); }
__device__ __forceinline__ float turn_b(float a, float b, float c, float s) { return fmaf(b, c, __fmul_rn(a, s)); }

__device__ __forceinline__ void fill_table(const zp_rope& rope, const RopeArgs& a, int t0, int nt, float2* cs) {
  const int half = a.rd >> 1;
  for (int i = threadIdx.x; i < nt * half; i += blockDim.x) {
    const int tk = i / half, pair = i - tk * half;
    const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(a.positions[t0 + tk])) * rope.turns[pair];
    float s, c;
    sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31
    cs[i] = make_float2(c * a.mscale, s * a.mscale);
  }
}

struct Row {
  const uint16_t* in;
  uint16_t* out;
  bool skip_rest;  // in place: values past rotary_dim stay
};

__device__ __forceinline__ Row row_of(const RopeArgs& a, int t, int head) {
  if (head < a.Hq)
    return {a.q + t * a.q_ts + head * a.q_hs, a.qo + t * a.qo_ts + head * a.qo_hs, a.inplace_q != 0};
  const int h = head - a.Hq;
  return {a.k + t * a.k_ts + h * a.k_hs, a.ko + t * a.ko_ts + h * a.ko_hs, a.inplace_k != 0};
}

// Wide form: rotary_dim and head_dim are multiples of 16 and every row is 16-byte aligned.  An
// item is two 16-byte vectors of a row: the two halves of 8 pairs (half layout), 8 adjacent pairs
// (interleaved), or 16 values that pass through.  A thread keeps its place in the row and walks the
// CTA's rows (token, head), so that no item costs a division.
template <bool INTER, int U>
__global__ void __launch_bounds__(kThreadsR) rope_wide_kernel(const __grid_constant__ zp_rope rope, const RopeArgs a) {
  __shared__ __align__(16) float2 cs[kMaxTokensR * 128];
  after_previous();
  next_may_start();
  const int t0 = blockIdx.x * a.tokens, nt = min(a.tokens, a.T - t0);
  const int per_row = a.d >> 4, rot = a.rd >> 4, half = a.rd >> 1, heads = a.Hq + a.Hkv;
  const int walk = kThreadsR / per_row, v = threadIdx.x % per_row;  // rows of a pass; place in the row
  const bool turn = v < rot;
  const int oa = (turn && !INTER) ? v * 8 : v * 16, ob = (turn && !INTER) ? half : 8;
  const int end = nt * heads;
  int row = threadIdx.x / per_row;
  if (row >= walk) row = end;  // threads that a pass does not need
  int tk = row / heads, head = row - tk * heads;
  bool table = false;
  while (row < end || !table) {
    uint4 va[U], vb[U];
    uint16_t* op[U];
    int ci[U];  // table index of the first pair
#pragma unroll
    for (int u = 0; u < U; ++u) {
      op[u] = nullptr;
      if (row < end) {
        const Row r = row_of(a, t0 + tk, head);
        ci[u] = tk * half + v * 8;
        if (turn || !r.skip_rest) {
          op[u] = r.out + oa;
          va[u] = *reinterpret_cast<const uint4*>(r.in + oa);
          vb[u] = *reinterpret_cast<const uint4*>(r.in + oa + ob);
        }
        row += walk;
        head += walk;
        while (head >= heads) head -= heads, ++tk;
      }
    }
    if (!table) {
      fill_table(rope, a, t0, nt, cs);
      __syncthreads();
      table = true;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!op[u]) continue;
      uint32_t xa[4] = {va[u].x, va[u].y, va[u].z, va[u].w}, xb[4] = {vb[u].x, vb[u].y, vb[u].z, vb[u].w};
      if (turn) {
        const float4* tab = reinterpret_cast<const float4*>(cs + ci[u]);  // (cos, sin) of two pairs
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 w = tab[e];
          if (INTER) {
            uint32_t& x0 = e < 2 ? xa[2 * e] : xb[2 * e - 4];
            uint32_t& x1 = e < 2 ? xa[2 * e + 1] : xb[2 * e - 3];
            x0 = pack_bf16x2(turn_a(bf16x2_lo(x0), bf16x2_hi(x0), w.x, w.y), turn_b(bf16x2_lo(x0), bf16x2_hi(x0), w.x, w.y));
            x1 = pack_bf16x2(turn_a(bf16x2_lo(x1), bf16x2_hi(x1), w.z, w.w), turn_b(bf16x2_lo(x1), bf16x2_hi(x1), w.z, w.w));
          } else {
            const float a0 = bf16x2_lo(xa[e]), a1 = bf16x2_hi(xa[e]), b0 = bf16x2_lo(xb[e]), b1 = bf16x2_hi(xb[e]);
            xa[e] = pack_bf16x2(turn_a(a0, b0, w.x, w.y), turn_a(a1, b1, w.z, w.w));
            xb[e] = pack_bf16x2(turn_b(a0, b0, w.x, w.y), turn_b(a1, b1, w.z, w.w));
          }
        }
      }
      *reinterpret_cast<uint4*>(op[u]) = make_uint4(xa[0], xa[1], xa[2], xa[3]);
      *reinterpret_cast<uint4*>(op[u] + ob) = make_uint4(xb[0], xb[1], xb[2], xb[3]);
    }
  }
}

// Any sizes and strides: an item is one pair, or one value that passes through.
template <bool INTER>
__global__ void __launch_bounds__(kThreadsR) rope_any_kernel(const __grid_constant__ zp_rope rope, const RopeArgs a) {
  __shared__ __align__(16) float2 cs[kMaxTokensR * 128];
  after_previous();
  next_may_start();
  const int t0 = blockIdx.x * a.tokens, nt = min(a.tokens, a.T - t0);
  const int half = a.rd >> 1, per_row = half + a.d - a.rd, heads = a.Hq + a.Hkv;
  fill_table(rope, a, t0, nt, cs);
  __syncthreads();
  for (int i = threadIdx.x; i < nt * heads * per_row; i += kThreadsR) {
    const int row = i / per_row, v = i - row * per_row;
    const int tk = row / heads, head = row - tk * heads;
    const Row r = row_of(a, t0 + tk, head);
    if (v >= half) {
      if (!r.skip_rest) r.out[v - half + a.rd] = r.in[v - half + a.rd];
      continue;
    }
    const int ia = INTER ? 2 * v : v, ib = INTER ? 2 * v + 1 : v + half;
    const float2 w = cs[tk * half + v];
    const float xa = bf16x2_lo(r.in[ia]), xb = bf16x2_lo(r.in[ib]);
    const uint32_t y = pack_bf16x2(turn_a(xa, xb, w.x, w.y), turn_b(xa, xb, w.x, w.y));
    r.out[ia] = static_cast<uint16_t>(y);
    r.out[ib] = static_cast<uint16_t>(y >> 16);
  }
}

}  // namespace
}  // namespace zp

using namespace zp;

extern "C" zp_status zp_rope_init(const zp_rope_config* c, zp_rope* out) {
  if (!c || !out) return ZP_ERR_INVALID_ARG;
  const int d = c->head_dim, rd = c->rotary_dim;
  if (d < 2 || d > 512 || d % 2 || rd < 2 || rd > d || rd > 256 || rd % 2) return ZP_ERR_INVALID_ARG;
  if (c->scaling < ZP_ROPE_NONE || c->scaling > ZP_ROPE_WAVELENGTH) return ZP_ERR_INVALID_ARG;
  if (!(c->theta > 1.0) || !std::isfinite(c->theta) || !std::isfinite(c->mscale)) return ZP_ERR_INVALID_ARG;
  if (c->scaling != ZP_ROPE_NONE && (!(c->factor >= 1.0) || !std::isfinite(c->factor))) return ZP_ERR_INVALID_ARG;
  const bool turns = c->scaling == ZP_ROPE_YARN || c->scaling == ZP_ROPE_WAVELENGTH;
  if (turns && (c->original_len <= 0 || !(c->low > 0.0) || !(c->high > c->low) || !std::isfinite(c->high)))
    return ZP_ERR_INVALID_ARG;
  if (c->scaling == ZP_ROPE_BASE && rd < 4) return ZP_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925286766559;
  const double theta = c->scaling == ZP_ROPE_BASE ? c->theta * std::pow(c->factor, double(rd) / (rd - 2)) : c->theta;
  // pair index (real-valued) that makes `n` turns over original_len positions
  const auto pair_of = [&](double n) {
    return rd * std::log(c->original_len / (n * two_pi)) / (2.0 * std::log(theta));
  };
  double lo = 0.0, hi = 0.0;
  if (c->scaling == ZP_ROPE_YARN) {
    lo = std::fmax(std::floor(pair_of(c->high)), 0.0);
    hi = std::fmin(std::ceil(pair_of(c->low)), rd - 1.0);
  }
  zp_rope r{};
  r.head_dim = d;
  r.rotary_dim = rd;
  r.interleaved = c->interleaved != 0;
  r.mscale = static_cast<float>(
      c->mscale != 0.0 ? c->mscale : (c->scaling == ZP_ROPE_YARN ? 0.1 * std::log(c->factor) + 1.0 : 1.0));
  for (int i = 0; i < rd / 2; ++i) {
    double f = std::pow(theta, -2.0 * i / rd);
    if (c->scaling == ZP_ROPE_LINEAR) f /= c->factor;
    if (c->scaling == ZP_ROPE_YARN) {
      const double ramp = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
      f = f * (1.0 - ramp) + f / c->factor * ramp;
    }
    if (c->scaling == ZP_ROPE_WAVELENGTH) {
      const double n = c->original_len * f / two_pi;
      const double mix = std::fmin(std::fmax((n - c->low) / (c->high - c->low), 0.0), 1.0);
      f = (1.0 - mix) * f / c->factor + mix * f;
    }
    // f <= 1, so at most 1 / (2 pi) of a turn per position: the product stays below 2^62
    r.turns[i] = static_cast<uint64_t>(std::llrint(f / two_pi * 18446744073709551616.0));
  }
  if (!std::isfinite(r.mscale)) return ZP_ERR_INVALID_ARG;
  *out = r;
  return ZP_OK;
}

extern "C" zp_status zp_rope_apply(const zp_rope* rope, const zp_rows* q, const zp_rows* q_out, int32_t num_q_heads,
                                   const zp_rows* k, const zp_rows* k_out, int32_t num_kv_heads,
                                   const int32_t* positions, int32_t T, zp_stream stream) {
  zp::NvtxRange nvtx_range("zp_rope_apply");
  if (!rope || T < 0 || num_q_heads < 0 || num_kv_heads < 0) return ZP_ERR_INVALID_ARG;
  const int d = rope->head_dim, rd = rope->rotary_dim;
  if (d < 2 || d > 512 || d % 2 || rd < 2 || rd > d || rd > 256 || rd % 2) return ZP_ERR_INVALID_ARG;
  const int Hq = q ? num_q_heads : 0, Hkv = k ? num_kv_heads : 0;
  if (Hq > 4096 || Hkv > 4096) return ZP_ERR_UNSUPPORTED;
  if (T == 0 || Hq + Hkv == 0) return ZP_OK;
  if (!positions) return ZP_ERR_INVALID_ARG;
  RopeArgs a{};
  bool vec = d % 16 == 0 && rd % 16 == 0;
  // rows are bf16 at 2-byte addresses; in place means the same rows, strides included
  const auto take = [&](const zp_rows* in, const zp_rows* out, int heads, int& same) {
    if (!out || !in->data || !out->data || !aligned(in->data, 2) || !aligned(out->data, 2)) return false;
    if (rows_overlap(*out, T, heads, d)) return false;
    same = in->data == out->data;
    if (same && (in->token_stride != out->token_stride || in->head_stride != out->head_stride)) return false;
    vec = vec && wide(in) && wide(out);
    return true;
  };
  if (Hq > 0) {
    if (!take(q, q_out, Hq, a.inplace_q)) return ZP_ERR_INVALID_ARG;
    a.q = static_cast<const uint16_t*>(q->data);
    a.qo = static_cast<uint16_t*>(q_out->data);
    a.q_ts = q->token_stride, a.q_hs = q->head_stride, a.qo_ts = q_out->token_stride, a.qo_hs = q_out->head_stride;
  }
  if (Hkv > 0) {
    if (!take(k, k_out, Hkv, a.inplace_k)) return ZP_ERR_INVALID_ARG;
    a.k = static_cast<const uint16_t*>(k->data);
    a.ko = static_cast<uint16_t*>(k_out->data);
    a.k_ts = k->token_stride, a.k_hs = k->head_stride, a.ko_ts = k_out->token_stride, a.ko_hs = k_out->head_stride;
  }
  a.positions = positions;
  a.T = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.d = d;
  a.rd = rd;
  a.mscale = rope->mscale;
  a.tokens = T >= kMaxTokensR * 512 ? kMaxTokensR : 1;
  const unsigned grid = static_cast<unsigned>((T + a.tokens - 1) / a.tokens);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool inter = rope->interleaved != 0;
  auto* const kernel = vec && a.tokens == 1 ? (inter ? rope_wide_kernel<true, kRowsOne> : rope_wide_kernel<false, kRowsOne>)
                       : vec                ? (inter ? rope_wide_kernel<true, kRowsR> : rope_wide_kernel<false, kRowsR>)
                                            : (inter ? rope_any_kernel<true> : rope_any_kernel<false>);
  return launch_in_order(kernel, dim3(grid), kThreadsR, 0, st, 1, *rope, a) == cudaSuccess ? ZP_OK : ZP_ERR_CUDA;
}
