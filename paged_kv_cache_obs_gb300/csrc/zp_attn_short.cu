// zp_attn_short.cu — attention of packed prompts that are short, over their own keys and values; sm_103a.
//
//   out[row] = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale <q_row, k_t>) over the t that the row sees
//
// A prompt of a hundred tokens is one tile for the tensor cores of zp_attn_tile.cuh, whose CTA fills an SM: its loads, products,
// softmax and stores follow one another, and nothing else is there to fill the gaps.  So here a CTA is small: 4 warps with 16
// rows each (queries times the heads of a group), 64 tokens of keys and values at a time in 48 KB, warp-level
// products, and four CTAs on an SM at different stages.  Bound by instructions (1670 a warp and tile were counted, 0.45 issued a
// cycle and scheduler, before masks, branches and the queries' addresses were made fewer: 64 prompts of 1 to 127 tokens, 32 heads on 8,
// 36 -> 31 us; with three CTAs an SM 34) and the latency of the chain: load, S, softmax, P V, store.
//
// Masks, weights (P rounded to bf16, sums and maxima fp32) and what a row does not see are as in the tiled kernel.  In a tile
// that some row does not see whole, values that are not finite would reach it as 0 * inf: such a tile, which the CTA
// looks for, is multiplied token by token.
#include "zp_attn.h"

#include "zp_launch.h"
#include "zp_ptx.cuh"

namespace zp {
namespace {

constexpr int kThreads = 128;
constexpr int kRows = 64;   // of a CTA
constexpr int kKeys = 64;   // of a tile

__device__ __forceinline__ void sts16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// 16 bytes, zeros where there is nothing to copy.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool have) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(have ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Byte offset of 16-byte chunk `ch` of row `row` of a tile of D columns: 8 rows of one chunk touch every bank once.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int row, int ch) {
  return row * (D * 2) + (((ch & ~7) | ((ch ^ row) & 7)) << 4);
}

// The thread's pieces of 64 rows: chunk `ch` of every kPer-th row from `row` on, `step` apart in memory.  Rows from `have` on are
// zeros; `any` is an address that a copy of nothing may name.
template <int D>
struct Pieces {
  static constexpr int kChunks = D / 8, kPer = kThreads / kChunks, N = 64 / kPer;  // kPer is a multiple of 8: the swizzle repeats
  int row, ch;
  uint32_t at;  // in shared memory
  __device__ __forceinline__ Pieces() : row(threadIdx.x / kChunks), ch(threadIdx.x % kChunks), at(chunk_at<D>(row, ch)) {}
  static constexpr uint32_t kStep = kPer * D * 2;
};
template <bool WIDE>
__device__ __forceinline__ void load_piece(uint32_t to, const uint16_t* from, bool have, const uint16_t* any) {
  if constexpr (WIDE) {
    copy16(to, have ? from : any, have);
  } else {
    uint32_t y[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (have) y[e] = static_cast<uint32_t>(from[2 * e]) | static_cast<uint32_t>(from[2 * e + 1]) << 16;
    sts16(to, make_uint4(y[0], y[1], y[2], y[3]));
  }
}
template <int D, bool WIDE>
__device__ __forceinline__ void load_tile(const Pieces<D>& p, uint32_t to, const uint16_t* base, int64_t step, int have) {
  const uint16_t* x = base + p.row * step + p.ch * 8;
#pragma unroll
  for (int u = 0; u < Pieces<D>::N; ++u) {
    load_piece<WIDE>(to + p.at + u * Pieces<D>::kStep, x, p.row + u * Pieces<D>::kPer < have, base);
    x += Pieces<D>::kPer * step;
  }
  if (WIDE) copies_end();
}

template <int D, bool WIDE>
__global__ void __launch_bounds__(kThreads, 4) short_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int kTile = 64 * D * 2;
  __shared__ __align__(128) uint8_t sm[3 * kTile];
  const uint32_t sq = smem_u32(sm), sk = sq + kTile, sv = sk + kTile;
  after_previous();
  next_may_start();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int r = blockIdx.z, h = blockIdx.y, per = kRows / a.G;  // queries of a CTA
  const int q0 = a.q_start[r];
  const int64_t n64 = static_cast<int64_t>(a.q_start[r + 1]) - q0;
  if (q0 < 0 || n64 < 0 || n64 > a.max_q || q0 + n64 > a.T) {
    if (blockIdx.x == 0 && h == 0 && tid == 0) atomicCAS(a.err, 0, ZP_ERR_BAD_TABLE);
    return;
  }
  const int n = static_cast<int>(n64), i0 = (static_cast<int>(gridDim.x) - 1 - static_cast<int>(blockIdx.x)) * per;  // long rows first
  if (i0 >= n) return;
  const int queries = min(per, n - i0), p_first = i0, p_last = i0 + queries - 1;
  const auto needed = [&](int t0) {  // some row sees some token of the tile
    return a.window == 0 || t0 + kKeys - 1 > p_first - a.window || t0 < a.sinks;
  };
  const auto next_tile = [&](int t0) {  // behind t0
    for (t0 += kKeys; t0 <= p_last && !needed(t0); t0 += kKeys) {
    }
    return t0;
  };
  const Pieces<D> mine;
  const uint16_t* const keys = a.k + static_cast<int64_t>(q0) * a.k_ts + h * a.k_hs;
  const uint16_t* const values = a.v + static_cast<int64_t>(q0) * a.v_ts + h * a.v_hs;
  const auto load_k = [&](int t) { load_tile<D, WIDE>(mine, sk, keys + t * a.k_ts, a.k_ts, n - t); };
  const auto load_v = [&](int t) { load_tile<D, WIDE>(mine, sv, values + t * a.v_ts, a.v_ts, n - t); };
  const int by_g = 65536 / a.G + 1;  // x / G is x * by_g >> 16 for x below 64
  int t0 = next_tile(-kKeys);
  {
    const uint16_t* const rows = a.q + static_cast<int64_t>(q0 + i0) * a.q_ts + static_cast<int64_t>(h * a.G) * a.q_hs;
    if (Pieces<D>::kPer % a.G == 0) {  // a fixed step from piece to piece
      const int i = mine.row * by_g >> 16, by = Pieces<D>::kPer * by_g >> 16;
      const uint16_t* x = rows + i * a.q_ts + (mine.row - i * a.G) * a.q_hs + mine.ch * 8;
      const int64_t step = by * a.q_ts;
#pragma unroll
      for (int u = 0; u < Pieces<D>::N; ++u) {
        load_piece<WIDE>(sq + mine.at + u * Pieces<D>::kStep, x, i + u * by < queries, a.q);
        x += step;
      }
    } else {
#pragma unroll
      for (int u = 0; u < Pieces<D>::N; ++u) {
        const int row = mine.row + u * Pieces<D>::kPer, i = row * by_g >> 16;
        load_piece<WIDE>(sq + mine.at + u * Pieces<D>::kStep, rows + i * a.q_ts + (row - i * a.G) * a.q_hs + mine.ch * 8, i < queries, a.q);
      }
    }
    if (WIDE) copies_end();
  }
  load_k(t0);
  load_v(t0);

  // where the lane's rows of the operands stand: 16 columns j of them at + off[j], or + off[j & 3] + 128 from the 64th on
  const int lo3 = lane & 7;
  const uint32_t qat = sq + (warp * 16 + (lane & 15)) * (D * 2), kat = sk + (((lane >> 4) << 3) + lo3) * (D * 2), vat = sv + (lane & 15) * (D * 2);
  uint32_t off_a[4], off_k[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    off_a[j] = ((2 * j + (lane >> 4)) ^ lo3) << 4;
    off_k[j] = ((2 * j + ((lane >> 3) & 1)) ^ lo3) << 4;
  }
  // the lane's rows: warp * 16 + g and 8 below
  int pos[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) pos[e] = i0 + min((warp * 16 + g + 8 * e) * by_g >> 16, queries - 1);
  const int p_warp = i0 + min((warp * 16 + 15) * by_g >> 16, queries - 1);  // the warp's last position
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f}, o[D / 8][4];
#pragma unroll
  for (int x = 0; x < D / 8; ++x) o[x][0] = o[x][1] = o[x][2] = o[x][3] = 0.0f;

  while (true) {
    const int next = next_tile(t0);
    const bool more = next <= p_last;
    // 16-token groups that some row of the warp may see: the others are left out
    const int groups = min(kKeys / 16, max(0, (p_warp - t0 + 16) >> 4));
    const bool whole = t0 + kKeys - 1 <= p_first && (a.window == 0 || t0 > p_last - a.window || t0 + kKeys <= a.sinks);
    copies_wait<1>();  // the queries and K, V may be on its way
    __syncthreads();
    float s[kKeys / 8][4];
#pragma unroll
    for (int x = 0; x < kKeys / 8; ++x) s[x][0] = s[x][1] = s[x][2] = s[x][3] = 0.0f;
    // two groups at a time, with the second's logits masked where no row sees it: a branch for each group and 16 dims cost more
#pragma unroll
    for (int y = 0; y < kKeys / 32; ++y) {
      if (2 * y >= groups) continue;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t qa[4];
        ldmatrix_x4(qat + off_a[ks & 3] + (ks >> 2) * 128, qa);
#pragma unroll
        for (int x = 2 * y; x < 2 * y + 2; ++x) {
          uint32_t kb[4];  // keys 16 x .. + 7 and + 8 .. + 15, dims 16 ks .. + 7 and + 8 .. + 15
          ldmatrix_x4(kat + off_k[ks & 3] + (ks >> 2) * 128 + x * (16 * D * 2), kb);
          mma_16816_bf16(s[2 * x], qa, kb[0], kb[1]);
          mma_16816_bf16(s[2 * x + 1], qa, kb[2], kb[3]);
        }
      }
    }
    // softmax; the tile's maximum joins the row's
    float top[2] = {-INFINITY, -INFINITY};
    if (!whole) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // columns up to `hi`, and above `lo` or below `sink`
        const int hi = pos[e] - t0 - 2 * c, lo = hi - a.window, sink = a.sinks - t0 - 2 * c;
#pragma unroll
        for (int x = 0; x < kKeys / 8; ++x) {
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            if (x * 8 + f > hi) s[x][2 * e + f] = -INFINITY;
          }
        }
        if (a.window == 0) continue;
#pragma unroll
        for (int x = 0; x < kKeys / 8; ++x) {
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const int col = x * 8 + f;
            if (col <= lo && col >= sink) s[x][2 * e + f] = -INFINITY;
          }
        }
      }
    }
#pragma unroll
    for (int x = 0; x < kKeys / 8; ++x) {
      if (x / 2 >= groups) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) top[e >> 1] = fmaxf(top[e >> 1], s[x][e]);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
      top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
      const float mn = fmaxf(m[e], top[e] * a.sl2), corr = m[e] == -INFINITY ? 0.0f : ex2(m[e] - mn), ref = mn == -INFINITY ? 0.0f : mn;
      if (t0 > 0) {
        l[e] *= corr;
#pragma unroll
        for (int x = 0; x < D / 8; ++x) {
          o[x][2 * e] *= corr;
          o[x][2 * e + 1] *= corr;
        }
      }
      m[e] = mn;
#pragma unroll
      for (int x = 0; x < kKeys / 8; ++x) {
        if (x / 2 >= groups) continue;  // 0, as they are
        s[x][2 * e] = ex2(fmaf(s[x][2 * e], a.sl2, -ref));
        s[x][2 * e + 1] = ex2(fmaf(s[x][2 * e + 1], a.sl2, -ref));
        l[e] += s[x][2 * e] + s[x][2 * e + 1];
      }
    }
    copies_wait<0>();
    bool odd = false;
    if (!whole) {  // values that are not finite: each thread looks at what it has copied
      uint32_t big = 0;
#pragma unroll
      for (int u = 0; u < Pieces<D>::N; ++u) {
        const uint4 x = lds16(sv + mine.at + u * Pieces<D>::kStep);
        big = max_u16x2(big, max_u16x2(max_u16x2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu), max_u16x2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
      }
      odd = (big & 0xFFFFu) >= 0x7F80u || big >= 0x7F800000u;
    }
    odd = __syncthreads_or(odd);  // and V is there, and K is free
    if (odd) {
      // token by token, P through K's place: the lane's dims (8 x + 2 c and the next) of its two rows
      float* const ps = reinterpret_cast<float*>(sm + kTile) + warp * 16 * kKeys / (D == 64 ? 2 : 1);  // 64-wide heads: half the tokens at a time
      constexpr int kHalf = D == 64 ? kKeys / 2 : kKeys;
#pragma unroll
      for (int half = 0; half < kKeys; half += kHalf) {
        __syncwarp();
#pragma unroll
        for (int x = half / 8; x < (half + kHalf) / 8; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) ps[(g + 8 * (e >> 1)) * kHalf + x * 8 - half + 2 * c + (e & 1)] = s[x][e];
        __syncwarp();
#pragma unroll 1
        for (int k = 0; k < kHalf; ++k) {
          const int t = t0 + half + k;
          if (t > p_last) break;
          float p[2];
          bool see[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            p[e] = ps[(g + 8 * e) * kHalf + k];
            see[e] = t <= pos[e] && (a.window == 0 || t > pos[e] - a.window || t < a.sinks);
          }
#pragma unroll
          for (int x = 0; x < D / 8; ++x) {
            const uint32_t v = *reinterpret_cast<const uint32_t*>(sm + 2 * kTile + chunk_at<D>(half + k, x) + c * 4);
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (see[e]) {
                o[x][2 * e] += p[e] * bf16x2_lo(v);
                o[x][2 * e + 1] += p[e] * bf16x2_hi(v);
              }
          }
        }
      }
      __syncthreads();
    }
    if (more) load_k(next);
    if (!odd) {
#pragma unroll
      for (int ks = 0; ks < kKeys / 16; ++ks) {
        if (ks >= groups) continue;
        const uint32_t pa[4] = {pack_bf16x2(s[2 * ks][0], s[2 * ks][1]), pack_bf16x2(s[2 * ks][2], s[2 * ks][3]),
                                pack_bf16x2(s[2 * ks + 1][0], s[2 * ks + 1][1]), pack_bf16x2(s[2 * ks + 1][2], s[2 * ks + 1][3])};
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          uint32_t vb[4];  // tokens 16 ks .. + 7 and + 8 .. + 15, dims 16 x .. + 7, then + 8 .. + 15
          ldmatrix_x4_trans(vat + off_a[x & 3] + (x >> 2) * 128 + ks * (16 * D * 2), vb);
          mma_16816_bf16(o[2 * x], pa, vb[0], vb[1]);
          mma_16816_bf16(o[2 * x + 1], pa, vb[2], vb[3]);
        }
      }
    }
    if (!more) break;
    __syncthreads();  // V is free
    load_v(next);
    t0 = next;
  }

  // rows through the queries' place (a warp's own), so that 16 bytes go out at a time
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
    const float inv = 1.0f / l[e];
#pragma unroll
    for (int x = 0; x < D / 8; ++x)
      *reinterpret_cast<uint32_t*>(sm + chunk_at<D>(warp * 16 + g + 8 * e, x) + c * 4) = pack_bf16x2(o[x][2 * e] * inv, o[x][2 * e + 1] * inv);
  }
  __syncwarp();
  constexpr int kChunks = D / 8;
#pragma unroll
  for (int u = 0; u < 16 * kChunks / 32; ++u) {
    const int at = u * 32 + lane, row = warp * 16 + at / kChunks, ch = at % kChunks, i = row * by_g >> 16;
    if (i >= queries) continue;
    const uint4 y = lds16(sq + chunk_at<D>(row, ch));
    uint16_t* const to = a.out + static_cast<int64_t>(q0 + i0 + i) * a.o_ts + (h * a.G + row - i * a.G) * a.o_hs + ch * 8;
    if ((reinterpret_cast<uintptr_t>(to) & 15) == 0) {
      *reinterpret_cast<uint4*>(to) = y;
    } else {
      const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        to[2 * e] = static_cast<uint16_t>(w[e]);
        to[2 * e + 1] = static_cast<uint16_t>(w[e] >> 16);
      }
    }
  }
}

}  // namespace

// Where this form is the faster one: prompts of up to 128 tokens, 256 with 64-wide heads, whose mean length is three quarters of that or
// less, or which leave the SMs' slots unfilled.  64 prompts, 32 heads on 8, d 128: of 1 to 32 tokens 11 us and 23 in the tiled form, of 1 to
// 127 tokens 31 and 41, of 96 tokens 40 and 44, of 112 tokens 48 and 46, of 128 tokens 56 and 47; one prompt of 128 tokens 6.5 us and 8.4.
// With d 64, 64 prompts, 16 heads on 2: of 128 tokens 19 us and 23, of 200 tokens 35 and 38, of 256 tokens 50 and 46.
bool short_prompts(const zp_params* p, int T, int B, int max_len) {
  const int64_t most = p->head_dim == 64 ? 256 : 128, per = kRows / (p->num_q_heads / p->num_kv_heads);
  const int64_t ctas = (max_len + per - 1) / per * p->num_kv_heads * B;
  return max_len <= most && (4 * static_cast<int64_t>(T) <= 3 * most * B || ctas <= 3 * plan_sms());
}

zp_status short_launch(AttnArgs a, const zp_params* p, int max_len, void* workspace, cudaStream_t st) {
  a.err = static_cast<int32_t*>(workspace);
  const auto fits = [](const uint16_t* x, int64_t ts, int64_t hs) { return aligned(x, 16) && ts % 8 == 0 && hs % 8 == 0; };
  const bool vec = fits(a.q, a.q_ts, a.q_hs) && fits(a.k, a.k_ts, a.k_hs) && fits(a.v, a.v_ts, a.v_hs);
  const int per = kRows / a.G;
  const dim3 grid(static_cast<unsigned>((max_len + per - 1) / per), static_cast<unsigned>(a.Hkv), static_cast<unsigned>(a.B));
  auto* const kernel = p->head_dim == 128 ? (vec ? short_kernel<128, true> : short_kernel<128, false>)
                                          : (vec ? short_kernel<64, true> : short_kernel<64, false>);
  return launch_in_order(kernel, grid, kThreads, 0, st, 1, a) == cudaSuccess ? ZP_OK : ZP_ERR_CUDA;
}

}  // namespace zp
