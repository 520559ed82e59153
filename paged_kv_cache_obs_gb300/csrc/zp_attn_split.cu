// zp_attn_split.cu — attention of a few query rows over a long paged cache, bf16 or E4M3, sm_103a:
// decode over the 8-bit pool, and decode (or a handful of new tokens) with a sliding window and
// first tokens that stay visible over the bf16 pool.
//
//   out[row] = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale <q_row, k_t>) over the t that the row sees
//
// The work is bound by the bytes of K and V; every byte is read once, straight from HBM into the
// registers from which the warp-level MMAs take it, with no shared memory on the way:
//   - S^T = K Q^T with the 16 tokens of a tile as the MMA's 16 rows and the query rows as its 8
//     columns.  The order of the contraction is free as long as K and Q agree, so a lane loads 16
//     contiguous bytes of a key and uses each 4 (or 8) of them in one k-step.
//   - O^T = V^T P^T with the values' dims as rows and tokens as the contraction.  A lane loads
//     contiguous dims of the 4 tokens that its A fragment holds; a byte permutation pairs two
//     tokens of a dim in a register.  Which dim a row of the product stands for is free too.
//   - P goes from the accumulator layout (a lane holds tokens) to the operand layout (a lane holds
//     a row) with movmatrix.
// E4M3 codes are converted to f16, which holds them exactly; queries are brought to f16 by a power
// of two per row, the block's K scale joins the logit scale, and its V scale multiplies the tile's
// own product, so scales of any size cost no precision.  P is f16 (11 bits; the accumulators and
// the sum are fp32).  With a bf16 pool P is a bf16 part plus a bf16 remainder (16 bits).
//
// The running maximum is kept lazily: a row's reference is raised only when a logit passes it by
// more than 8 (in log2), so that P stays below 2^8 and most tiles need one vote in place of
// reductions and rescaling.
//
// Grid (split, kv head, request), 4 warps a CTA; a split is a range of the request's visible
// 16-token tiles.  With more than one split the CTA that finishes a row last merges the partials in
// the order of the splits, so results do not depend on the order in which CTAs run.
#include "zp_attn.h"

#include <algorithm>

#include "zp_ptx.cuh"

namespace zp {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 16;                    // tokens
constexpr int kMaxTps = 32 * kWarps;         // a lane holds the block id of each of its warp's tiles
constexpr float kLazy = 8.0f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }
// the low and the high two E4M3 codes of a word, as f16 pairs
__device__ __forceinline__ void dec4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The pool is read once: loads that skip L1.
__device__ __forceinline__ uint4 ldg16(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ldg8(const uint8_t* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// What a (request, kv head) sees.
struct Span {
  int L, n, q0;      // tokens in the cache, queries, first row of q
  int p0;            // position of the first query
  int sink_tiles;    // list entries that are the cache's first tiles
  int win_tile;      // tile of list entry sink_tiles
  int tiles;         // list entries
};

// False: the request is skipped (`bad`: and reported).
__device__ __forceinline__ bool span_of(const AttnArgs& a, int r, Span& s, bool& bad) {
  s.L = a.seq_lens[r];
  s.q0 = r;
  s.n = 1;
  bad = false;
  if (a.q_start) {
    s.q0 = a.q_start[r];
    const int64_t n = static_cast<int64_t>(a.q_start[r + 1]) - s.q0;
    s.n = static_cast<int>(n);
    bad = s.q0 < 0 || n < 0 || n > a.max_q || s.q0 + n > a.T;
    if (!bad && n == 0) return false;
  }
  bad = bad || s.L < 0 || s.L > static_cast<int64_t>(a.max_blocks) * a.b || (a.q_start && s.n > s.L);
  if (bad) return false;
  s.p0 = max(0, s.L - s.n);
  const int first = a.window == 0 ? 0 : max(0, s.p0 - a.window + 1);
  s.win_tile = first / kTile;
  s.sink_tiles = min((min(a.sinks, s.L) + kTile - 1) / kTile, s.win_tile);
  s.tiles = s.sink_tiles + (s.L + kTile - 1) / kTile - s.win_tile;
  return true;
}

__device__ __forceinline__ void store_row4(const AttnArgs& a, const Span& s, int h, int row, int dim, const float (&v)[4]) {
  if (row >= a.G * s.n) return;
  const int i = row / a.G, g = row - i * a.G;
  uint16_t* const o = a.out + (s.q0 + i) * a.o_ts + (h * a.G + g) * a.o_hs + dim;
  const uint32_t lo = pack_bf16(v[0], v[1]), hi = pack_bf16(v[2], v[3]);
  if ((reinterpret_cast<uintptr_t>(o) & 7) == 0) {
    *reinterpret_cast<uint2*>(o) = make_uint2(lo, hi);
  } else {
    o[0] = static_cast<uint16_t>(lo);
    o[1] = static_cast<uint16_t>(lo >> 16);
    o[2] = static_cast<uint16_t>(hi);
    o[3] = static_cast<uint16_t>(hi >> 16);
  }
}

template <bool FP8, int D, int NT>
__global__ void __launch_bounds__(kThreads) split_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int ES = FP8 ? 1 : 2;              // bytes per value
  constexpr int ROWS = 8 * NT;
  constexpr int KC = D * ES / 64;              // 16-byte chunks of a key that a lane holds
  constexpr int KS = D / 16;                   // k-steps of S
  constexpr int MT = D / 16;                   // 16-dim row tiles of O^T
  constexpr int VW = D * ES / 32;              // words of a value row that a lane holds: 2, 4 or 8
  __shared__ float sm_m[kWarps][ROWS], sm_l[kWarps][ROWS];
  __shared__ __align__(16) float sm_acc[kWarps][ROWS][D];
  __shared__ int sm_last;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  const int split = blockIdx.x, h = blockIdx.y, r = blockIdx.z;
  Span s;
  bool bad;
  if (!span_of(a, r, s, bad)) {
    if (bad && split == 0 && h == 0 && tid == 0) atomicCAS(a.err, 0, ZP_ERR_BAD_TABLE);
    return;
  }
  const int ns = max(1, (s.tiles + a.tps - 1) / a.tps);
  if (split >= ns) return;
  const int tile0 = split * a.tps, tile1 = min(s.tiles, tile0 + a.tps);
  const int cnt = max(0, (tile1 - tile0 - warp + kWarps - 1) / kWarps);  // tiles of this warp

  // lane i: block id (and scales) of the warp's i-th tile
  const int tpb = a.b / kTile;
  int my_phys = 0, my_tile = 0;
  float my_ks = 0.0f, my_vs = 0.0f;
  bool my_bad = false;
  const int64_t layer_base = static_cast<int64_t>(a.layer) * a.num_blocks;
  if (lane < cnt) {
    const int li = tile0 + warp + kWarps * lane;
    my_tile = li < s.sink_tiles ? li : s.win_tile + li - s.sink_tiles;
    my_phys = a.tables[static_cast<int64_t>(r) * a.max_blocks + my_tile / tpb];
    my_bad = my_phys < 0 || my_phys >= a.num_blocks;
    if (FP8 && !my_bad) {
      const float* sc = a.scales + (layer_base + my_phys) * 2 * a.Hkv + h;
      my_ks = sc[0];
      my_vs = sc[a.Hkv];
    }
  }
  const bool cta_bad = __syncthreads_or(my_bad);
  if (cta_bad && tid == 0) atomicCAS(a.err, 0, ZP_ERR_BAD_TABLE);
  const int todo = cta_bad ? 0 : cnt;

  // queries as B fragments: column (row of the output) nt*8 + g
  uint32_t qb[NT][KS][2];
  float qs[NT][2];  // logit scale of columns nt*8 + 2c, +1
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row = nt * 8 + g;
    const bool have = row < a.G * s.n;
    const int i = have ? row / a.G : 0, gi = have ? row - i * a.G : 0;
    const uint16_t* const q = a.q + (s.q0 + i) * a.q_ts + (h * a.G + gi) * a.q_hs;
    // two values at dim e of the row (e even); queries may start at any 2-byte address
    const auto two = [&](int e) {
      return have ? static_cast<uint32_t>(q[e]) | static_cast<uint32_t>(q[e + 1]) << 16 : 0u;
    };
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      // 16-byte chunk c + 4j of a key: FP8 holds 4 k-steps, bf16 holds 2
      const int e = FP8 ? 16 * (c + 4 * (ks >> 2)) + 4 * (ks & 3) : 8 * (c + 4 * (ks >> 1)) + 4 * (ks & 1);
      qb[nt][ks][0] = two(e);
      qb[nt][ks][1] = two(e + 2);
    }
    float mult = 1.0f;
    if (FP8) {
      // to f16 by a power of two that brings the row's largest magnitude to [1, 2): values below
      // 2^-14 of it lose bits, far below what the fp32 sums hold
      uint32_t m = 0;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int e = 0; e < 2; ++e) m = max(m, max(qb[nt][ks][e] & 0x7FFFu, (qb[nt][ks][e] >> 16) & 0x7FFFu));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const int ex = min(max(static_cast<int>(m >> 7), 1), 253);  // biased exponent, both 2^+-(ex - 127) are normal
      const float inv = __uint_as_float(static_cast<uint32_t>(254 - ex) << 23);
      mult = __uint_as_float(static_cast<uint32_t>(ex) << 23);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int e = 0; e < 2; ++e) qb[nt][ks][e] = pack_f16(lo_f(qb[nt][ks][e]) * inv, hi_f(qb[nt][ks][e]) * inv);
    }
    qs[nt][0] = a.sl2 * __shfl_sync(0xffffffffu, mult, 8 * c);
    qs[nt][1] = a.sl2 * __shfl_sync(0xffffffffu, mult, 8 * c + 4);
  }

  float m[NT][2], l[NT][2], o[NT][MT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt][0] = m[nt][1] = -INFINITY;
    l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) o[nt][mt][0] = o[nt][mt][1] = o[nt][mt][2] = o[nt][mt][3] = 0.0f;
  }

  // K: rows g and g + 8 of the tile; V: tokens 2c, 2c+1, 2c+8, 2c+9
  uint4 kr[2][KC];
  uint32_t vr[4][VW];
  const int64_t head_bytes = static_cast<int64_t>(a.b) * D * ES;
  const auto tile_ptr = [&](int i) {
    const int phys = __shfl_sync(0xffffffffu, my_phys, i), tile = __shfl_sync(0xffffffffu, my_tile, i);
    return a.pool + ((layer_base + phys) * 2 * a.Hkv + h) * head_bytes + (tile % tpb) * (kTile * D * ES);
  };
  const auto load_k = [&](const uint8_t* p) {
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int j = 0; j < KC; ++j) kr[half][j] = ldg16(p + (g + 8 * half) * (D * ES) + (c + 4 * j) * 16);
  };
  const auto load_v = [&](const uint8_t* p) {
    p += a.Hkv * head_bytes;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint8_t* const row = p + (2 * c + (t & 1) + 8 * (t >> 1)) * (D * ES);
      if constexpr (VW == 2) {
        const uint2 x = ldg8(row + g * 8);
        vr[t][0] = x.x;
        vr[t][1] = x.y;
      } else {
#pragma unroll
        for (int j = 0; j < VW / 4; ++j) {
          const uint4 x = ldg16(row + (g + 8 * j) * 16);
          vr[t][4 * j] = x.x;
          vr[t][4 * j + 1] = x.y;
          vr[t][4 * j + 2] = x.z;
          vr[t][4 * j + 3] = x.w;
        }
      }
    }
  };
  const uint8_t* cur = nullptr;
  if (todo > 0) {
    cur = tile_ptr(0);
    load_k(cur);
    load_v(cur);
  }
  const int p_last = s.p0 + s.n - 1;
  for (int i = 0; i < todo; ++i) {
    const int t0 = __shfl_sync(0xffffffffu, my_tile, i) * kTile;
    const float ks_scale = FP8 ? __shfl_sync(0xffffffffu, my_ks, i) : 1.0f;
    const float vs_scale = FP8 ? __shfl_sync(0xffffffffu, my_vs, i) : 1.0f;
    const bool more = i + 1 < todo;
    const uint8_t* const next = more ? tile_ptr(i + 1) : nullptr;

    float x[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.0f;
#pragma unroll
    for (int j = 0; j < KC; ++j) {
      const uint32_t w0[4] = {kr[0][j].x, kr[0][j].y, kr[0][j].z, kr[0][j].w};
      const uint32_t w1[4] = {kr[1][j].x, kr[1][j].y, kr[1][j].z, kr[1][j].w};
      if constexpr (FP8) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t a0, a1, a2, a3;
          dec4(w0[w], a0, a2);
          dec4(w1[w], a1, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma<true>(x[nt], a0, a1, a2, a3, qb[nt][4 * j + w][0], qb[nt][4 * j + w][1]);
        }
      } else {
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma<false>(x[nt], w0[2 * w], w1[2 * w], w0[2 * w + 1], w1[2 * w + 1], qb[nt][2 * j + w][0], qb[nt][2 * j + w][1]);
      }
    }
    if (more) load_k(next);

#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[nt][e] *= qs[nt][e & 1] * ks_scale;
    // tokens t0 .. t0 + 15: seen by every row, or row by row
    const bool full = t0 + kTile - 1 <= s.p0 && (a.window == 0 || t0 > p_last - a.window || t0 + kTile <= a.sinks);
    if (!full) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = nt * 8 + 2 * c + (e & 1), t = t0 + g + (e >> 1) * 8;
          const int p = s.p0 + min(row / a.G, s.n - 1);
          if (!(t <= p && (a.window == 0 || t > p - a.window || t < a.sinks))) x[nt][e] = -INFINITY;
        }
      // values that no row sees: zero times anything must be zero
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int tt = t0 + 2 * c + (t & 1) + 8 * (t >> 1);
        if (!(tt <= p_last && (a.window == 0 || tt > s.p0 - a.window || tt < a.sinks))) {
#pragma unroll
          for (int w = 0; w < VW; ++w) vr[t][w] = 0;
        }
      }
    }
    bool raise = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) raise |= fmaxf(x[nt][e], x[nt][e + 2]) > m[nt][e] + kLazy;
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(x[nt][e], x[nt][e + 2]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          if (mx > m[nt][e]) {
            const float corr = ex2(m[nt][e] - mx);  // 0 from -inf
            m[nt][e] = mx;
            l[nt][e] *= corr;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              o[nt][mt][e] *= corr;
              o[nt][mt][e + 2] *= corr;
            }
          }
        }
    }
    uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float ref = m[nt][e & 1] == -INFINITY ? 0.0f : m[nt][e & 1];
        x[nt][e] = ex2(x[nt][e] - ref);
        l[nt][e & 1] += x[nt][e];
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (FP8) {
          ph[nt][e] = transpose8(pack_f16(x[nt][2 * e], x[nt][2 * e + 1]));
        } else {
          const uint32_t hi = pack_bf16(x[nt][2 * e], x[nt][2 * e + 1]);
          ph[nt][e] = transpose8(hi);
          pl[nt][e] = transpose8(pack_bf16(x[nt][2 * e] - lo_f(hi), x[nt][2 * e + 1] - hi_f(hi)));
        }
      }
    }
    bool redo = false;
    if (!FP8 && !full && s.n > 1) {
      // a value that some rows see and others do not must not reach the others as 0 * inf
      bool odd = false;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int w = 0; w < VW; ++w)
          odd |= (vr[t][w] & 0x7F80u) == 0x7F80u || (vr[t][w] & 0x7F800000u) == 0x7F800000u;
      redo = __any_sync(0xffffffffu, odd);
    }
    if (!FP8 && redo) {
      // plain products, token by token, for the rows that see it
      for (int tt = 0; tt < kTile; ++tt) {
        const uint8_t* const row = cur + a.Hkv * head_bytes + tt * (D * ES);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float pa = __shfl_sync(0xffffffffu, x[nt][e], (tt & 7) * 4 + c);
            const float pb = __shfl_sync(0xffffffffu, x[nt][e + 2], (tt & 7) * 4 + c);
            const float pt = tt < 8 ? pa : pb;
            const int p = s.p0 + min((nt * 8 + 2 * c + e) / a.G, s.n - 1), t = t0 + tt;
            if (t <= p && (a.window == 0 || t > p - a.window || t < a.sinks)) {
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(row + (g + 8 * (mt >> 2)) * 16 + (mt & 3) * 4);
                o[nt][mt][e] += pt * lo_f(w);
                o[nt][mt][e + 2] += pt * hi_f(w);
              }
            }
          }
      }
    } else if constexpr (FP8) {
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        const uint32_t l01 = __byte_perm(vr[0][w], vr[1][w], 0x5140), h01 = __byte_perm(vr[0][w], vr[1][w], 0x7362);
        const uint32_t l23 = __byte_perm(vr[2][w], vr[3][w], 0x5140), h23 = __byte_perm(vr[2][w], vr[3][w], 0x7362);
        uint32_t f[8];
        dec4(l01, f[0], f[1]);
        dec4(l23, f[2], f[3]);
        dec4(h01, f[4], f[5]);
        dec4(h23, f[6], f[7]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            mma<true>(y, f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3], ph[nt][0], ph[nt][1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][2 * w + k][e] = fmaf(y[e], vs_scale, o[nt][2 * w + k][e]);
          }
      }
    } else {
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        const uint32_t a0 = __byte_perm(vr[0][w], vr[1][w], 0x5410), a1 = __byte_perm(vr[0][w], vr[1][w], 0x7632);
        const uint32_t a2 = __byte_perm(vr[2][w], vr[3][w], 0x5410), a3 = __byte_perm(vr[2][w], vr[3][w], 0x7632);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma<false>(o[nt][w], a0, a1, a2, a3, ph[nt][0], ph[nt][1]);
          mma<false>(o[nt][w], a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
        }
      }
    }
    if (more) load_v(next);
    cur = next;
  }

  // the warps' sums, then the CTA's; lane (g, c) holds columns 2c, 2c+1 of its dims
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = nt * 8 + 2 * c + e;
      float sum = l[nt][e];
      sum += __shfl_xor_sync(0xffffffffu, sum, 4);
      sum += __shfl_xor_sync(0xffffffffu, sum, 8);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      if (g == 0) {
        sm_m[warp][row] = m[nt][e];
        sm_l[warp][row] = sum;
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        // FP8: dims (D/8) g + 2 mt, +1;  bf16: dims 8 (g + 8 (mt / 4)) + 2 (mt % 4), +1
        const int dim = FP8 ? (D / 8) * g + 2 * mt : 8 * (g + 8 * (mt >> 2)) + 2 * (mt & 3);
        *reinterpret_cast<float2*>(&sm_acc[warp][row][dim]) = make_float2(o[nt][mt][e], o[nt][mt][e + 2]);
      }
    }
  __syncthreads();
  const int rows = a.G * s.n;
  const int64_t unit = static_cast<int64_t>(r) * a.Hkv + h;
  float* const part = a.part + unit * a.max_splits * ROWS * (D + 2);  // [split][row][D sums, max, sum]
  for (int idx = tid; idx < rows * (D / 4); idx += kThreads) {
    const int row = idx / (D / 4), dim = (idx % (D / 4)) * 4;
    float M = -INFINITY, Ls = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w][row]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float mw = sm_m[w][row];
      // a warp without a maximum has sums of 0, or NaN if every logit was
      const float cw = mw == -INFINITY ? 1.0f : ex2(mw - M);
      const float4 y = *reinterpret_cast<const float4*>(&sm_acc[w][row][dim]);
      Ls += sm_l[w][row] * cw;
      v[0] += y.x * cw;
      v[1] += y.y * cw;
      v[2] += y.z * cw;
      v[3] += y.w * cw;
    }
    if (ns == 1) {
      if (cta_bad) continue;
      const float inv = Ls == 0.0f ? 0.0f : 1.0f / Ls;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] *= inv;
      store_row4(a, s, h, row, dim, v);
    } else {
      float* const p = part + (static_cast<int64_t>(split) * ROWS + row) * (D + 2);
      *reinterpret_cast<float2*>(p + dim) = make_float2(v[0], v[1]);
      *reinterpret_cast<float2*>(p + dim + 2) = make_float2(v[2], v[3]);
      if (dim == 0) {
        p[D] = cta_bad ? NAN : M;  // a maximum is never NaN: marks a split with a bad block id
        p[D + 1] = Ls;
      }
    }
  }
  if (ns == 1) return;
  __threadfence();
  __syncthreads();
  if (tid == 0) {
    const uint32_t before = atomicAdd(&a.done[unit], 1u);
    sm_last = before == static_cast<uint32_t>(ns - 1);
    if (sm_last) a.done[unit] = 0;  // as the next call expects it
  }
  __syncthreads();
  if (!sm_last) return;
  __threadfence();
  for (int idx = tid; idx < rows * (D / 4); idx += kThreads) {
    const int row = idx / (D / 4), dim = (idx % (D / 4)) * 4;
    const float* const p = part + static_cast<int64_t>(row) * (D + 2);
    const int64_t step = static_cast<int64_t>(ROWS) * (D + 2);
    float M = -INFINITY, Ls = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    bool skip = false;
    for (int k = 0; k < ns; ++k) {
      const float mk = __ldcg(p + k * step + D);
      skip |= isnan(mk);
      M = fmaxf(M, mk);
    }
    if (skip) continue;
    for (int k = 0; k < ns; ++k) {
      const float mk = __ldcg(p + k * step + D);
      const float ck = mk == -INFINITY ? 1.0f : ex2(mk - M);
      const float2 y0 = __ldcg(reinterpret_cast<const float2*>(p + k * step + dim));
      const float2 y1 = __ldcg(reinterpret_cast<const float2*>(p + k * step + dim + 2));
      Ls += __ldcg(p + k * step + D + 1) * ck;
      v[0] += y0.x * ck;
      v[1] += y0.y * ck;
      v[2] += y1.x * ck;
      v[3] += y1.y * ck;
    }
    const float inv = Ls == 0.0f ? 0.0f : 1.0f / Ls;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] *= inv;
    store_row4(a, s, h, row, dim, v);
  }
}

template <bool FP8, int D, int NT>
cudaError_t launch(const AttnArgs& a, cudaStream_t st) {
  split_kernel<FP8, D, NT><<<dim3(a.max_splits, a.Hkv, a.B), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <bool FP8>
cudaError_t dispatch(const AttnArgs& a, int d, int rows, cudaStream_t st) {
  if (d == 128) return rows == 8 ? launch<FP8, 128, 1>(a, st) : launch<FP8, 128, 2>(a, st);
  return rows == 8 ? launch<FP8, 64, 1>(a, st) : launch<FP8, 64, 2>(a, st);
}

}  // namespace

// CTAs that a launch aims at; a split is at least two tiles per warp and at most what lanes hold.
constexpr int64_t kTargetCtas = 152 * 6;
constexpr int kMinTps = 2 * kWarps;

SplitPlan split_plan(const zp_params* p, int B, int max_q, int64_t max_tokens, int window, int sinks) {
  SplitPlan s{};
  const int G = p->num_q_heads / p->num_kv_heads;
  s.rows = G * max_q <= 8 ? 8 : 16;
  int64_t tiles = (max_tokens + kTile - 1) / kTile;
  if (window > 0) {
    const int64_t seen = (static_cast<int64_t>(window) + max_q - 1 + kTile - 1) / kTile + 1 +
                         (static_cast<int64_t>(sinks) + kTile - 1) / kTile;
    tiles = std::min(tiles, seen);
  }
  const int64_t units = std::max<int64_t>(1, static_cast<int64_t>(B) * p->num_kv_heads);
  const int64_t want = (kTargetCtas + units - 1) / units;
  const int64_t even = ((tiles + want - 1) / want + kWarps - 1) / kWarps * kWarps;
  s.tps = static_cast<int>(std::min<int64_t>(std::max<int64_t>(even, kMinTps), kMaxTps));
  s.splits = static_cast<int>(std::max<int64_t>(1, (tiles + s.tps - 1) / s.tps));
  return s;
}

size_t split_bytes(const zp_params* p, int B, int max_q, int64_t max_tokens) {
  const int64_t units = std::max<int64_t>(1, static_cast<int64_t>(B) * p->num_kv_heads);
  const int64_t tiles = (max_tokens + kTile - 1) / kTile;
  // the most splits that split_plan gives to `tiles` or fewer
  const int64_t splits = std::min((tiles + kMinTps - 1) / kMinTps,
                                  std::max((kTargetCtas + units - 1) / units, (tiles + kMaxTps - 1) / kMaxTps));
  const int rows = p->num_q_heads / p->num_kv_heads * max_q <= 8 ? 8 : 16;
  size_t bytes = 256 + (static_cast<size_t>(units) * 4 + 255) / 256 * 256;
  if (splits > 1) bytes += static_cast<size_t>(units) * splits * rows * (p->head_dim + 2) * sizeof(float);
  return bytes;
}

zp_status split_launch(AttnArgs a, bool fp8, int head_dim, const SplitPlan& plan, void* workspace, cudaStream_t st) {
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  a.tps = plan.tps;
  a.max_splits = plan.splits;
  a.err = reinterpret_cast<int32_t*>(ws);
  a.done = reinterpret_cast<uint32_t*>(ws + 256);
  a.part = reinterpret_cast<float*>(ws + 256 + (static_cast<size_t>(a.B) * a.Hkv * 4 + 255) / 256 * 256);
  const cudaError_t e = fp8 ? dispatch<true>(a, head_dim, plan.rows, st) : dispatch<false>(a, head_dim, plan.rows, st);
  return e == cudaSuccess ? ZP_OK : ZP_ERR_CUDA;
}

}  // namespace zp
