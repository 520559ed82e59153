// zp_attn_tile.cu — attention of many query rows with a sliding window and first tokens that stay
// visible, over the paged bf16 pool, on the 5th-generation tensor cores; sm_103a.
//
// A CTA holds 2 tiles of 128 query rows of one (request, kv head) — 128 / G queries times the G
// heads of the group, so K and V are read once for the whole group — and walks the 128-token
// tiles of the cache that any of its rows sees: first the blocks with always-visible first
// tokens, then the window's.  Blocks between the two are never loaded.
//
// Roles: a producer warp brings K and V through the block table (one TMA box per block and
// 64-column half, 128-byte swizzle, two-stage rings); an MMA warp issues S = Q K^T and
// O += P V with tcgen05; two groups of four warps (thread = row, one group per query tile) turn
// S into P.  S, P and O stay in TMEM: P (bf16) overwrites S and is the A operand of the second
// product, V its B operand with the dims contiguous.  While one tile's group works on its
// softmax, the tensor core multiplies for the other tile.
//
// The running maximum is kept lazily (raised only when a logit passes it by more than 8 in
// log2), so O is rescaled in TMEM rarely.  Sums and maxima are fp32; P is rounded to bf16 (off by
// at most 2^-9 of itself), as the second product's operand type asks.
//
// A tile in which some row does not see some token ("mixed": the diagonal, the window's edge, the
// first tokens, the list's end) takes the masked path.  There the softmax groups also look V over in
// shared memory: tokens that no row sees are zeroed, and if a value that only some rows see is not
// finite, the CTA's rows are computed again by a plain loop, so that 0 * inf never reaches a row
// that does not see it.
#include "zp_attn.h"

#include "zp_ptx.cuh"

namespace zp {
namespace {

constexpr int kRows = 128;            // rows of a query tile = TMEM lanes
constexpr int kKeys = 128;            // tokens of a KV tile
constexpr int kStages = 2;
constexpr int kProdWarp = 8, kMmaWarp = 9;
constexpr int kThreads = 320;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr float kLazy = 8.0f;
constexpr uint32_t kTmemCols = 512;   // S0 S1 O0 O1, 128 columns each

template <int D>
struct __align__(1024) TileSmem {
  uint8_t q[2][D / 64][kRows * 128];         // [tile][64-column half][row][128 B], 128-byte swizzle
  uint8_t k[kStages][D / 64][kKeys * 128];
  uint8_t v[kStages][D / 64][kKeys * 128];
  uint64_t q_full, k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  uint64_t s_full[2], p_full[2], o_full[2], v_clean, drain;
  uint32_t tmem;
  int abort, redo;
};

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
__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Waits for phase `parity` of `bar`; gives up (false) after the time limit, or when another role
// has given up.  A thread that gives up raises the flag.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const uint32_t addr = smem_u32(bar);
  if (mbar_try_wait(addr, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (mbar_try_wait(addr, parity)) return true;
    if (*abort) return false;
    if (globaltimer_ns() - t0 > kWaitNs) {
      *abort = 1;
      return false;
    }
  }
}

// D[tmem] (+)= A[tmem] * B[smem], issued by a single thread.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Shared-memory descriptor of an operand whose MN dimension is contiguous, 128-byte swizzle:
// 64-element (128-byte) rows, one per K index; 8 rows per 1024-byte atom, `mn_stride` bytes from
// one 64-element chunk of the MN dimension to the next.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t addr, uint32_t mn_stride) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(mn_stride >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}
constexpr uint32_t kTransposeB = 1u << 16;  // instruction descriptor: B is MN-major

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
      "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]),
      "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// What a CTA walks.
struct Walk {
  int L, n, q0, p0;        // tokens, queries, first row of q, position of the request's first query
  int i0, queries;         // first query of the CTA, how many
  int sink_blocks, win_block, blocks, tiles;
};

// Token of column `col` of list tile j.
__device__ __forceinline__ int token_of(const AttnArgs& a, const Walk& w, int j, int col) {
  const int e = j * kKeys + col, sink = w.sink_blocks * a.b;
  return e < sink ? e : w.win_block * a.b + e - sink;
}

__device__ __forceinline__ bool sees(const AttnArgs& a, int p, int t) {
  return t <= p && (a.window == 0 || t > p - a.window || t < a.sinks);
}

// Rows of the CTA by plain loops: one warp per row, a lane per token for the logits and a lane per
// dims for the sums.  For the rare inputs that the tiles cannot take.
template <int D>
__device__ __noinline__ void rows_plainly(const AttnArgs& a, const Walk& w, int r, int h, int warp, int lane) {
  constexpr int DL = D / 32;
  const int64_t tile_bytes = static_cast<int64_t>(a.b) * D;  // values of a (block, K|V, head)
  const uint16_t* const pool = reinterpret_cast<const uint16_t*>(a.pool);
  for (int rr = warp; rr < w.queries * a.G; rr += 8) {
    const int i = w.i0 + rr / a.G, g = rr % a.G, p = w.p0 + i;
    const uint16_t* const q = a.q + (w.q0 + i) * a.q_ts + (h * a.G + g) * a.q_hs;
    float m = -INFINITY, l = 0.0f, o[DL];
#pragma unroll
    for (int e = 0; e < DL; ++e) o[e] = 0.0f;
    for (int j = 0; j < w.tiles; ++j)
      for (int c0 = 0; c0 < kKeys; c0 += 32) {
        const int e = j * kKeys + c0 + lane, t = token_of(a, w, j, c0 + lane);
        const bool on = e < w.blocks * a.b && sees(a, p, t);
        float x = -INFINITY;
        const uint16_t* kv = nullptr;
        if (on) {
          const int64_t phys = a.tables[static_cast<int64_t>(r) * a.max_blocks + t / a.b];
          kv = pool + (((static_cast<int64_t>(a.layer) * a.num_blocks + phys) * 2 * a.Hkv + h) * tile_bytes) + (t % a.b) * D;
          x = 0.0f;
          for (int dd = 0; dd < D; ++dd) x = fmaf(lo_f(q[dd]), lo_f(kv[dd]), x);
          x *= a.sl2;
        }
        float mx = x;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
        const float mn = fmaxf(m, mx);
        const float ref = mn == -INFINITY ? 0.0f : mn;
        const float corr = m == -INFINITY ? 1.0f : ex2(m - ref);
        const float pt = on ? ex2(x - ref) : 0.0f;
        m = mn;
        l *= corr;
#pragma unroll
        for (int e2 = 0; e2 < DL; ++e2) o[e2] *= corr;
        uint32_t vote = __ballot_sync(0xffffffffu, on);
        while (vote) {
          const int src = __ffs(vote) - 1;
          vote &= vote - 1;
          const float ps = __shfl_sync(0xffffffffu, pt, src);
          const uint16_t* const vt = reinterpret_cast<const uint16_t*>(
              __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(kv), src)) + a.Hkv * tile_bytes;
          l += ps;
#pragma unroll
          for (int e2 = 0; e2 < DL; ++e2) o[e2] = fmaf(ps, lo_f(vt[lane * DL + e2]), o[e2]);
        }
      }
    uint16_t* const out = a.out + (w.q0 + i) * a.o_ts + (h * a.G + g) * a.o_hs;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int e = 0; e < DL; e += 2) {
      const uint32_t y = pack_bf16(o[e] * inv, o[e + 1] * inv);
      out[lane * DL + e] = static_cast<uint16_t>(y);
      out[lane * DL + e + 1] = static_cast<uint16_t>(y >> 16);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) tile_kernel(const __grid_constant__ CUtensorMap tm, const __grid_constant__ AttnArgs a) {
  constexpr int NH = D / 64;
  extern __shared__ uint8_t dyn[];
  TileSmem<D>& s = *reinterpret_cast<TileSmem<D>*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.y, r = blockIdx.z;
  const int qpt = kRows / a.G;  // queries per tile

  Walk w;
  w.L = a.seq_lens[r];
  w.q0 = a.q_start[r];
  const int64_t n64 = static_cast<int64_t>(a.q_start[r + 1]) - w.q0;
  bool bad = w.q0 < 0 || n64 < 0 || n64 > a.max_q || w.q0 + n64 > a.T;
  bad = bad || (n64 > 0 && (w.L < n64 || w.L > static_cast<int64_t>(a.max_blocks) * a.b));
  if (bad) {
    if (blockIdx.x == 0 && h == 0 && tid == 0) atomicCAS(a.err, 0, ZP_ERR_BAD_TABLE);
    return;
  }
  w.n = static_cast<int>(n64);
  w.i0 = (static_cast<int>(gridDim.x) - 1 - static_cast<int>(blockIdx.x)) * 2 * qpt;  // the last queries see the most
  if (w.i0 >= w.n) return;
  w.queries = min(2 * qpt, w.n - w.i0);
  w.p0 = w.L - w.n;
  const int p_first = w.p0 + w.i0, p_last = p_first + w.queries - 1;
  const int first = a.window == 0 ? 0 : max(0, p_first - a.window + 1);
  w.win_block = first / a.b;
  w.sink_blocks = min((min(a.sinks, w.L) + a.b - 1) / a.b, w.win_block);
  w.blocks = w.sink_blocks + p_last / a.b + 1 - w.win_block;
  w.tiles = (w.blocks * a.b + kKeys - 1) / kKeys;
  const bool two = w.queries > qpt;  // the second tile has rows

  bool bad_id = false;
  for (int e = tid; e < w.blocks; e += kThreads) {
    const int blk = e < w.sink_blocks ? e : w.win_block + e - w.sink_blocks;
    const int id = a.tables[static_cast<int64_t>(r) * a.max_blocks + blk];
    bad_id |= id < 0 || id >= a.num_blocks;
  }
  if (tid == 0) {
    mbar_init(&s.q_full, two ? 8 : 4);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.k_full[i], 1);
      mbar_init(&s.k_empty[i], 1);
      mbar_init(&s.v_full[i], 1);
      mbar_init(&s.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.p_full[i], 4);
      mbar_init(&s.o_full[i], 1);
    }
    mbar_init(&s.v_clean, two ? 8 : 4);
    mbar_init(&s.drain, 1);
    s.abort = 0;
    s.redo = 0;
    fence_mbar_init();
    prefetch_tensormap(&tm);
  }
  if (__syncthreads_or(bad_id)) {
    if (tid == 0) atomicCAS(a.err, 0, ZP_ERR_BAD_TABLE);
    return;
  }
  if (warp == kMmaWarp) tmem_alloc(&s.tmem, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = s.tmem;
  volatile int* const abort = &s.abort;
  const int bpt = kKeys / a.b;  // blocks per tile
  // some row of the CTA does not see some token of list tile j
  const auto mixed_tile = [&](int j) {
    const int t_lo = token_of(a, w, j, 0), t_hi = token_of(a, w, j, kKeys - 1);
    return !(t_hi - t_lo == kKeys - 1 && (j + 1) * kKeys <= w.blocks * a.b && t_hi <= p_first &&
             (a.window == 0 || t_lo > p_last - a.window || t_hi < a.sinks));
  };

  if (warp == kProdWarp) {
    int issued = 0;  // 2 j + 1 after K of tile j, 2 j + 2 after its V
    for (int j = 0; j < w.tiles; ++j) {
      const int st = j % kStages;
      const uint32_t ph = (j / kStages) & 1;
      const int nb = min(bpt, w.blocks - j * bpt);
      int z = 0;
      if (lane < nb) {
        const int e = j * bpt + lane, blk = e < w.sink_blocks ? e : w.win_block + e - w.sink_blocks;
        z = a.layer * static_cast<int>(a.num_blocks) + a.tables[static_cast<int64_t>(r) * a.max_blocks + blk];
      }
      bool go = true;
      for (int kv = 0; kv < 2 && go; ++kv) {
        uint64_t* const full = kv ? &s.v_full[st] : &s.k_full[st];
        if (lane == 0) {
          if (j >= kStages) go = wait(kv ? &s.v_empty[st] : &s.k_empty[st], ph ^ 1, abort);
          if (go) mbar_arrive_expect_tx(full, static_cast<uint32_t>(nb * a.b * D * 2));
        }
        go = __shfl_sync(0xffffffffu, go, 0);
        if (!go) break;
        if (lane < nb)
#pragma unroll
          for (int hd = 0; hd < NH; ++hd)
            tma_load_3d((kv ? s.v[st][hd] : s.k[st][hd]) + lane * a.b * 128, &tm, full, hd * 64, (kv * a.Hkv + h) * a.b, z);
        __syncwarp();
        issued = 2 * j + kv + 1;
      }
      if (!go) break;
    }
    // copies still in flight after a give-up land before the shared memory is released
    if (lane == 0 && *abort)
      for (int x = max(0, issued - 2 * kStages); x < issued; ++x) {
        const int j = x >> 1;
        mbar_wait_bounded((x & 1) ? &s.v_full[j % kStages] : &s.k_full[j % kStages], (j / kStages) & 1, kWaitNs);
      }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    if (lane == 0) {
      const uint32_t idesc_s = idesc_bf16_f32(kRows, kKeys);
      const uint32_t idesc_o = idesc_bf16_f32(kRows, D) | kTransposeB;
      const int nt = two ? 2 : 1;
      const auto issue_s = [&](int t, int st) {
        for (int kk = 0; kk < D / 16; ++kk)
          mma_bf16(tbase + t * kKeys, smem_desc_sw128(smem_u32(&s.q[t][kk >> 2][(kk & 3) * 32])),
                   smem_desc_sw128(smem_u32(&s.k[st][kk >> 2][(kk & 3) * 32])), idesc_s, kk > 0);
        mma_commit(&s.s_full[t]);
      };
      bool ok = wait(&s.q_full, 0, abort) && wait(&s.k_full[0], 0, abort);
      if (ok) {
        tc_fence_after();
        for (int t = 0; t < nt; ++t) issue_s(t, 0);
        mma_commit(&s.k_empty[0]);
      }
      uint32_t cleaned = 0;  // mixed tiles so far
      for (int j = 0; ok && j < w.tiles; ++j) {
        const int st = j % kStages, nst = (j + 1) % kStages;
        const bool more = j + 1 < w.tiles;
        ok = wait(&s.v_full[st], (j / kStages) & 1, abort);
        if (ok && mixed_tile(j)) ok = wait(&s.v_clean, cleaned++ & 1, abort);
        for (int t = 0; ok && t < nt; ++t) {
          ok = wait(&s.p_full[t], j & 1, abort);
          if (!ok) break;
          tc_fence_after();
          for (int kk = 0; kk < kKeys / 16; ++kk)
            mma_bf16_ts(tbase + 256 + t * 128, tbase + t * kKeys + kk * 8,
                        smem_desc_mn_sw128(smem_u32(&s.v[st][0][kk * 16 * 128]), kKeys * 128), idesc_o, j > 0 || kk > 0);
          if (t == nt - 1) mma_commit(&s.v_empty[st]);
          if (more) {
            if (t == 0) ok = wait(&s.k_full[nst], ((j + 1) / kStages) & 1, abort);
            if (!ok) break;
            tc_fence_after();
            issue_s(t, nst);
            if (t == nt - 1) mma_commit(&s.k_empty[nst]);
          } else {
            mma_commit(&s.o_full[t]);
          }
        }
      }
      // products still in flight after a give-up complete before TMEM is released
      if (!ok) {
        mma_commit(&s.drain);
        mbar_wait_bounded(&s.drain, 0, kWaitNs);
      }
    }
    __syncwarp();
  } else {
    const int t = warp >> 2, row = tid & 127;
    const int group = two ? 256 : 128;  // threads of the softmax groups
    if (t == 0 || two) {
      // the row's query into the swizzled tile; rows past the queries are zero
      const int qi = row / a.G, gi = row - qi * a.G;
      const int i = t * qpt + qi;  // query of the CTA
      const bool have = qi < qpt && i < w.queries;
      const int p = p_first + min(i, w.queries - 1);
      {
        const uint16_t* const q = have ? a.q + (w.q0 + w.i0 + i) * a.q_ts + (h * a.G + gi) * a.q_hs : a.q;
        const bool vec = (reinterpret_cast<uintptr_t>(q) & 15) == 0;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          uint4 x = make_uint4(0, 0, 0, 0);
          if (have) {
            if (vec) {
              x = *reinterpret_cast<const uint4*>(q + c * 8);
            } else {
              uint32_t y[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                y[e] = static_cast<uint32_t>(q[c * 8 + 2 * e]) | static_cast<uint32_t>(q[c * 8 + 2 * e + 1]) << 16;
              x = make_uint4(y[0], y[1], y[2], y[3]);
            }
          }
          *reinterpret_cast<uint4*>(&s.q[t][c >> 3][row * 128 + (((c & 7) ^ (row & 7)) << 4)]) = x;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.q_full);

      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t ts = tbase + lanes + t * kKeys, to = tbase + lanes + 256 + t * 128;
      float m = -INFINITY, l = 0.0f;
      bool ok = true;
      for (int j = 0; j < w.tiles; ++j) {
        const int st = j % kStages;
        const bool mixed = mixed_tile(j);
        ok = wait(&s.s_full[t], j & 1, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        uint32_t x[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32_issue(ts + c * 32, x[c]);
        tmem_wait_ld(x[0]);
        tmem_ld_dep(x[1]);
        tmem_ld_dep(x[2]);
        tmem_ld_dep(x[3]);
        if (mixed) {
          const int left = w.blocks * a.b - j * kKeys;  // columns that the list has
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const int col = c * 32 + e;
              if (!(col < left && sees(a, p, token_of(a, w, j, col)))) x[c][e] = __float_as_uint(-INFINITY);
            }
          // V: see the head of this file
          ok = wait(&s.v_full[st], (j / kStages) & 1, abort);
          bool odd = false;
          if (ok)
            for (int y = (t * 128 + row); y < kKeys * (D / 8); y += group) {
              const int col = y / (D / 8), c = y % (D / 8);
              uint4* const at = reinterpret_cast<uint4*>(&s.v[st][c >> 3][col * 128 + (((c & 7) ^ (col & 7)) << 4)]);
              const int tk = token_of(a, w, j, col);
              // the span of positions that see the token contains some row's
              const bool any = col < left && tk <= p_last && (a.window == 0 || tk > p_first - a.window || tk < a.sinks);
              if (!any) {
                *at = make_uint4(0, 0, 0, 0);
              } else {
                const uint4 v = *at;
                const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) odd |= (u[e] & 0x7F80u) == 0x7F80u || (u[e] & 0x7F800000u) == 0x7F800000u;
              }
            }
          if (odd) s.redo = 1;
          fence_proxy_async_smem();
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) mbar_arrive(&s.v_clean);
        }
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e) mx = fmaxf(mx, __uint_as_float(x[c][e]));
        mx *= a.sl2;
        if (__any_sync(0xffffffffu, mx > m + kLazy)) {
          const float mn = fmaxf(m, mx), corr = m == -INFINITY ? 0.0f : ex2(m - mn);
          if (j > 0) {  // O of the tiles so far, complete since s_full follows their products
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32_issue(to + c * 32, o);
              tmem_wait_ld(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
              tmem_st32(to + c * 32, o);
            }
          }
          l *= corr;
          m = mn;
        }
        const float ref = m == -INFINITY ? 0.0f : m;
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const uint32_t (&src)[32] = x[2 * c + (e >> 4)];
            const float y0 = ex2(fmaf(__uint_as_float(src[(2 * e) & 31]), a.sl2, -ref));
            const float y1 = ex2(fmaf(__uint_as_float(src[(2 * e + 1) & 31]), a.sl2, -ref));
            sum[e & 3] += y0 + y1;
            pk[e] = pack_bf16(y0, y1);
          }
          tmem_st32(ts + c * 32, pk);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.p_full[t]);
      }
      if (ok) ok = wait(&s.o_full[t], 0, abort);
      ok = __all_sync(0xffffffffu, ok);
      if (ok) {
        tc_fence_after();
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        uint16_t* const out = have ? a.out + (w.q0 + w.i0 + i) * a.o_ts + (h * a.G + gi) * a.o_hs : a.out;
        const bool vec = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32_issue(to + c * 32, o);
          tmem_wait_ld(o);
          if (have) {
            uint32_t y[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = pack_bf16(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
            if (vec) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                *reinterpret_cast<uint4*>(out + c * 32 + e * 8) = make_uint4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                out[c * 32 + 2 * e] = static_cast<uint16_t>(y[e]);
                out[c * 32 + 2 * e + 1] = static_cast<uint16_t>(y[e] >> 16);
              }
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && s.abort) atomicCAS(a.err, 0, ZP_ERR_TIMEOUT);
  if (warp == kMmaWarp) tmem_dealloc(tbase, kTmemCols);
  if (s.redo && !s.abort && warp < 8) rows_plainly<D>(a, w, r, h, warp, lane);
}

static_assert(sizeof(TileSmem<128>) + 1024 <= 227 * 1024, "shared memory of one CTA");

template <int D>
cudaError_t launch(const CUtensorMap& tm, const AttnArgs& a, cudaStream_t st) {
  constexpr int bytes = sizeof(TileSmem<D>) + 1024;
  static PerDeviceInit attrs;
  const cudaError_t e = attrs.run(
      [] { return cudaFuncSetAttribute(tile_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); });
  if (e != cudaSuccess) return e;
  const int per_cta = 2 * (kRows / a.G);
  tile_kernel<D><<<dim3((a.max_q + per_cta - 1) / per_cta, a.Hkv, a.B), kThreads, bytes, st>>>(tm, a);
  return cudaGetLastError();
}

}  // namespace

zp_status tile_launch(AttnArgs a, const zp_kv_pool* pool, const zp_params* p, void* workspace, cudaStream_t st) {
  a.err = static_cast<int32_t*>(workspace);
  const int d = p->head_dim;
  CUtensorMap tm;
  // the pool as {d, 2*Hkv*b rows per (layer, block), layers*num_blocks}; box = one block's b rows
  // of one (K or V, head), 64 columns
  if (!encode_tmap_3d_bf16(&tm, pool->base, d, static_cast<uint64_t>(2) * a.Hkv * a.b,
                           static_cast<uint64_t>(p->num_layers) * pool->num_blocks, static_cast<uint64_t>(d) * 2,
                           static_cast<uint64_t>(2) * a.Hkv * a.b * d * 2, 64, a.b, 1))
    return ZP_ERR_CUDA;
  const cudaError_t e = d == 128 ? launch<128>(tm, a, st) : launch<64>(tm, a, st);
  return e == cudaSuccess ? ZP_OK : ZP_ERR_CUDA;
}

}  // namespace zp
