// zp_attn_split.cu — attention of a few query rows over a long paged cache, bf16 or E4M3, sm_103a:
// decode over the 8-bit pool, and decode (or a handful of new tokens) with a sliding window and
// first tokens that stay visible over the bf16 pool.
//
//   out[row] = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale <q_row, k_t>) over the t that the row sees
//
// The work is bound by the bytes of K and V.  Every warp streams its tiles of 16 tokens through a
// ring of its own (TMA, one box each for K and V, completing on the stage's mbarrier) and multiplies
// with the warp-level MMAs, whose operands come from plain 16-byte shared loads:
//   - S^T = K Q^T with the 16 tokens of a tile as the MMA's 16 rows and the query rows as its 8
//     columns.  The order of the contraction is free as long as K and Q agree, so a lane takes 16
//     contiguous bytes of a key and uses each 4 (or 8) of them in one k-step.
//   - O^T = V^T P^T with the values' dims as rows and tokens as the contraction.  A lane takes
//     contiguous dims of the 4 tokens that its A fragment holds; a byte permutation pairs two
//     tokens of a dim in a register.  Which dim a row of the product stands for is free too.
//   - P goes from the accumulator layout (a lane holds tokens) to the operand layout (a lane holds
//     a row) with movmatrix.
// E4M3 codes are converted to f16, which holds them exactly; queries are brought to f16 by a power
// of two per row, the block's K scale joins the logit scale, and its V scale multiplies P or the tile's
// own product, so that scales of any size cost no precision.  P is f16 (11 bits; the accumulators and
// the sum are fp32).  With a bf16 pool P is a bf16 part plus a bf16 remainder (off by at most 2^-16).  The part
// is P cut off and P's lowest bit is set, so that the remainder of a weight is above 0 as well: both times
// an infinite value are that infinity (a remainder of 0 or below made it NaN).  Weights below 2^-103 have
// no room for it.
//
// The running maximum is kept lazily: a row's reference is set 8 (in log2) above the largest logit so far,
// and again only when a logit passes it, so that most tiles need one vote in place of reductions and
// rescaling.  P is at most 1, so sums over V overflow no earlier than the weighted sum itself.
//
// Grid (split, kv head, request), 4 warps a CTA; a row's visible 16-token tiles are dealt evenly
// over its splits.  Up to 8 splits are one thread-block cluster, which joins its sums through
// distributed shared memory; with more, each cluster leaves one part, and a second kernel joins
// the parts.  Both join in the order of the splits, so results do not depend on the order in which
// CTAs run, and nothing in the workspace has to be zero.
//
// Measured (one layer): 8 requests of 100000 to 131072 E4M3 tokens, 28 heads on 4, d 128: 160 us, 5.9
// TB/s; 224 requests of 1 to 2048, 32 heads on 8: 84 us, 5.6 TB/s; 64 requests that see 1028 bf16 tokens
// of 8 heads: 45 us, 5.6 TB/s.  The long case fills 54 % of its
// issue slots, many of them with turning codes into f16; the warp-level MMA that takes E4M3 operands
// ran 20 % more instructions in all and was slower.
#include "zp_attn.h"

#include <algorithm>
#include <climits>

#include "zp_launch.h"
#include "zp_ptx.cuh"

namespace zp {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 16;                    // tokens
constexpr float kLazy = 8.0f;
constexpr float kGain = 32768.0f;            // E4M3: what P is multiplied by for f16
constexpr float kLeastRef = 3.85185989e-34f;  // 2^-111: kGain over a V scale and a scale over kGain are normal numbers

// x + y, where subnormal numbers count as 0
__device__ __forceinline__ float add_ftz(float x, float y) {
  float z;
  asm("add.rn.ftz.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
  return z;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
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
// c (16x8 fp32) = or += a (16x16) * b (16x8), f16 or bf16
template <bool F16, bool ADD = true>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  const float z[4] = {ADD ? c[0] : 0.0f, ADD ? c[1] : 0.0f, ADD ? c[2] : 0.0f, ADD ? c[3] : 0.0f};
  if (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(z[0]), "f"(z[1]), "f"(z[2]), "f"(z[3]));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(z[0]), "f"(z[1]), "f"(z[2]), "f"(z[3]));
}

__device__ __forceinline__ uint2 lds8(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float ld_cluster_f1(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// Token of a tile that stands in row (and, for V, contraction index) k of the products.  With
// 128-byte rows under the 128-byte swizzle this order lets the 16-byte loads of K (rows 2i and
// 2i+1 together) and of V (rows 0, 2, 4, 6 or 1, 3, 5, 7 together) touch every bank once.
__device__ __forceinline__ int token_at(int k) { return k ^ ((k & 1) << 2); }

// Byte offset of 16-byte chunk `ch` of row `row` of a tile of 16 rows of RB bytes, as the TMA
// stores it: 128-byte swizzle, rows above 128 bytes as two halves; 64-byte swizzle for 64.
template <int RB>
__device__ __forceinline__ uint32_t chunk_at(int row, int ch) {
  if constexpr (RB == 64) return row * 64 + ((ch ^ ((row >> 1) & 3)) << 4);
  return (ch >> 3) * (kTile * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4);
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

// The request that comes z-th when the long ones come first: in four classes by the quarters of the
// longest, in their own order within a class.  Every CTA finds its own (as many ballots as 32 requests
// a class, and one scan), so nothing is shared between CTAs.
constexpr int kMaxOrdered = 1024;
__device__ __forceinline__ int request_at(const AttnArgs& a, int z, uint32_t* words, int* tops) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kMost = 1 << 30;  // above any length that is taken
  int mx = 0;
  for (int i = tid; i < a.B; i += kThreads) mx = max(mx, min(a.seq_lens[i], kMost));
  mx = __reduce_max_sync(0xffffffffu, mx);
  if (lane == 0) tops[warp] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) mx = max(mx, tops[w]);
  const int step = mx / 4 + 1, nw = (a.B + kThreads - 1) / kThreads * kWarps;  // words of a class
  for (int base = 0; base < a.B; base += kThreads) {
    const int v = base + tid < a.B ? min(a.seq_lens[base + tid], kMost) : 0;
    const int k = (v >= step) + (v >= 2 * step) + (v >= 3 * step);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t vote = __ballot_sync(0xffffffffu, base + tid < a.B && k == 3 - c);
      if (lane == 0) words[c * nw + base / 32 + warp] = vote;
    }
  }
  __syncthreads();
  for (int w0 = 0;; w0 += 32) {
    uint32_t word = w0 + lane < 4 * nw ? words[w0 + lane] : 0;
    const int n = __popc(word);
    int sum = n;
#pragma unroll
    for (int x = 1; x < 32; x *= 2) {
      const int y = __shfl_up_sync(0xffffffffu, sum, x);
      if (lane >= x) sum += y;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, sum > z);
    if (past == 0 && w0 + 32 < 4 * nw) {
      z -= __shfl_sync(0xffffffffu, sum, 31);
      continue;
    }
    const int at = __ffs(past) - 1;
    word = __shfl_sync(0xffffffffu, word, at);
    for (int skip = z - __shfl_sync(0xffffffffu, sum - n, at); skip > 0; --skip) word &= word - 1;
    return (w0 + at) % nw * 32 + __ffs(word) - 1;
  }
}

// v and l += another part's sums, brought from its maximum to M.  A part without a maximum has sums of
// 0, or NaN if every logit was.
__device__ __forceinline__ void join(float (&v)[4], float& l, float4 y, float yl, float ym, float M) {
  const float w = ym == -INFINITY ? 1.0f : ex2(ym - M);
  l = fmaf(yl, w, l);
  v[0] = fmaf(y.x, w, v[0]);
  v[1] = fmaf(y.y, w, v[1]);
  v[2] = fmaf(y.z, w, v[2]);
  v[3] = fmaf(y.w, w, v[3]);
}

// Four dims of an output row: sums over the sum of weights.  A row whose logits are all -inf has weights
// of 0 alone, and is 0 / 0 like the softmax of them.
__device__ __forceinline__ void store_row4(const AttnArgs& a, const Span& s, int h, int row, int dim, const float (&v)[4], float l) {
  const int i = row / a.G, g = row - i * a.G;
  uint16_t* const o = a.out + (s.q0 + i) * a.o_ts + (h * a.G + g) * a.o_hs + dim;
  const float inv = 1.0f / l;
  const uint32_t lo = pack_bf16x2(v[0] * inv, v[1] * inv), hi = pack_bf16x2(v[2] * inv, v[3] * inv);
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
struct Shape {
  static constexpr int ES = FP8 ? 1 : 2;                  // bytes per value
  static constexpr int RB = D * ES;                       // bytes of a row
  static constexpr int ROWS = 8 * NT;
  static constexpr int TILE = kTile * RB;                 // bytes of K (or V) of a tile
  static constexpr int SUB = RB <= 64 ? 2 : 1;            // tiles that a warp takes at a time
  static constexpr int HALF = SUB * TILE;                 // K or V of what a warp takes at a time
  // A warp's ring has slots of K and V together (one wait for both); but rows of 256 bytes in three
  // slots of K or V, which leaves room for a fourth CTA on the SM (64 requests with a window of 1024:
  // 50 -> 44 us; with E4M3 rows the further waits cost 5 %).
  static constexpr bool JOINT = RB < 256 || NT == 2;
  static constexpr int SLOTS = JOINT ? 2 : 3;
  static constexpr int SLOT = (JOINT ? 2 : 1) * HALF;
  static constexpr int RING = kWarps * SLOTS * SLOT;
  static constexpr int ACC = kWarps * ROWS * D * 4;       // the warps' sums, in the ring's place
  static constexpr int SMEM = (RING > ACC ? RING : ACC) + 1024;
  // CTAs of an SM: what shared memory and, with 16 rows, registers hold
  static constexpr int CTAS = NT == 2 ? (D == 128 ? 2 : 3) : 4;
};

// Where 16-byte chunk `ch` of a row's sums stands: spread so that neither the warps' writes nor the
// joining reads meet in a bank.
template <bool FP8>
__device__ __forceinline__ int acc_at(int row, int ch) {
  const int c = (row >> 1) & 3;
  return ch ^ (FP8 ? c : (c & 1) | (c & 2) << 1);
}

template <bool FP8, int D, int NT>
__global__ void __launch_bounds__(kThreads, (Shape<FP8, D, NT>::CTAS)) split_kernel(const __grid_constant__ CUtensorMap tm, const __grid_constant__ AttnArgs a) {
  using Sh = Shape<FP8, D, NT>;
  constexpr int ROWS = Sh::ROWS, RB = Sh::RB, SLOTS = Sh::SLOTS, TILE = Sh::TILE, SUB = Sh::SUB;
  constexpr int KC = RB / 64;                  // 16-byte chunks of a key that a lane holds
  constexpr int KS = D / 16;                   // k-steps of S
  constexpr int MT = D / 16;                   // 16-dim row tiles of O^T
  constexpr int VW = RB / 32;                  // words of a value row that a lane holds: 2, 4 or 8
  __shared__ float sm_m[kWarps][ROWS], sm_l[kWarps][ROWS], cta_m[ROWS], cta_l[ROWS];
  __shared__ __align__(8) uint64_t full[kWarps][SLOTS + 1];  // and one that nothing completes, for the test hook
  __shared__ int sm_bad;
  __shared__ uint32_t words[4 * kMaxOrdered / 32];
  __shared__ int tops[kWarps];
  extern __shared__ uint8_t dyn[];
  uint8_t* const ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  if (tid == 0) {
    prefetch_tensormap(&tm);
    sm_bad = 0;
  }
  if (lane == 0) {
    for (int i = 0; i <= SLOTS; ++i) mbar_init(&full[warp][i], 1);
    fence_mbar_init();
  }
  after_previous();
  next_may_start();
  const int split = blockIdx.x, h = blockIdx.y;
  const int r = a.ordered ? request_at(a, blockIdx.z, words, tops) : blockIdx.z;
  const int bshift = a.b == 2 * kTile ? 1 : 0;  // tiles per block, as a shift
  const int32_t* const table = a.tables + static_cast<int64_t>(r) * a.max_blocks;
  const int first = split * kWarps + warp;  // the warp's first group of SUB tiles
  // Without a window the warp's tiles do not depend on the row's length, and their block ids are on
  // their way together with it.
  const bool early = a.window == 0;
  int early_id = 0;
  if (early) {
    const int64_t blk = ((first + static_cast<int64_t>(lane / SUB) * (a.splits * kWarps)) * SUB + lane % SUB) >> bshift;
    if (blk < a.max_blocks) early_id = table[blk];
  }
  Span s;
  bool bad;
  if (!span_of(a, r, s, bad)) {  // the same for every CTA of the cluster
    if (bad && split == 0 && h == 0 && tid == 0) atomicCAS(a.err, 0, ZP_ERR_BAD_TABLE);
    return;
  }
  if (s.L == 0) {  // a padded row: zeros
    if (split == 0)
      for (int i = tid; i < a.G * D; i += kThreads) a.out[s.q0 * a.o_ts + (h * a.G + i / D) * a.o_hs + i % D] = 0;
    return;
  }
  // the row's tiles are dealt out one by one to the warps of its splits
  const int stride = a.splits * kWarps;
  const int groups = (s.tiles + SUB - 1) / SUB;
  const int todo = max(0, (groups - first + stride - 1) / stride);  // groups of SUB tiles of this warp

  __syncthreads();

  // Lane i holds the block id (and scales) of tile i of the warp's list, 32 tiles at a time, and the
  // next 32 besides.  An id outside the pool is reported, and block 0 read in its place.
  constexpr int BATCH = 32 / SUB;  // groups whose ids a warp holds
  const int64_t layer_base = static_cast<int64_t>(a.layer) * a.num_blocks;
  const auto tile_of = [&](int i, int sub) {  // tile of the cache; past the list's end: >= 2^30
    const int li = (first + stride * i) * SUB + sub;
    return li < s.sink_tiles ? li : li < s.tiles ? s.win_tile + li - s.sink_tiles : 1 << 30;
  };
  int phys[2] = {0, 0};
  float kscale[2] = {0.0f, 0.0f}, vscale[2] = {0.0f, 0.0f};
  bool bad_id = false;
  const auto load_ids = [&](int n) {
    const int tile = tile_of(n * BATCH + lane / SUB, lane % SUB);
    int id = 0;
    if (tile < 1 << 30) id = (early && n == 0) ? early_id : table[tile >> bshift];
    const bool out = id < 0 || id >= a.num_blocks;
    bad_id |= out;
    id = out ? 0 : id;
    if (n & 1) phys[1] = id;
    else phys[0] = id;
  };
  const auto load_scales = [&](int n) {
    if (!FP8) return;
    const float* const sc = a.scales + (layer_base + ((n & 1) ? phys[1] : phys[0])) * 2 * a.Hkv + h;
    const float x = sc[0], y = sc[a.Hkv];
    if (n & 1) kscale[1] = x, vscale[1] = y;
    else kscale[0] = x, vscale[0] = y;
  };
  uint8_t* const my_ring = ring + warp * (SLOTS * Sh::SLOT);
  // The pool is the tensor {d, 2 Hkv b rows, layers * blocks}: K rows of head h start at h b, V rows
  // at (Hkv + h) b.
  // What fills slot after slot: fill n is group n, or K (n even) or V of group n / 2.
  constexpr int FILLS = Sh::JOINT ? 1 : 2;  // of a group
  const auto issue = [&](int n, int slot) {
    const int i = n / FILLS;
    int id[SUB];
#pragma unroll
    for (int sub = 0; sub < SUB; ++sub)
      id[sub] = __shfl_sync(0xffffffffu, ((i / BATCH) & 1) ? phys[1] : phys[0], (i % BATCH) * SUB + sub);
    if (lane == 0) {
      uint64_t* const bar = &full[warp][slot];
      const bool all = SUB == 1 || tile_of(i, SUB - 1) < 1 << 30;  // the list's last group may be short
      mbar_arrive_expect_tx(bar, (all ? SUB : 1) * (2 / FILLS) * TILE);
#pragma unroll
      for (int sub = 0; sub < SUB; ++sub) {
        if (sub > 0 && !all) break;
        const int row = h * a.b + (bshift ? (tile_of(i, sub) & 1) * kTile : 0), z = static_cast<int>(layer_base) + id[sub];
#pragma unroll
        for (int kv = 0; kv < 2 / FILLS; ++kv) {
          uint8_t* const to = my_ring + slot * Sh::SLOT + kv * Sh::HALF + sub * TILE;
          const int r0 = (Sh::JOINT ? kv : n & 1) ? a.Hkv * a.b + row : row;
#pragma unroll
          for (int hd = 0; hd < (RB > 128 ? 2 : 1); ++hd) tma_load_3d(to + hd * kTile * 128, &tm, bar, hd * 64, r0, z);
        }
      }
    }
  };
  load_ids(0);
  for (int n = 0; n < SLOTS && n < FILLS * todo; ++n) issue(n, n);
  load_scales(0);

  // queries as B fragments: column (row of the output) nt*8 + g
  uint32_t qb[NT][KS][2];
  float qs[NT][2];  // logit scale of columns nt*8 + 2c, +1
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row = nt * 8 + g;
    const bool have = row < a.G * s.n;
    const int i = have ? row / a.G : 0, gi = have ? row - i * a.G : 0;
    const uint16_t* const q = a.q + (s.q0 + i) * a.q_ts + (h * a.G + gi) * a.q_hs;
    // the lane's 16-byte chunk c + 4j of a key holds 4 k-steps (E4M3) or 2 (bf16)
    if (!have) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) qb[nt][ks][0] = qb[nt][ks][1] = 0;
    } else if ((reinterpret_cast<uintptr_t>(q) & 15) == 0) {
#pragma unroll
      for (int v = 0; v < KS / 2; ++v) {  // 8 values
        const int e = FP8 ? 16 * (c + 4 * (v >> 1)) + 8 * (v & 1) : 8 * (c + 4 * v);
        const uint4 x = *reinterpret_cast<const uint4*>(q + e);
        qb[nt][2 * v][0] = x.x;
        qb[nt][2 * v][1] = x.y;
        qb[nt][2 * v + 1][0] = x.z;
        qb[nt][2 * v + 1][1] = x.w;
      }
    } else {  // queries may start at any 2-byte address
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int e = FP8 ? 16 * (c + 4 * (ks >> 2)) + 4 * (ks & 3) : 8 * (c + 4 * (ks >> 1)) + 4 * (ks & 1);
        qb[nt][ks][0] = static_cast<uint32_t>(q[e]) | static_cast<uint32_t>(q[e + 1]) << 16;
        qb[nt][ks][1] = static_cast<uint32_t>(q[e + 2]) | static_cast<uint32_t>(q[e + 3]) << 16;
      }
    }
    float mult = 1.0f;
    if (FP8) {
      // to f16 by a power of two that brings the row's largest magnitude to [2^14, 2^15): exact for values
      // down to 2^-31 of it (8 bits fit f16's subnormals from 2^-17 on), less than the fp32 sums hold
      uint32_t m = 0;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int e = 0; e < 2; ++e) m = max(m, max(qb[nt][ks][e] & 0x7FFFu, (qb[nt][ks][e] >> 16) & 0x7FFFu));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const int ex = min(max(static_cast<int>(m >> 7), 15), 253);  // biased exponent, both 2^+-(ex - 141) are normal
      const float inv = __uint_as_float(static_cast<uint32_t>(268 - ex) << 23);
      mult = __uint_as_float(static_cast<uint32_t>(ex - 14) << 23);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int e = 0; e < 2; ++e) qb[nt][ks][e] = pack_f16(bf16x2_lo(qb[nt][ks][e]) * inv, bf16x2_hi(qb[nt][ks][e]) * inv);
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

  const int p_last = s.p0 + s.n - 1;
  float vref = 0.0f, vinv = 0.0f;  // FP8: V scale that o is in units of (over kGain), and its inverse
  bool ok = true;
  int fill = 0;                    // the fill that comes next
  int slot = a.stall ? SLOTS : 0;  // its slot; the test hook starts at the barrier that nothing completes
  uint32_t phase = 0;      // of the ring's current round
  // waits for it, and what follows its last use
  const auto arrived = [&] { return __all_sync(0xffffffffu, mbar_wait_bounded(&full[warp][slot], phase, a.limit_ns)) != 0; };
  const auto used = [&] {
    __syncwarp();  // every lane has read it
    if (fill + SLOTS < FILLS * todo) issue(fill + SLOTS, slot);
    ++fill;
    if (++slot == SLOTS) slot = 0, phase ^= 1;
  };
  for (int i = 0; i < todo; ++i) {
    if (i % BATCH == 0 && i + BATCH < todo) load_ids(i / BATCH + 1);
    if (i % BATCH == BATCH / 4 && i - BATCH / 4 + BATCH < todo) load_scales(i / BATCH + 1);
    float ks[SUB], vs[SUB];
#pragma unroll
    for (int sub = 0; sub < SUB; ++sub) {
      const int src = (i % BATCH) * SUB + sub;
      ks[sub] = FP8 ? __shfl_sync(0xffffffffu, ((i / BATCH) & 1) ? kscale[1] : kscale[0], src) : 1.0f;
      vs[sub] = FP8 ? __shfl_sync(0xffffffffu, ((i / BATCH) & 1) ? vscale[1] : vscale[0], src) : 1.0f;
    }
    ok = arrived();
    if (!ok) break;
    const uint32_t kbuf = smem_u32(my_ring + slot * Sh::SLOT);

    // S^T, tokens of rows g and g + 8 of each tile's product
    float x[SUB][NT][4];
#pragma unroll
    for (int sub = 0; sub < SUB; ++sub) {
#pragma unroll
      for (int j = 0; j < KC; ++j) {
        const uint4 k0 = lds16(kbuf + sub * TILE + chunk_at<RB>(token_at(g), c + 4 * j));
        const uint4 k1 = lds16(kbuf + sub * TILE + chunk_at<RB>(token_at(g) + 8, c + 4 * j));
        const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
        for (int w = 0; w < (FP8 ? 4 : 2); ++w) {
          uint32_t a0, a1, a2, a3;
          if constexpr (FP8) {
            dec4(w0[w], a0, a2);
            dec4(w1[w], a1, a3);
          } else {
            a0 = w0[2 * w], a1 = w1[2 * w], a2 = w0[2 * w + 1], a3 = w1[2 * w + 1];
          }
          const int kstep = (FP8 ? 4 : 2) * j + w;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (kstep == 0) mma<FP8, false>(x[sub][nt], a0, a1, a2, a3, qb[nt][kstep][0], qb[nt][kstep][1]);
            else mma<FP8>(x[sub][nt], a0, a1, a2, a3, qb[nt][kstep][0], qb[nt][kstep][1]);
          }
        }
      }
    }
    if constexpr (!Sh::JOINT) used();
    // tokens seen by every row, or row by row
    bool full_sub[SUB], none[SUB];
    int t0[SUB];
    bool raise = false;
#pragma unroll
    for (int sub = 0; sub < SUB; ++sub) {
      const int tile = tile_of(i, sub);
      none[sub] = sub > 0 && tile >= 1 << 30;  // past the list's end: above every position
      t0[sub] = none[sub] ? INT_MAX - kTile : tile * kTile;
      full_sub[sub] = !none[sub] && t0[sub] + kTile - 1 <= s.p0 &&
                      (a.window == 0 || t0[sub] > p_last - a.window || t0[sub] + kTile <= a.sinks);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[sub][nt][e] *= FP8 ? qs[nt][e & 1] * ks[sub] : qs[nt][e & 1];
      if (!full_sub[sub]) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = nt * 8 + 2 * c + (e & 1), t = t0[sub] + token_at(g) + (e >> 1) * 8;
            const int p = s.p0 + min(row / a.G, s.n - 1);
            if (!(t <= p && (a.window == 0 || t > p - a.window || t < a.sinks))) x[sub][nt][e] = -INFINITY;
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) raise |= fmaxf(x[sub][nt][e], x[sub][nt][e + 2]) > m[nt][e];
    }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(x[0][nt][e], x[0][nt][e + 2]);
          if (SUB > 1) mx = fmaxf(mx, fmaxf(x[SUB - 1][nt][e], x[SUB - 1][nt][e + 2]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          mx += kLazy;
          if (mx > m[nt][e]) {  // every row whose maximum has grown, once some row's has to
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
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float ref = m[nt][e & 1] == -INFINITY ? 0.0f : m[nt][e & 1];
#pragma unroll
        for (int sub = 0; sub < SUB; ++sub) {
          x[sub][nt][e] = ex2(x[sub][nt][e] - ref);
          // bf16: the lowest bit (see above), which is neither summed nor, alone, left over by rounding to bf16
          if (!FP8) x[sub][nt][e] = __uint_as_float(__float_as_uint(x[sub][nt][e]) | 1u);
          l[nt][e & 1] = FP8 ? l[nt][e & 1] + x[sub][nt][e] : add_ftz(l[nt][e & 1], x[sub][nt][e]);
        }
      }
    if constexpr (!Sh::JOINT) {
      ok = arrived();
      if (!ok) break;
    }
#pragma unroll
    for (int sub = 0; sub < SUB; ++sub) {
      if (none[sub]) continue;
      const uint32_t vbuf = smem_u32(my_ring + slot * Sh::SLOT + (Sh::JOINT ? Sh::HALF : 0)) + sub * TILE;
      // V of contraction indices 2c, 2c+1, 2c+8, 2c+9
      uint32_t vr[4][VW];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int row = token_at(2 * c + (t & 1)) + 8 * (t >> 1);
        if constexpr (VW == 2) {
          const uint2 y = lds8(vbuf + chunk_at<RB>(row, g >> 1) + (g & 1) * 8);
          vr[t][0] = y.x;
          vr[t][1] = y.y;
        } else {
#pragma unroll
          for (int j = 0; j < VW / 4; ++j) {
            const uint4 y = lds16(vbuf + chunk_at<RB>(row, g + 8 * j));
            vr[t][4 * j] = y.x;
            vr[t][4 * j + 1] = y.y;
            vr[t][4 * j + 2] = y.z;
            vr[t][4 * j + 3] = y.w;
          }
        }
      }
      bool redo = false;
      if (!full_sub[sub]) {
        // values that no row sees: zero times anything must be zero
        bool odd = false;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int tt = t0[sub] + token_at(2 * c + (t & 1)) + 8 * (t >> 1);
          const bool any = tt <= p_last && (a.window == 0 || tt > s.p0 - a.window || tt < a.sinks);
#pragma unroll
          for (int w = 0; w < VW; ++w) {
            if (!any) vr[t][w] = 0;
            if (!FP8) odd |= (vr[t][w] & 0x7F80u) == 0x7F80u || (vr[t][w] & 0x7F800000u) == 0x7F800000u;
          }
        }
        // a value that some rows see and others do not must not reach the others as 0 * inf
        if (!FP8 && s.n > 1) redo = __any_sync(0xffffffffu, odd);
      }
      if constexpr (FP8) {
        // o is in units of vref, which follows the tiles' V scales: P times their ratio is what
        // meets the codes.  vref is the largest scale so far, so the ratio is at most 1, and P times it
        // and kGain = 2^15 fits f16: all 11 bits down to 2^-29 of the row's reference.  A ratio below 1/8
        // would cost small weights more than three powers of two of that, so such a tile's product is made
        // by itself and scaled in fp32: in sum, weights keep 11 bits down to 2^-18 of the row's largest
        // (where the reference stands at most 2^8 above it), and 2^-28 of it is the last that counts.
        if (fabsf(vs[sub]) > vref) {
          const float next = fmaxf(fabsf(vs[sub]), kLeastRef), inv = 1.0f / next, corr = vref * inv;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[nt][mt][e] *= corr;
          vref = next;
          vinv = kGain * inv;
        }
        const float gained = vs[sub] * vinv, ratio = gained * (1.0f / kGain);
        const bool small = fabsf(ratio) < 0.125f;
        const float pm = small ? kGain : gained;
        uint32_t ph[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) ph[nt][e] = transpose8(pack_f16(x[sub][nt][2 * e] * pm, x[sub][nt][2 * e + 1] * pm));
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
              if (!small) {
                mma<true>(o[nt][2 * w + k], f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3], ph[nt][0], ph[nt][1]);
              } else {
                float y[4];
                mma<true, false>(y, f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3], ph[nt][0], ph[nt][1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nt][2 * w + k][e] = fmaf(y[e], ratio, o[nt][2 * w + k][e]);
              }
            }
        }
      } else if (redo) {
        // plain products, token by token, for the rows that see it
        for (int k = 0; k < kTile; ++k) {
          const int tt = token_at(k);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float pa = __shfl_sync(0xffffffffu, x[sub][nt][e], (k & 7) * 4 + c);
              const float pb = __shfl_sync(0xffffffffu, x[sub][nt][e + 2], (k & 7) * 4 + c);
              const float pt = k < 8 ? pa : pb;
              const int p = s.p0 + min((nt * 8 + 2 * c + e) / a.G, s.n - 1), t = t0[sub] + tt;
              if (t <= p && (a.window == 0 || t > p - a.window || t < a.sinks)) {
#pragma unroll
                for (int j = 0; j < VW / 4; ++j) {
                  const uint4 v = lds16(vbuf + chunk_at<RB>(tt, g + 8 * j));
                  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                  for (int mt = 0; mt < 4; ++mt) {
                    o[nt][4 * j + mt][e] += pt * bf16x2_lo(w[mt]);
                    o[nt][4 * j + mt][e + 2] += pt * bf16x2_hi(w[mt]);
                  }
                }
              }
            }
        }
      } else {
        uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float y0 = x[sub][nt][2 * e], y1 = x[sub][nt][2 * e + 1];
            ph[nt][e] = transpose8(__byte_perm(__float_as_uint(y0), __float_as_uint(y1), 0x7632));
            pl[nt][e] = transpose8(pack_bf16x2(y0 - bf16x2_hi(__float_as_uint(y0)), y1 - bf16x2_hi(__float_as_uint(y1))));
          }
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
    }
    used();
  }
  if (!ok) {
    // copies still in flight after a failed wait land (bounded) before the ring is used again
    if (slot == SLOTS) slot = 0;
    for (int n = fill; n < min(FILLS * todo, fill + SLOTS); ++n) {
      mbar_wait_bounded(&full[warp][slot], phase, kWaitNs);
      if (++slot == SLOTS) slot = 0, phase ^= 1;
    }
    if (lane == 0) atomicCAS(a.err, 0, ZP_ERR_TIMEOUT);
  }
  if (__any_sync(0xffffffffu, bad_id) && lane == 0) {
    atomicCAS(a.err, 0, ZP_ERR_BAD_TABLE);
    sm_bad = 1;
  }
  __syncthreads();  // the ring is free
  float* const sm_acc = reinterpret_cast<float*>(ring);  // [warp][row][dim]

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
      const float unit = FP8 ? vref * (1.0f / kGain) : 1.0f;
      float4* const dst = reinterpret_cast<float4*>(sm_acc) + (warp * ROWS + row) * (D / 4);
#pragma unroll
      for (int mt = 0; mt < MT; mt += 2) {
        // FP8: dims (D/8) g + 2 mt .. + 3;  bf16: dims 8 (g + 8 (mt / 4)) + 2 (mt % 4) .. + 3
        const int dim = FP8 ? (D / 8) * g + 2 * mt : 8 * (g + 8 * (mt >> 2)) + 2 * (mt & 3);
        dst[acc_at<FP8>(row, dim / 4)] = make_float4(o[nt][mt][e] * unit, o[nt][mt][e + 2] * unit, o[nt][mt + 1][e] * unit,
                                                     o[nt][mt + 1][e + 2] * unit);
      }
    }
  __syncthreads();
  // the CTA's sums (in the first warp's place), then the cluster's: CTA k of the cluster joins every
  // CLth group of 128 vectors, in the order of the CTAs
  const int rows = a.G * s.n, vecs = rows * (D / 4);
  const bool cta_bad = sm_bad != 0;
  for (int idx = tid; idx < vecs; idx += kThreads) {
    const int row = idx / (D / 4), dim = (idx % (D / 4)) * 4;
    float M = -INFINITY, Ls = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w][row]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      join(v, Ls, reinterpret_cast<const float4*>(sm_acc)[(w * ROWS + row) * (D / 4) + acc_at<FP8>(row, dim / 4)], sm_l[w][row],
           sm_m[w][row], M);
    reinterpret_cast<float4*>(sm_acc)[row * (D / 4) + acc_at<FP8>(row, dim / 4)] = make_float4(v[0], v[1], v[2], v[3]);
    if (dim == 0) {
      cta_m[row] = cta_bad ? NAN : M;  // a maximum is never NaN: marks a bad block id
      cta_l[row] = Ls;
    }
  }
  const uint32_t cl = cluster_nctarank(), rank = cluster_ctarank();
  const int parts = a.splits / static_cast<int>(cl);
  if (cl > 1) cluster_sync();
  else __syncthreads();
  const int64_t unit = static_cast<int64_t>(r) * a.Hkv + h;
  for (int idx = static_cast<int>(rank) * kThreads + tid; idx < vecs; idx += static_cast<int>(cl) * kThreads) {
    const int row = idx / (D / 4), dim = (idx % (D / 4)) * 4;
    float M = -INFINITY, Ls = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    bool skip = false;
    for (uint32_t k = 0; k < cl; ++k) {
      const float mk = ld_cluster_f1(mapa(smem_u32(&cta_m[row]), k));
      skip |= isnan(mk);
      M = fmaxf(M, mk);
    }
    for (uint32_t k = 0; k < cl; ++k)
      join(v, Ls, ld_cluster_f4(mapa(smem_u32(&sm_acc[row * D + acc_at<FP8>(row, dim / 4) * 4]), k)), ld_cluster_f1(mapa(smem_u32(&cta_l[row]), k)),
           ld_cluster_f1(mapa(smem_u32(&cta_m[row]), k)), M);
    if (parts == 1) {
      if (!skip) store_row4(a, s, h, row, dim, v, Ls);
    } else {
      float* const p = a.part + ((unit * parts + split / static_cast<int>(cl)) * ROWS + row) * (D + 4);
      *reinterpret_cast<float4*>(p + dim) = make_float4(v[0], v[1], v[2], v[3]);
      if (dim == 0) {
        p[D] = skip ? NAN : M;
        p[D + 1] = Ls;
      }
    }
  }
  if (cl > 1) cluster_sync();  // no CTA leaves while another reads its shared memory
}

// Joins the parts of a row: one warp a row, in the order of the parts.
template <int D>
__global__ void __launch_bounds__(kThreads) join_kernel(const __grid_constant__ AttnArgs a, int parts, int ROWS) {
  after_previous();  // the split kernel's writes are visible
  next_may_start();
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int row = static_cast<int>(w % ROWS), h = static_cast<int>(w / ROWS % a.Hkv);
  const int64_t r = w / ROWS / a.Hkv;
  if (r >= a.B) return;
  Span s;
  bool bad;
  if (!span_of(a, static_cast<int>(r), s, bad) || s.L == 0 || row >= a.G * s.n) return;
  const float* const p = a.part + ((r * a.Hkv + h) * parts * ROWS + row) * (D + 4);
  const int64_t step = static_cast<int64_t>(ROWS) * (D + 4);
  float M = -INFINITY;
  bool skip = false;
  for (int k = lane; k < parts; k += 32) {
    const float mk = p[k * step + D];
    skip |= isnan(mk);
    M = fmaxf(M, mk);
  }
  if (__any_sync(0xffffffffu, skip)) return;
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
  if (lane * 4 >= D) return;
  float Ls = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
  for (int k = 0; k < parts; ++k)
    join(v, Ls, *reinterpret_cast<const float4*>(p + k * step + lane * 4), p[k * step + D + 1], p[k * step + D], M);
  store_row4(a, s, h, row, lane * 4, v, Ls);
}

template <bool FP8, int D, int NT>
cudaError_t launch(const CUtensorMap& tm, const AttnArgs& a, const SplitPlan& plan, cudaStream_t st) {
  constexpr int smem = Shape<FP8, D, NT>::SMEM;
  static PerDeviceInit attrs;
  cudaError_t e = attrs.run(
      [] { return cudaFuncSetAttribute(split_kernel<FP8, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
  if (e != cudaSuccess) return e;
  e = launch_in_order(split_kernel<FP8, D, NT>, dim3(plan.splits, a.Hkv, a.B), kThreads, smem, st, plan.cluster, tm, a);
  if (e != cudaSuccess || plan.splits == plan.cluster) return e;
  const int64_t rows = static_cast<int64_t>(a.B) * a.Hkv * plan.rows;
  return launch_in_order(join_kernel<D>, dim3(static_cast<unsigned>((rows + kWarps - 1) / kWarps)), kThreads, 0, st, 1, a,
                         plan.splits / plan.cluster, plan.rows);
}

template <bool FP8>
cudaError_t dispatch(const CUtensorMap& tm, const AttnArgs& a, int d, const SplitPlan& plan, cudaStream_t st) {
  if (d == 128) return plan.rows == 8 ? launch<FP8, 128, 1>(tm, a, plan, st) : launch<FP8, 128, 2>(tm, a, plan, st);
  return plan.rows == 8 ? launch<FP8, 64, 1>(tm, a, plan, st) : launch<FP8, 64, 2>(tm, a, plan, st);
}

}  // namespace

// How many CTAs share a (request, kv head): what one wave of CTAs allows, each with two tiles per
// warp at least.  A wave counts 7/8 of the CTAs that fit the SMs, since clusters of 8 do not fill
// every GPC: a 131072-token request of 4 kv heads takes 35 us with 16 clusters a head (512 CTAs) and
// 47 us with 19 (608).  Batches that fill a wave by themselves are not split: every further CTA
// costs about 5 us of an SM's slot in latencies (224 requests of 1 to 2048 tokens, 8 kv heads: 90 us
// unsplit, 106 us with 2, 139 us with 4), while 4 requests of 100 to 500 tokens take 6.9 us with 4
// splits and 10.3 us unsplit.
//
// An unsplit batch of more than a wave takes its long requests first, so that no CTA starts on one when
// the others are done: those 224 requests in random order take 84 us so and 90 us as they come.
// Finding the order costs a CTA about 0.5 us, too much where nothing is gained: with a window, whose
// rows have nearly equal work (64 requests with a window of 1024: 44.0 us as they come, 43.4 us if
// the caller has them in order), within a wave, and past 1024 requests, where the last ones are little.
SplitPlan split_plan(const zp_params* p, int B, int max_q, int max_blocks, int window, int sinks, size_t room) {
  const int64_t sms = plan_sms();
  SplitPlan s{};
  s.rows = p->num_q_heads / p->num_kv_heads * max_q <= 8 ? 8 : 16;
  int64_t tiles = (static_cast<int64_t>(max_blocks) * p->block_size + kTile - 1) / kTile;
  if (window > 0) {
    const int64_t seen = (static_cast<int64_t>(window) + max_q - 1 + kTile - 1) / kTile + 1 +
                         (static_cast<int64_t>(sinks) + kTile - 1) / kTile;
    tiles = std::min(tiles, seen);
  }
  const int64_t units = std::max<int64_t>(1, static_cast<int64_t>(B) * p->num_kv_heads);
  const int64_t wave = sms * (s.rows == 16 ? 2 : 4) * 7 / 8;
  const int64_t n = std::min((tiles + 2 * kWarps - 1) / (2 * kWarps), wave / units);
  s.cluster = n >= 8 ? 8 : n >= 4 ? 4 : n >= 2 ? 2 : 1;
  const size_t part = static_cast<size_t>(units) * s.rows * (p->head_dim + 4) * sizeof(float);  // of one cluster a row
  const int64_t fit = room > kHeader ? static_cast<int64_t>(std::min<size_t>((room - kHeader) / part, INT_MAX)) : 0;
  s.splits = n >= 8 ? static_cast<int>(std::max<int64_t>(1, std::min(n / 8, fit))) * 8 : s.cluster;
  s.ordered = window == 0 && n < 2 && units > sms * (s.rows == 16 ? 2 : 4) && B <= kMaxOrdered;
  const int parts = s.splits / s.cluster;  // does not fall as tiles grow, so a window never needs more
  s.bytes = kHeader;
  if (parts > 1) s.bytes += (parts * part + 255) / 256 * 256;
  return s;
}

zp_status split_launch(AttnArgs a, const zp_params* p, bool fp8, const SplitPlan& plan, void* workspace, cudaStream_t st) {
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  a.splits = plan.splits;
  a.ordered = plan.ordered;
  a.err = reinterpret_cast<int32_t*>(ws);
  a.part = reinterpret_cast<float*>(ws + kHeader);
  const int d = p->head_dim;
  const uint64_t rows = static_cast<uint64_t>(2) * a.Hkv * a.b, blocks = static_cast<uint64_t>(p->num_layers) * a.num_blocks;
  CUtensorMap tm;
  // box: 16 rows of one (block, K or V, head), all of an 8-bit row or 64 columns of a bf16 one
  const bool ok = fp8 ? encode_tmap_3d_u8(&tm, a.pool, d, rows, blocks, d, rows * d, d, kTile, 1, d)
                      : encode_tmap_3d_bf16(&tm, a.pool, d, rows, blocks, static_cast<uint64_t>(d) * 2, rows * d * 2, 64, kTile, 1);
  if (!ok) return ZP_ERR_CUDA;
  const cudaError_t e = fp8 ? dispatch<true>(tm, a, d, plan, st) : dispatch<false>(tm, a, d, plan, st);
  return e == cudaSuccess ? ZP_OK : ZP_ERR_CUDA;
}

}  // namespace zp
