// zp_attn_tile.cu — attention of many query rows with a sliding window and first tokens that stay
// visible, over the paged bf16 pool, on the 5th-generation tensor cores; sm_103a.
//
// An item is 2 tiles of 128 query rows of one (request, kv head) — 128 / G queries times the G
// heads of the group, so K and V are read once for the whole group — and walks the 128-token
// tiles of the cache that any of its rows sees: first the blocks with always-visible first
// tokens, then the window's.  Blocks between the two are never loaded.  A resident CTA per SM takes
// its share of the items one after another.  Where a call has fewer items than SMs, the tiles of an item are shared by
// several CTAs, whose sums a second kernel joins.
//
// Roles: a producer warp brings K and V through the block table (one TMA box per block and
// 64-column half, 128-byte swizzle, two-stage rings); a warp brings the next item's queries as soon
// as the last product that reads them is done; an MMA warp issues S = Q K^T and O += P V with
// tcgen05; two groups of four warps (thread = row, one group per query tile) turn S into P.  S, P
// and O stay in TMEM (all 512 columns): P (bf16) overwrites S and is the A operand of the second
// product, V its B operand with the dims contiguous.  While one tile's group works on its
// softmax, the tensor core multiplies for the other tile; the next item's first products start
// while the last sums are still being written out.
//
// The running maximum is kept lazily: a row's reference is set 24 (in log2) above the largest logit so
// far, and again only when a logit passes it, so O is rescaled in TMEM rarely (with 8 in place of 24
// 2048-token chunks took 5 % longer).  P is at most 1, so sums over V overflow no earlier than the
// weighted sum itself; weights below 2^-102 of the largest are 0.  Sums and maxima are fp32; P is rounded
// to bf16 (off by at most 2^-8 of itself), as the second product's operand type asks.
//
// A tile in which some row does not see some token ("mixed": the diagonal, the window's edge, the
// first tokens, the list's end) takes the masked path.  There a warp also looks V over in shared memory:
// tokens that no row sees are zeroed, and so are values that are not finite and that only some rows see
// (0 * inf must not reach the others).  The rows that do see them get them added to their sums at the
// item's end: an infinity or NaN times a weight above 0 is itself, so no weight has to be known.  That
// takes a look at the tiles concerned alone, however long the cache is: 30 us for a tile with one such
// value, 1 ms where all of its tokens have some.
//
// Measured: 4 requests of 2048 new tokens, 32 heads on 8, d 128, a window of 2048: 191 us, 1270 TFLOP/s
// over the pairs that are seen; a prompt of 8191 tokens, 28 heads on 4, a window of 4096: 244 us, 1480
// TFLOP/s (a dozen calls after a pause; 200 and 262 us in calls that follow one another for seconds, where
// the power limit takes the clock from 2.07 to 1.97 and 1.94 GHz).  What bounds it is the chain of one query tile: softmax of 128 x 128 logits (1100 to 1250
// cycles), hand-over to the tensor core (300), its PV and its next S (1024), and back (370), since
// with d = 128 S, S, O and O fill TMEM and the next S can only take P's place.  Two tiles in turn keep
// the tensor core at 2048 of about 2900 cycles; an item's end and start cost another two tiles' time.
// Halving the loads (K and V of every second tile) gained 5 % at most: they do not bound it.
#include "zp_attn.h"

#include <algorithm>
#include <climits>
#include <type_traits>

#include "zp_launch.h"
#include "zp_ptx.cuh"

namespace zp {
namespace {

constexpr int kRows = 128;            // rows of a query tile = TMEM lanes
constexpr int kKeys = 128;            // tokens of a KV tile
constexpr int kStages = 2;
constexpr int kKWarp = 8, kMmaWarp = 9, kCleanWarp = 10, kVWarp = 11;
constexpr int kThreads = 384;         // two softmax groups, and a group of the other roles
constexpr float kLazy = 24.0f;
constexpr uint32_t kTmemCols = 512;   // S0 S1 O0 O1, 128 columns each
constexpr int kFlags = 8;             // items: K's warp is at most 6 ahead of a softmax group (the ring's 3, 2 stages, one)

// An item: which, and what it walks.
struct Item {
  int r, h, split;         // r < 0: there are no more
  int L, n, q0, p0;        // tokens, queries, first row of q, position of the request's first query
  int i0, queries;         // first query of the item, how many
  int p_first, p_last;     // positions of its first and last query
  int sink_blocks, win_block, blocks;
  int j0, j1;              // its tiles of the list
  int c0, c1, c2;          // tiles below c0 and from c1 to c2 - 1 are seen whole by every row; the others are mixed
  bool two;                // the second query tile has rows
};

// Ring of items that the MMA warp hands to the softmax groups.  A slot is taken again when both groups
// are done with its item: the second group has no part in items of one query tile, so nothing else
// would keep the others from running away from it while it writes a long item out.
constexpr int kItems = 4;

template <int D>
struct __align__(1024) TileSmem {
  uint8_t q[2][D / 64][kRows * 128];         // [tile][64-column half][row][128 B], 128-byte swizzle
  uint8_t k[kStages][D / 64][kKeys * 128];
  uint8_t v[kStages][D / 64][kKeys * 128];
  uint64_t q_full, q_empty, k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  uint64_t v_mixed[kStages], v_clean[kStages];  // in place of v_full where a tile is mixed: loaded, and looked over
  uint64_t s_full[2], p_full[2], o_full[2], o_empty[2], drain, item_full[kItems], item_empty[kItems];
  uint64_t never;                            // the test hook's, completed by nothing
  uint32_t tmem;
  int abort;
  Item items[kItems];
  int bad[kFlags], odd[kFlags];              // the last item (counted from 1) that a block id or a value marked
  int odd_lo[kFlags], odd_hi[kFlags];        // the first and last tile with such values
};


__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Waits for phase `parity` of `bar`; gives up (false) after the time limit, or when another role
// has given up.  A thread that gives up raises the flag.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns = kWaitNs) {
  const uint32_t addr = smem_u32(bar);
  if (mbar_try_wait(addr, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (mbar_try_wait(addr, parity)) return true;
    if (*abort) return false;
    if (globaltimer_ns() - t0 > limit_ns) {
      *abort = 1;
      return false;
    }
  }
}

__device__ __forceinline__ void sts16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// 32 bytes to a 32-byte boundary.
__device__ __forceinline__ void st_global_32(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]),
               "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// True in one lane of the (whole) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
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

// Two fp32 values in a register pair, and what Blackwell does with both at once.
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ uint64_t pair2(float x) { return pair(__float_as_uint(x), __float_as_uint(x)); }

// The lowest n bits, n clamped to 0 .. 32.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; }

// What an item needs from memory, loaded one item ahead.
struct Raw {
  int L, q0, q1;
};
__device__ __forceinline__ Raw load_raw(const AttnArgs& a, int item, int items) {
  Raw raw{0, 0, 0};
  if (item < items) {
    const int r = static_cast<int>(static_cast<uint32_t>(item) / static_cast<uint32_t>(a.splits * a.Hkv) % static_cast<uint32_t>(a.B));
    raw.L = a.seq_lens[r];
    raw.q0 = a.q_start[r];
    raw.q1 = a.q_start[r + 1];
  }
  return raw;
}

// Items in order of queries from the last (which see the most) to the first, request, kv head,
// and part of the tiles.  False: nothing to do (`bad`: the request is reported).
__device__ __forceinline__ bool take_item(const AttnArgs& a, int item, int nx, const Raw& raw, Item& w, bool& bad) {
  const int qpt = kRows / a.G;  // queries per tile
  uint32_t u = static_cast<uint32_t>(item);
  w.split = 0;
  if (a.splits > 1) {
    w.split = static_cast<int>(u % static_cast<uint32_t>(a.splits));
    u /= static_cast<uint32_t>(a.splits);
  }
  w.h = static_cast<int>(u % static_cast<uint32_t>(a.Hkv));
  u /= static_cast<uint32_t>(a.Hkv);
  w.r = static_cast<int>(u % static_cast<uint32_t>(a.B));
  const int x = static_cast<int>(u / static_cast<uint32_t>(a.B));
  w.L = raw.L;
  w.q0 = raw.q0;
  const int64_t n = static_cast<int64_t>(raw.q1) - raw.q0;
  bad = w.q0 < 0 || n < 0 || n > a.max_q || w.q0 + n > a.T;
  bad = bad || (n > 0 && (w.L < n || w.L > static_cast<int64_t>(a.max_blocks) * a.b));
  if (bad) return false;
  w.n = static_cast<int>(n);
  w.i0 = (nx - 1 - x) * 2 * qpt;
  if (w.i0 >= w.n) return false;
  w.queries = min(2 * qpt, w.n - w.i0);
  w.p0 = w.L - w.n;
  w.p_first = w.p0 + w.i0;
  w.p_last = w.p_first + w.queries - 1;
  const int bs = a.b == 16 ? 4 : 5;
  const int first = a.window == 0 ? 0 : max(0, w.p_first - a.window + 1);
  w.win_block = first >> bs;
  w.sink_blocks = min((min(a.sinks, w.L) + a.b - 1) >> bs, w.win_block);
  w.blocks = w.sink_blocks + (w.p_last >> bs) + 1 - w.win_block;
  const int tiles = ((w.blocks << bs) + kKeys - 1) / kKeys;  // at most 2^23, and as many splits as SMs
  w.j0 = 0;
  w.j1 = tiles;
  if (a.splits > 1) {
    w.j0 = static_cast<int>(static_cast<uint32_t>(tiles) * w.split / static_cast<uint32_t>(a.splits));
    w.j1 = static_cast<int>(static_cast<uint32_t>(tiles) * (w.split + 1) / static_cast<uint32_t>(a.splits));
  }
  w.two = w.queries > qpt;
  // runs of the list: first tokens' blocks, where column e is token e, and the window's, where it is
  // token e + shift (the window's alone where there are no first tokens); one run where the two meet
  const int shift = (w.win_block - w.sink_blocks) << bs, sink = shift ? w.sink_blocks << bs : 0;
  w.c0 = min(min(sink, a.sinks), w.p_first + 1) / kKeys;
  w.c1 = (max(sink, a.window == 0 ? 0 : w.p_last - a.window + 1 - shift) + kKeys - 1) / kKeys;
  w.c2 = min(w.p_first + 1 - shift, w.blocks << bs) / kKeys;
  return true;
}

// Token of column `col` of list tile j.
__device__ __forceinline__ int token_of(const AttnArgs& a, const Item& w, int j, int col) {
  const int e = j * kKeys + col, sink = w.sink_blocks * a.b;
  return e < sink ? e : w.win_block * a.b + e - sink;
}

__device__ __forceinline__ bool sees(const AttnArgs& a, int p, int t) {
  return t <= p && (a.window == 0 || t > p - a.window || t < a.sinks);
}

// Some row of the item does not see some token of list tile j.
__device__ __forceinline__ bool mixed_tile(const Item& w, int j) { return j >= w.c0 && (j < w.c1 || j >= w.c2); }

// The columns c0 .. c0 + 31 of a run of tokens base + col that position p sees, as bits.
__device__ __forceinline__ uint32_t run_bits(const AttnArgs& a, int p, int base, int c0) {
  const uint32_t upto = low_bits(p - base - c0 + 1);
  if (a.window == 0) return upto;
  // t > p - window, or t < sinks
  const uint32_t gone = low_bits(p - a.window - base - c0 + 1), kept = low_bits(a.sinks - base - c0);
  return upto & (~gone | kept);
}
// The same of list tile j, which may join the first tokens' run and the window's.
__device__ __forceinline__ uint32_t tile_bits(const AttnArgs& a, const Item& w, int j, int p, int c0) {
  const int cut = w.sink_blocks * a.b - j * kKeys, left = w.blocks * a.b - j * kKeys;  // columns of the first run, of the list
  const uint32_t in_sink = low_bits(cut - c0);
  return low_bits(left - c0) & ((run_bits(a, p, j * kKeys, c0) & in_sink) |
                                (run_bits(a, p, w.win_block * a.b - cut, c0) & ~in_sink));
}

// Where a row's results go: the output, or its part of a split item.
struct Sink {
  uint16_t* out;   // NULL: no such row
  float* part;     // D sums, maximum, sum of weights
};
template <int D>
__device__ __forceinline__ Sink sink_of(const AttnArgs& a, const Item& w, int i, int g, bool have) {
  Sink s{nullptr, nullptr};
  if (!have) return s;
  const int64_t t = w.q0 + w.i0 + i, head = w.h * a.G + g;
  s.out = a.out + t * a.o_ts + head * a.o_hs;
  if (a.splits > 1) s.part = a.part + ((static_cast<int64_t>(w.split) * a.T + t) * (a.Hkv * a.G) + head) * (D + 4);
  return s;
}

// Whether the 8 tokens from t0 on, which stand in one block, are seen by every row of the item.
__device__ __forceinline__ bool whole8(const AttnArgs& a, const Item& w, int t0) {
  return t0 + 7 <= w.p_first && (a.window == 0 || t0 > w.p_last - a.window || t0 + 7 < a.sinks);
}
// Whether some row of the item sees token t.
__device__ __forceinline__ bool seen_by_some(const AttnArgs& a, const Item& w, int t) {
  return t <= w.p_last && (a.window == 0 || t > w.p_first - a.window || t < a.sinks);
}
// Whether the low or the high bf16 of a word is not finite.
__device__ __forceinline__ bool odd_lo(uint32_t x) { return (x & 0x7F80u) == 0x7F80u; }
__device__ __forceinline__ bool odd_hi(uint32_t x) { return (x & 0x7F800000u) == 0x7F800000u; }

// Adds what look_over took out of V in tiles lo to hi to the rows of one query tile that see it, whose
// results stand in memory: 32 rows a warp, D / 32 dims a lane.  Rolled and a call of its own: with its loop over
// tokens unrolled, calls that never come here took 1 % longer.
template <int D>
__device__ __noinline__ void add_odd_values(const AttnArgs& a, const Item& w, int lo, int hi, int t, int warp, int lane) {
  constexpr int DW = D / 64;  // words of a lane
  const int qpt = kRows / a.G;
  const int64_t tile_values = static_cast<int64_t>(a.b) * D;  // of a (block, K|V, head)
  const uint16_t* const pool = reinterpret_cast<const uint16_t*>(a.pool) + lane * (2 * DW);
  for (int e = lo * (kKeys / 8); e < (hi + 1) * (kKeys / 8); ++e) {
    const int j = e / (kKeys / 8), t0 = token_of(a, w, j, e % (kKeys / 8) * 8);
    if (!mixed_tile(w, j) || e * 8 >= w.blocks * a.b || whole8(a, w, t0)) continue;
    const int64_t phys = a.tables[static_cast<int64_t>(w.r) * a.max_blocks + t0 / a.b];
    const uint16_t* const k = pool + ((static_cast<int64_t>(a.layer) * a.num_blocks + phys) * 2 * a.Hkv + w.h) * tile_values + t0 % a.b * D;
    const uint16_t* const v = k + a.Hkv * tile_values;
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
      for (int i = 0; i < DW; ++i) top = max_u16x2(top, reinterpret_cast<const uint32_t*>(v + c * D)[i] & 0x7FFF7FFFu);
    if (!__any_sync(0xffffffffu, odd_lo(top) || odd_hi(top))) continue;
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
      uint32_t x[DW];
      bool odd = false;
#pragma unroll
      for (int i = 0; i < DW; ++i) {
        x[i] = reinterpret_cast<const uint32_t*>(v + c * D)[i];
        odd |= odd_lo(x[i]) || odd_hi(x[i]);
      }
      if (!seen_by_some(a, w, t0 + c) || !__any_sync(0xffffffffu, odd)) continue;
      // A weight of 0 (a logit of -inf) makes NaN of it, and only an infinite key can give one; a key of
      // NaN has made the whole row NaN.
      uint32_t kw[DW];
      bool inf = false, nan = false;
#pragma unroll
      for (int i = 0; i < DW; ++i) {
        kw[i] = reinterpret_cast<const uint32_t*>(k + c * D)[i];
        inf |= odd_lo(kw[i]) || odd_hi(kw[i]);
        nan |= (kw[i] & 0x7FFFu) > 0x7F80u || (kw[i] & 0x7FFF0000u) > 0x7F800000u;
      }
      if (__any_sync(0xffffffffu, nan)) continue;
      inf = __any_sync(0xffffffffu, inf);
      for (int rr = warp * 32; rr < warp * 32 + 32; ++rr) {
        const int qi = rr / a.G, i = t * qpt + qi;
        if (qi >= qpt || i >= w.queries) break;
        if (!sees(a, w.p_first + i, t0 + c)) continue;
        bool nothing = false;
        if (inf) {
          const uint16_t* const q = a.q + (w.q0 + w.i0 + i) * a.q_ts + (w.h * a.G + rr - qi * a.G) * a.q_hs + lane * (2 * DW);
          float dot = 0.0f;
#pragma unroll
          for (int d = 0; d < DW; ++d) {
            dot = fmaf(bf16x2_lo(q[2 * d]), bf16x2_lo(kw[d]), dot);
            dot = fmaf(bf16x2_lo(q[2 * d + 1]), __uint_as_float(kw[d] & 0xFFFF0000u), dot);
          }
#pragma unroll
          for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, s);
          nothing = dot == -INFINITY;
        }
        const Sink to = sink_of<D>(a, w, i, rr - qi * a.G, true);
#pragma unroll
        for (int d = 0; d < 2 * DW; ++d) {
          const uint32_t word = x[d >> 1];
          if (!(d & 1 ? odd_hi(word) : odd_lo(word))) continue;
          const float value = nothing ? NAN : d & 1 ? __uint_as_float(word & 0xFFFF0000u) : bf16x2_lo(word);
          const int dim = lane * (2 * DW) + d;
          if (to.part) to.part[dim] += value;
          else to.out[dim] = static_cast<uint16_t>(pack_bf16x2(bf16x2_lo(to.out[dim]) + value, 0.0f));
        }
      }
    }
  }
}

// Looks V of mixed tile j over in shared memory (one warp): tokens that no row sees are zeroed, and values
// that are not finite where only some rows see them; true if there were any of those.  8 tokens at a
// time, which are tokens of one block; a lane holds 16-byte chunk lane % (D / 8) of every (256 / D)th of them.
template <int D>
__device__ __forceinline__ bool look_over(const AttnArgs& a, const Item& w, int j, uint8_t* v, int lane) {
  constexpr int kPer = 256 / D, kLoads = 8 / kPer;
  const int ch = lane % (D / 8), sub = lane / (D / 8);
  uint8_t* at[kLoads];
#pragma unroll
  for (int y = 0; y < kLoads; ++y) {
    const int col = y * kPer + sub;
    at[y] = v + (ch >> 3) * (kKeys * 128) + col * 128 + (((ch & 7) ^ col) << 4);
  }
  // lane g < 16: whether the g-th 8 tokens need a look (blocks past the list's end are zeros)
  const int t0 = token_of(a, w, j, (lane & 15) * 8);
  const bool listed = j * kKeys + (lane & 15) * 8 < w.blocks * a.b;
  const uint32_t look = __ballot_sync(0xffffffffu, listed && !whole8(a, w, t0)) & 0xFFFFu;
  uint32_t todo = look;
  uint32_t top = 0;
  while (todo) {
    const int g = __ffs(todo) - 1;
    todo &= todo - 1;
    const int tk = __shfl_sync(0xffffffffu, t0, g) + sub;
    uint4 x[kLoads];
#pragma unroll
    for (int y = 0; y < kLoads; ++y) x[y] = *reinterpret_cast<const uint4*>(at[y] + g * 1024);
#pragma unroll
    for (int y = 0; y < kLoads; ++y) {
      if (seen_by_some(a, w, tk + y * kPer)) {
        top = max_u16x2(max_u16x2(top, x[y].x & 0x7FFF7FFFu), x[y].y & 0x7FFF7FFFu);
        top = max_u16x2(max_u16x2(top, x[y].z & 0x7FFF7FFFu), x[y].w & 0x7FFF7FFFu);
      } else {
        *reinterpret_cast<uint4*>(at[y] + g * 1024) = make_uint4(0, 0, 0, 0);
      }
    }
  }
  if (!__any_sync(0xffffffffu, (top & 0xFFFFu) >= 0x7F80u || top >= 0x7F800000u)) return false;
  for (todo = look; todo; todo &= todo - 1) {
    const int g = __ffs(todo) - 1;
#pragma unroll 1
    for (int y = 0; y < kLoads; ++y) {
      uint32_t* const x = reinterpret_cast<uint32_t*>(v + (ch >> 3) * (kKeys * 128) + (y * kPer + sub) * 128 + (((ch & 7) ^ (y * kPer + sub)) << 4) + g * 1024);
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        uint32_t z = x[i];
        if (odd_lo(z)) z &= 0xFFFF0000u;
        if (odd_hi(z)) z &= 0x0000FFFFu;
        x[i] = z;
      }
    }
  }
  return true;
}

// Q_TMA: the queries' rows are aligned and come by TMA (one box per tile and 64-column half: the
// group's heads of 128 / G tokens, which is the order of the tile's rows); else by plain loads.
// PARTS: items are split, and leave sums for the joining kernel.
template <int D, bool Q_TMA, bool PARTS>
__global__ void __launch_bounds__(kThreads, 1) tile_kernel(const __grid_constant__ CUtensorMap tm, const __grid_constant__ CUtensorMap tq,
                                                           const __grid_constant__ AttnArgs a, int nx, int items) {
  constexpr int NH = D / 64;
  extern __shared__ uint8_t dyn[];
  TileSmem<D>& s = *reinterpret_cast<TileSmem<D>*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int qpt = kRows / a.G;
  // The CTA's items: the grid takes a run of gridDim.x items in one direction, the next in the other,
  // so that the sums of what its CTAs get come near one another (items get lighter along the list).
  const int step = static_cast<int>(gridDim.x);
  const auto next_item = [&](int item) {
    const int in = item % step;
    return item - in + step + (step - 1 - in);
  };

  if (tid == 0) {
    mbar_init(&s.q_full, Q_TMA ? 1 : 32);
    mbar_init(&s.q_empty, 1);
    mbar_init(&s.drain, 1);
    mbar_init(&s.never, 1);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.k_full[i], 1);
      mbar_init(&s.k_empty[i], 1);
      mbar_init(&s.v_full[i], 1);
      mbar_init(&s.v_empty[i], 1);
      mbar_init(&s.v_mixed[i], 1);
      mbar_init(&s.v_clean[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.p_full[i], 4);
      mbar_init(&s.o_full[i], 1);
      mbar_init(&s.o_empty[i], 4);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&s.item_full[i], 1);
      mbar_init(&s.item_empty[i], 8);
    }
    s.abort = 0;
    for (int i = 0; i < kFlags; ++i) s.bad[i] = s.odd[i] = 0;
    fence_mbar_init();
    prefetch_tensormap(&tm);
    if (Q_TMA) prefetch_tensormap(&tq);
  }
  // rows of the query tiles that no query fills stay zero
  for (int i = tid; i < static_cast<int>(sizeof(s.q) / 16); i += kThreads)
    reinterpret_cast<uint4*>(&s.q[0][0][0])[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (warp == kMmaWarp) tmem_alloc(&s.tmem, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  after_previous();
  next_may_start();
  const uint32_t tbase = s.tmem;
  volatile int* const abort = &s.abort;

  // Registers follow the roles: 2 x 128 x 208 + 128 x 88 of the 384 x 168 that the launch gave.  With 200 the
  // softmax groups spill inside their loop (2048-token chunks 210 us, 200 us with 208).
  if (warp >= 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  Item w;
  bool bad;
  Raw raw = load_raw(a, blockIdx.x, items);
  int count = 0;       // items with work so far
  uint32_t tiles = 0;  // KV tiles of the items before

  if (warp == kKWarp || warp == kVWarp) {
    // One warp each: K of the next tile is wanted a product earlier than its V, and in one warp it
    // waited behind the V before it.
    const int kv = warp == kVWarp;
    uint64_t* const empties = kv ? s.v_empty : s.k_empty;
    const int bpt = kKeys / a.b;  // blocks per tile
    bool go = true;
    uint32_t done = 0;            // tiles issued
    int q_loads = 0;              // items whose queries were
    uint64_t* last[kStages] = {};  // barrier of each stage's last tile, and how often each was used
    uint32_t used_full = 0, used_mixed = 0, last_parity = 0;  // bits by stage
    for (int item = blockIdx.x; go && item < items; item = next_item(item)) {
      const Raw now = raw;
      raw = load_raw(a, next_item(item), items);
      if (!take_item(a, item, nx, now, w, bad)) {
        if (bad && lane == 0) atomicCAS(a.err, 0, ZP_ERR_BAD_TABLE);
        continue;
      }
      ++count;
      const int32_t* const table = a.tables + static_cast<int64_t>(w.r) * a.max_blocks;
      const auto id_of = [&](int j) {  // block id that the lane loads for tile j
        const int e = j * bpt + lane;
        if (lane >= bpt || e >= w.blocks || j >= w.j1) return 0;
        return table[e < w.sink_blocks ? e : w.win_block + e - w.sink_blocks];
      };
      // K's warp brings the item's queries too, once the last product that reads the ones before is
      // done; behind the first K, whose stage is free earlier.  (In the warp that looks V over they came
      // up to 3 us late.)
      const auto load_q = [&] {
        if (lane == 0 && count > 1) go = wait(&s.q_empty, count & 1, abort);  // completion count - 1
        go = __shfl_sync(0xffffffffu, go, 0);
        if (!go) return;
        q_loads = count;
        if constexpr (Q_TMA) {
          if (lane == 0) {
            mbar_arrive_expect_tx(&s.q_full, static_cast<uint32_t>((w.two ? 2 : 1) * qpt * a.G * D * 2));
            for (int t = 0; t < (w.two ? 2 : 1); ++t)
              for (int hd = 0; hd < NH; ++hd) tma_load_3d(s.q[t][hd], &tq, &s.q_full, hd * 64, w.h * a.G, w.q0 + w.i0 + t * qpt);
          }
        } else {
          for (int rr = lane; rr < w.queries * a.G; rr += 32) {
            const int i = rr / a.G, g = rr - i * a.G, t = i >= qpt, row = (i - t * qpt) * a.G + g;
            const uint16_t* const q = a.q + (w.q0 + w.i0 + i) * a.q_ts + (w.h * a.G + g) * a.q_hs;
            for (int c = 0; c < D / 8; ++c) {
              uint32_t y[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                y[e] = static_cast<uint32_t>(q[c * 8 + 2 * e]) | static_cast<uint32_t>(q[c * 8 + 2 * e + 1]) << 16;
              *reinterpret_cast<uint4*>(&s.q[t][c >> 3][row * 128 + (((c & 7) ^ (row & 7)) << 4)]) = make_uint4(y[0], y[1], y[2], y[3]);
            }
          }
          fence_proxy_async_smem();
          mbar_arrive(&s.q_full);
        }
        __syncwarp();
      };
      if (!kv && w.j0 == w.j1) load_q();  // a part without tiles
      int id = id_of(w.j0);
      for (int j = w.j0; go && j < w.j1; ++j, ++done) {
        const uint32_t st = done % kStages, ph = (done / kStages) & 1;
        const int nb = min(bpt, w.blocks - j * bpt);
        // an id outside the pool: the item's rows are not written, and block 0 is read in its place
        const bool out = id < 0 || id >= a.num_blocks;
        if (__any_sync(0xffffffffu, out) && lane == 0) {
          *reinterpret_cast<volatile int*>(&s.bad[count % kFlags]) = count;
          atomicCAS(a.err, 0, ZP_ERR_BAD_TABLE);
        }
        // blocks past the list's end have a coordinate past the tensor's: they come as zeros
        const int z = lane < nb ? a.layer * static_cast<int>(a.num_blocks) + (out ? 0 : id) : a.layers * static_cast<int>(a.num_blocks);
        id = id_of(j + 1);
        uint64_t* full = kv ? &s.v_full[st] : &s.k_full[st];
        uint32_t* used = &used_full;
        if (kv && mixed_tile(w, j)) {
          full = &s.v_mixed[st];
          used = &used_mixed;
        }
        if (lane == 0) {
          if (done >= kStages) go = wait(&empties[st], ph ^ 1, abort);
          if (go) mbar_arrive_expect_tx(full, kKeys * D * 2);
        }
        go = __shfl_sync(0xffffffffu, go, 0);
        if (!go) break;
        if (lane < bpt)
#pragma unroll
          for (int hd = 0; hd < NH; ++hd)
            tma_load_3d((kv ? s.v[st][hd] : s.k[st][hd]) + lane * a.b * 128, &tm, full, hd * 64, (kv * a.Hkv + w.h) * a.b, z);
        if (!kv && j == w.j0) load_q();
        last[st] = full;
        last_parity = (last_parity & ~(1u << st)) | (*used & (1u << st));
        *used ^= 1u << st;
        __syncwarp();
      }
    }
    // Copies still in flight land before the shared memory is released.  A role may give up after this
    // warp is through, so it waits for its last ones in any case (they have landed, but for that).
    if (lane == 0)
      for (int st = 0; st < kStages; ++st)
        if (last[st]) mbar_wait_bounded(last[st], (last_parity >> st) & 1, kWaitNs);
    if (Q_TMA && lane == 0 && q_loads > 0) mbar_wait_bounded(&s.q_full, (q_loads - 1) & 1, kWaitNs);
    __syncwarp();
  } else if (warp == kCleanWarp) {
    // V of the mixed tiles: see the head of this file
    bool go = true;
    uint32_t seen_mixed = 0;  // phases by stage
    for (int item = blockIdx.x; go && item < items; item = next_item(item)) {
      const Raw now = raw;
      raw = load_raw(a, next_item(item), items);
      if (!take_item(a, item, nx, now, w, bad)) continue;
      ++count;
      for (int j = w.j0; j < w.j1; ++j) {
        if (!mixed_tile(w, j)) continue;
        const uint32_t st = (tiles + static_cast<uint32_t>(j - w.j0)) % kStages;
        go = __all_sync(0xffffffffu, wait(&s.v_mixed[st], (seen_mixed >> st) & 1, abort));
        if (!go) break;
        seen_mixed ^= 1u << st;
        if (look_over<D>(a, w, j, s.v[st][0], lane) && lane == 0) {
          const int f = count % kFlags;
          if (s.odd[f] != count) s.odd[f] = count, s.odd_lo[f] = j;
          s.odd_hi[f] = j;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.v_clean[st]);
      }
      tiles += static_cast<uint32_t>(w.j1 - w.j0);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // The whole warp walks, and one thread of it issues: addresses and descriptors that the compiler
    // knows to be the warp's own stay in uniform registers, where the products take them from.
    // (Issued by a thread of a divergent warp, each product cost 95 cycles in place of its 64.)
    // Descriptors are made once; a step along the contraction adds to their start address (in
    // units of 16 bytes).
    static_assert(kStages == 2, "descriptors below");
    const uint32_t idesc_s = idesc_bf16_f32(kRows, kKeys);
    const uint32_t idesc_o = idesc_bf16_f32(kRows, D) | kTransposeB;
    const uint32_t tb = __shfl_sync(0xffffffffu, tbase, 0);
    const uint64_t qd0 = smem_desc_sw128(smem_u32(s.q[0])), qd1 = smem_desc_sw128(smem_u32(s.q[1]));
    const uint64_t kd0 = smem_desc_sw128(smem_u32(s.k[0])), kd1 = smem_desc_sw128(smem_u32(s.k[1]));
    const uint64_t vd0 = smem_desc_mn_sw128(smem_u32(s.v[0]), kKeys * 128), vd1 = smem_desc_mn_sw128(smem_u32(s.v[1]), kKeys * 128);
    const bool one = elect_one();
    const auto issue_s = [&](int t, uint32_t st) {
      const uint64_t qd = t ? qd1 : qd0, kd = st ? kd1 : kd0;
      const uint32_t d = tb + t * kKeys;
      if (one) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          constexpr int kHalf = kRows * 128 / 16;  // from one 64-column half to the next
          const int at = (kk >> 2) * kHalf + (kk & 3) * 2;
          mma_bf16(d, qd + at, kd + at, idesc_s, kk > 0);
        }
        mma_commit(&s.s_full[t]);
      }
      __syncwarp();
    };
    const auto issue_o = [&](int t, uint32_t st, bool add) {
      const uint64_t vd = st ? vd1 : vd0;
      const uint32_t d = tb + 256 + t * 128, p = tb + t * kKeys;
      if (one) {
        mma_bf16_ts(d, p, vd, idesc_o, add);
#pragma unroll
        for (int kk = 1; kk < kKeys / 16; ++kk) mma_bf16_ts(d, p + kk * 8, vd + kk * 128, idesc_o, 1);
      }
      __syncwarp();
    };
    const auto commit = [&](uint64_t* bar) {
      if (one) mma_commit(bar);
      __syncwarp();
    };
    // the warp's answer: every lane waits
    const auto wait_all = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity, abort)) != 0; };
    bool ok = true;
    uint32_t seen_clean = 0, seen_full = 0;  // phases by stage
    uint32_t p_seen[2] = {0, 0}, o_used[2] = {0, 0};
    // the next item with work, one item ahead of its products; the softmax groups take it from here
    int item = blockIdx.x;
    int n_next = 0, c0_next = 0, c1_next = 0, c2_next = 0;
    bool two_next = false;
    const auto publish = [&](int k) {  // the k-th (from 0)
      Item next;
      next.two = false;
      next.j0 = next.c0 = next.c1 = next.c2 = 0;
      bool have = false;
      while (!have && item < items) {
        const Raw now = raw;
        const int cur = item;
        item = next_item(item);
        raw = load_raw(a, item, items);
        have = take_item(a, cur, nx, now, next, bad);
      }
      if (!have) next.r = -1;
      if (k >= kItems) ok = wait_all(&s.item_empty[k % kItems], (k / kItems - 1) & 1);
      if (!ok) return;
      if (one) {
        s.items[k % kItems] = next;
        mbar_arrive(&s.item_full[k % kItems]);
      }
      __syncwarp();
      // what the products need of it: tiles (-1: no more items), and which of them are mixed
      n_next = __shfl_sync(0xffffffffu, have ? next.j1 - next.j0 : -1, 0);
      two_next = __shfl_sync(0xffffffffu, static_cast<int>(next.two), 0) != 0;
      c0_next = next.c0 - next.j0, c1_next = next.c1 - next.j0, c2_next = next.c2 - next.j0;
    };
    publish(0);
    while (ok && n_next >= 0) {
      const int n = n_next, c0 = c0_next, c1 = c1_next, c2 = c2_next;
      const bool two = two_next;
      ok = wait_all(&s.q_full, count & 1);
      ++count;
      uint32_t st = __shfl_sync(0xffffffffu, tiles & 1, 0);
      if (ok && n > 0) ok = wait_all(&s.k_full[st], (tiles >> 1) & 1);
      if (!ok) break;
      tc_fence_after();
      if (n > 0) {
        issue_s(0, st);
        if (two) issue_s(1, st);
        commit(&s.k_empty[st]);
      }
      if (n <= 1) commit(&s.q_empty);
      publish(count);  // while the softmax groups have their first tile
      // the test hook gives up here, with copies and products in flight
      if (a.stall) ok = __all_sync(0xffffffffu, wait(&s.never, 0, abort, a.limit_ns));
      for (int j = 0; ok && j < n; ++j, ++tiles, st ^= 1) {
        const bool more = j + 1 < n;
        if (j >= c0 && (j < c1 || j >= c2)) {
          ok = wait_all(&s.v_clean[st], (seen_clean >> st) & 1);
          seen_clean ^= 1u << st;
        } else {
          ok = wait_all(&s.v_full[st], (seen_full >> st) & 1);
          seen_full ^= 1u << st;
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok || (t == 1 && !two)) break;
          const bool last = t == 1 || !two;
          ok = wait_all(&s.p_full[t], p_seen[t]++ & 1);
          if (ok && j == 0 && o_used[t]++ > 0) ok = wait_all(&s.o_empty[t], o_used[t] & 1);
          if (!ok) break;
          tc_fence_after();
          issue_o(t, st, j > 0);
          if (last) commit(&s.v_empty[st]);
          if (more) {
            if (t == 0) ok = wait_all(&s.k_full[st ^ 1], ((tiles + 1) >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            issue_s(t, st ^ 1);
            if (last) {
              commit(&s.k_empty[st ^ 1]);
              if (j + 2 == n) commit(&s.q_empty);  // no further product reads the queries
            }
          } else {
            commit(&s.o_full[t]);
          }
        }
      }
    }
    // products still in flight after a give-up, of whichever role, complete before TMEM is released
    commit(&s.drain);
    mbar_wait_bounded(&s.drain, 0, kWaitNs);
    __syncwarp();
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    int count = 0;  // items so far
    const int t = warp >> 2, row = tid & 127;
    const int qi = row / a.G, gi = row - qi * a.G;
    const int i = t * qpt + qi;  // query of the item
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tbase + lanes + t * kKeys, to = tbase + lanes + 256 + t * 128;
    const uint64_t sl2x2 = pair2(a.sl2);
    uint32_t s_seen = 0, o_seen = 0;
    bool ok = true;
    while (true) {
      ok = __all_sync(0xffffffffu, wait(&s.item_full[count % kItems], (count / kItems) & 1, abort));
      if (!ok) break;
      const Item& w = s.items[count % kItems];  // stays until every warp has let go of it
      uint64_t* const let_go = &s.item_empty[count % kItems];
      if (w.r < 0) break;
      ++count;
      if (t == 1 && !w.two) {
        __syncwarp();
        if (lane == 0) mbar_arrive(let_go);
        continue;
      }
      float m = -INFINITY, l = 0.0f;
      for (int j = w.j0; j < w.j1; ++j) {
        const bool mixed = mixed_tile(w, j);  // before the wait: shared memory's latency is out of the way
        ok = __all_sync(0xffffffffu, wait(&s.s_full[t], s_seen++ & 1, abort));
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
          const int p = w.p_first + min(i, w.queries - 1);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t bits = tile_bits(a, w, j, p, c * 32);
            // a warp's rows are a few queries, so most of its 32-column pieces are whole
            if (__all_sync(0xffffffffu, bits == 0xFFFFFFFFu)) continue;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(bits >> e & 1)) x[c][e] = __float_as_uint(-INFINITY);
          }
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 32; ++e)
#pragma unroll
          for (int c = 0; c < 4; ++c) mx[c] = fmaxf(mx[c], __uint_as_float(x[c][e]));
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.sl2;
        if (__any_sync(0xffffffffu, top > m)) {
          const float mn = fmaxf(m, top + kLazy), corr = m == -INFINITY ? 0.0f : ex2(m - mn);
          if (j > w.j0) {  // O of the tiles so far, complete since s_full follows their products
#pragma unroll 1
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
        const uint64_t ref = pair2(m == -INFINITY ? 0.0f : -m);
        uint64_t sum = 0;  // a pair of +0
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const uint32_t (&src)[32] = x[2 * c + (e >> 4)];
            float y0, y1;
            unpair(fma2(pair(src[(2 * e) & 31], src[(2 * e + 1) & 31]), sl2x2, ref), y0, y1);
            y0 = ex2(y0);
            y1 = ex2(y1);
            sum = add2(sum, pair(__float_as_uint(y0), __float_as_uint(y1)));
            pk[e] = pack_bf16x2(y0, y1);
          }
          tmem_st32(ts + c * 32, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.p_full[t]);
        float a0, a1;
        unpair(sum, a0, a1);
        l += a0 + a1;
      }
      if (!ok) break;
      const bool empty = w.j0 == w.j1;  // a part without tiles
      if (!empty) {
        ok = __all_sync(0xffffffffu, wait(&s.o_full[t], o_seen++ & 1, abort));
        if (!ok) break;
        tc_fence_after();
      }
      const bool have = qi < qpt && i < w.queries;
      const Sink to_row = sink_of<D>(a, w, i, gi, have);
      const bool marked = *reinterpret_cast<volatile int*>(&s.bad[count % kFlags]) == count;
      const bool odd = *reinterpret_cast<volatile int*>(&s.odd[count % kFlags]) == count;
      const bool write = have && !marked;
      if (to_row.part && (write || marked || empty)) {
        to_row.part[D] = marked ? NAN : m;  // a maximum is never NaN: marks a part with a bad block id
        to_row.part[D + 1] = l;
      }
      if (!empty) {
        const float inv = 1.0f / l;  // a row sees itself; logits of -inf alone give 0 / 0, as their softmax
        // Rolled: code that runs once an item comes from far away, and its size is time.
        if constexpr (PARTS) {
          // Through shared memory, 128 bytes of each row at a time, so that 8 lanes write one row's.  The CTA's only
          // item is done with its queries.
          static_assert(sizeof(s.q) >= 8 * 32 * 128, "a warp's rows");
          const uint32_t stage = smem_u32(s.q) + warp * (32 * 128), put = stage + lane * 128, get = stage + (lane >> 3) * 128;
          float* const mine = write ? to_row.part : nullptr;
          unsigned long long rows[8];  // where the lane's 16 bytes of rows 4 q + lane / 8 go
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            rows[q] = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), q * 4 + (lane >> 3));
            if (rows[q]) rows[q] += (lane & 7) * 16;
          }
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32_issue(to + c * 32, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              sts16(put + ((e ^ (lane & 7)) << 4), make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]));
            __syncwarp();
            uint4 v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = lds16(get + q * 512 + (((lane & 7) ^ ((q * 4 + (lane >> 3)) & 7)) << 4));
#pragma unroll
            for (int q = 0; q < 8; ++q)
              if (rows[q]) *reinterpret_cast<uint4*>(rows[q] + c * 128) = v[q];
            __syncwarp();
          }
        } else {
          const uint32_t align = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(to_row.out));
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32], y[16];
            tmem_ld32_issue(to + c * 32, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = pack_bf16x2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
            uint16_t* const dst = to_row.out + c * 32;
            if (!write) continue;
            if ((align & 31) == 0) {
              st_global_32(dst, y);
              st_global_32(dst + 16, y + 8);
            } else if ((align & 15) == 0) {
#pragma unroll
              for (int e = 0; e < 4; ++e) reinterpret_cast<uint4*>(dst)[e] = make_uint4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                dst[2 * e] = static_cast<uint16_t>(y[e]);
                dst[2 * e + 1] = static_cast<uint16_t>(y[e] >> 16);
              }
            }
          }
        }
        tc_fence_before();  // the next item may use O
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.o_empty[t]);
        if (odd && !marked) {
          __syncwarp();  // the rows as written
          const volatile int* const lo = &s.odd_lo[count % kFlags], *const hi = &s.odd_hi[count % kFlags];
          add_odd_values<D>(a, s.items[(count - 1) % kItems], *lo, *hi, t, warp & 3, lane);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(let_go);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && s.abort) atomicCAS(a.err, 0, ZP_ERR_TIMEOUT);
  if (warp == kMmaWarp) tmem_dealloc(tbase, kTmemCols);
}

// Joins the parts of split items: one warp a row (token, head), in the order of the parts.
template <int D>
__global__ void __launch_bounds__(128) tile_join_kernel(const __grid_constant__ AttnArgs a) {
  after_previous();  // the parts are complete and visible
  next_may_start();
  const int lane = threadIdx.x & 31, heads = a.Hkv * a.G;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int64_t t = w / heads;
  if (t >= a.T) return;
  const int head = static_cast<int>(w - t * heads);
  // the request of row t: rows of none, and of requests that were skipped, have no parts
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.q_start[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int64_t q0 = a.q_start[lo], n = a.q_start[lo + 1] - q0, L = a.seq_lens[lo];
  if (q0 < 0 || t < q0 || t >= q0 + n || n > a.max_q || q0 + n > a.T || L < n || L > static_cast<int64_t>(a.max_blocks) * a.b) return;
  const float* const p = a.part + w * (D + 4);
  const int64_t step = static_cast<int64_t>(a.T) * heads * (D + 4);
  float M = -INFINITY;
  bool skip = false;
  for (int k = lane; k < a.splits; k += 32) {
    const float mk = p[k * step + D];
    skip |= isnan(mk);
    M = fmaxf(M, mk);
  }
  if (__any_sync(0xffffffffu, skip)) return;
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
  if (lane * 4 >= D) return;
  float l = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int k = 0; k < a.splits; ++k) {
    const float2 ml = *reinterpret_cast<const float2*>(p + k * step + D);
    float4 y = *reinterpret_cast<const float4*>(p + k * step + lane * 4);
    if (ml.x == -INFINITY && ml.y == 0.0f) y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);  // a part that saw nothing: its sums may be unset
    const float c = ml.x == -INFINITY ? 1.0f : ex2(ml.x - M);
    l = fmaf(ml.y, c, l);
    v[0] = fmaf(y.x, c, v[0]);
    v[1] = fmaf(y.y, c, v[1]);
    v[2] = fmaf(y.z, c, v[2]);
    v[3] = fmaf(y.w, c, v[3]);
  }
  const float inv = 1.0f / l;
  uint16_t* const out = a.out + t * a.o_ts + head * a.o_hs + lane * 4;
  const uint32_t y0 = pack_bf16x2(v[0] * inv, v[1] * inv), y1 = pack_bf16x2(v[2] * inv, v[3] * inv);
  out[0] = static_cast<uint16_t>(y0);
  out[1] = static_cast<uint16_t>(y0 >> 16);
  out[2] = static_cast<uint16_t>(y1);
  out[3] = static_cast<uint16_t>(y1 >> 16);
}

static_assert(sizeof(TileSmem<128>) + 1024 <= 227 * 1024, "shared memory of one CTA");

template <int D, bool Q_TMA, bool PARTS>
cudaError_t launch(const CUtensorMap& tm, const CUtensorMap& tq, const AttnArgs& a, const TilePlan& plan, cudaStream_t st) {
  const int nx = plan.nx, items = static_cast<int>(plan.items);
  constexpr int bytes = sizeof(TileSmem<D>) + 1024;
  static PerDeviceInit attrs;
  cudaError_t e = attrs.run(
      [] { return cudaFuncSetAttribute(tile_kernel<D, Q_TMA, PARTS>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); });
  if (e != cudaSuccess) return e;
  // Calls of one item a CTA come in early (64 queries over 16000 tokens 34.2 -> 33.4 us).  Longer ones do not: 2048-token
  // chunks take 192 us so and 196.6 when they come in early, for a reason that was not found.
  if (items <= plan.ctas) {
    e = launch_in_order(tile_kernel<D, Q_TMA, PARTS>, dim3(items), kThreads, bytes, st, 1, tm, tq, a, nx, items);
  } else {
    tile_kernel<D, Q_TMA, PARTS><<<plan.ctas, kThreads, bytes, st>>>(tm, tq, a, nx, items);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess || !PARTS) return e;
  const int64_t rows = static_cast<int64_t>(a.T) * a.Hkv * a.G;
  return launch_in_order(tile_join_kernel<D>, dim3(static_cast<unsigned>((rows + 3) / 4)), 128, 0, st, 1, a);
}

}  // namespace

TilePlan tile_plan(const zp_params* p, int T, int B, int max_q, int max_blocks, int window, int sinks, size_t room) {
  TilePlan plan{};
  plan.ctas = plan_sms();
  int64_t tokens = static_cast<int64_t>(max_blocks) * p->block_size;
  const int per_item = 2 * (kRows / (p->num_q_heads / p->num_kv_heads));
  const auto items_of = [&](int64_t n) { return (n + per_item - 1) / per_item; };  // of a request and head with n queries
  // max_q may be a loose bound: no request has more queries than the call, or than its blocks hold.
  // Splits follow the bound alone, so that a workspace for many rows is enough for fewer.
  const int64_t most = std::min<int64_t>(max_q, tokens), heads = static_cast<int64_t>(p->num_kv_heads) * B;
  const int64_t items = items_of(most) * heads;
  const int64_t nx = items_of(std::min<int64_t>(most, std::max(T, 1)));
  if (window > 0) tokens = std::min(tokens, static_cast<int64_t>(window) + per_item + sinks + 2 * p->block_size);
  const int64_t tiles = (tokens + kKeys - 1) / kKeys;
  // a part has four tiles at least: below that its sums cost more than the tiles
  const size_t part = static_cast<size_t>(std::max(T, 1)) * p->num_q_heads * (p->head_dim + 4) * sizeof(float);  // of every row
  const int64_t fit = room > kHeader ? static_cast<int64_t>(std::min<size_t>((room - kHeader) / part, INT_MAX)) : 0;
  plan.splits = static_cast<int>(std::max<int64_t>(1, std::min(std::min<int64_t>(plan.ctas / std::max<int64_t>(items, 1), tiles / 4), fit)));
  plan.nx = static_cast<int>(std::min<int64_t>(nx, INT_MAX));
  plan.items = nx * heads * plan.splits;
  plan.bytes = kHeader;
  if (plan.splits > 1 && T > 0) plan.bytes += (plan.splits * part + 255) / 256 * 256;
  return plan;
}

zp_status tile_launch(AttnArgs a, const zp_kv_pool* pool, const zp_params* p, const TilePlan& plan, void* workspace, cudaStream_t st) {
  if (plan.items > INT_MAX / 2) return ZP_ERR_UNSUPPORTED;
  if (plan.splits > 1 && static_cast<int64_t>(a.T) * p->num_q_heads > INT_MAX) return ZP_ERR_UNSUPPORTED;  // rows to join
  a.err = static_cast<int32_t*>(workspace);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kHeader);
  a.splits = plan.splits;
  const int d = p->head_dim;
  CUtensorMap tm, tq{};
  // the pool as {d, 2*Hkv*b rows per (layer, block), layers*num_blocks}; box = one block's b rows
  // of one (K or V, head), 64 columns
  if (!encode_tmap_3d_bf16(&tm, pool->base, d, static_cast<uint64_t>(2) * a.Hkv * a.b,
                           static_cast<uint64_t>(p->num_layers) * pool->num_blocks, static_cast<uint64_t>(d) * 2,
                           static_cast<uint64_t>(2) * a.Hkv * a.b * d * 2, 64, a.b, 1))
    return ZP_ERR_CUDA;
  // the queries as {d, heads, T}; rows behind the last token come as zeros
  const bool q_tma = aligned(a.q, 16) && a.q_ts > 0 && a.q_hs > 0 && a.q_ts % 8 == 0 && a.q_hs % 8 == 0 &&
                     encode_tmap_3d_bf16(&tq, a.q, d, static_cast<uint64_t>(a.Hkv) * a.G, a.T, static_cast<uint64_t>(a.q_hs) * 2,
                                         static_cast<uint64_t>(a.q_ts) * 2, 64, a.G, kRows / a.G);
  cudaError_t e;
  const auto pick = [&](auto dim, auto tma) {
    constexpr int kD = decltype(dim)::value;
    constexpr bool kTma = decltype(tma)::value;
    return plan.splits > 1 ? launch<kD, kTma, true>(tm, tq, a, plan, st) : launch<kD, kTma, false>(tm, tq, a, plan, st);
  };
  using D128 = std::integral_constant<int, 128>;
  using D64 = std::integral_constant<int, 64>;
  if (d == 128) e = q_tma ? pick(D128{}, std::true_type{}) : pick(D128{}, std::false_type{});
  else e = q_tma ? pick(D64{}, std::true_type{}) : pick(D64{}, std::false_type{});
  return e == cudaSuccess ? ZP_OK : ZP_ERR_CUDA;
}

}  // namespace zp
