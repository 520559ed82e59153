// zp_attn_tile.cuh — attention of many query rows with a sliding window and first tokens that stay
// visible, on the 5th-generation tensor cores; sm_103a.  Keys and values come from the paged bf16 pool, from the paged
// 8-bit pool, or as rows of packed prompts (Source; one translation unit each).
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
// Over the 8-bit pool four more warps bring the codes and turn them into f16, which holds them exactly, times what their
// blocks' scales are of the tile's (a power of two of them, as the library writes scales, is exact): the tile's K scale joins
// the logits', its V scale the exponent of the weights.  Queries are brought to f16 by a power of two for each row, by the
// softmax groups as they come.  P is f16, in units of 2^-15 of a reference 11 (in log2) above the largest weight times its tile's V
// scale (which may be that of another block): 11 bits down to 2^-18 of it, 2^-29 of it is the last that counts; sums of weights
// are fp32 throughout.
// 4 requests of 2048 new tokens over 0 to 6144, 32 heads on 8: 539 us, 1020 TFLOP/s over the pairs that are seen.  The tensor core
// works 49 % of the time: the softmax of a tile takes 2.3 times as long beside the warps that turn codes (without them
// the call takes 396 us), for issue slots and instruction fetches that they share.
//
// Measured: 4 requests of 2048 new tokens, 32 heads on 8, d 128, a window of 2048: 191 us, 1270 TFLOP/s
// over the pairs that are seen; a prompt of 8191 tokens, 28 heads on 4, a window of 4096: 244 us, 1480
// TFLOP/s (a dozen calls after a pause; 200 and 262 us in calls that follow one another for seconds, where
// the power limit takes the clock from 2.07 to 1.97 and 1.94 GHz).  What bounds it is the chain of one query tile: softmax of 128 x 128 logits (1100 to 1250
// cycles), hand-over to the tensor core (300), its PV and its next S (1024), and back (370), since
// with d = 128 S, S, O and O fill TMEM and the next S can only take P's place.  Two tiles in turn keep
// the tensor core at 2048 of about 2900 cycles; an item's end and start cost another two tiles' time.
// Halving the loads (K and V of every second tile) gained 5 % at most: they do not bound it.
#pragma once

#include "zp_attn.h"

#include <algorithm>
#include <cfloat>
#include <climits>
#include <cstddef>
#include <type_traits>

#include "zp_launch.h"
#include "zp_ptx.cuh"

namespace zp {
namespace {

constexpr int kRows = 128;            // rows of a query tile = TMEM lanes
constexpr int kKeys = 128;            // tokens of a KV tile
constexpr int kStages = 2;
constexpr int kKWarp = 8, kMmaWarp = 9, kCleanWarp = 10, kVWarp = 11;
// Where keys and values come from: blocks of the bf16 pool, rows of packed prompts, blocks of the 8-bit pool.
enum class Source { kPaged, kRows, kPaged8 };
template <Source SRC>
constexpr bool kCodes = SRC == Source::kPaged8;  // which a group of four warps turns into f16
// Two softmax groups, a group of the other roles, and the one that turns codes.
template <Source SRC>
constexpr int kThreads = kCodes<SRC> ? 512 : 384;
constexpr int kTurnWarp = 12;         // the first of the four
constexpr float kLazy = 24.0f, kLazyCodes = 11.0f;
constexpr float kGain = 15.0f;        // codes: log2 of what weights are multiplied by for f16
constexpr uint32_t kTmemCols = 512;   // S0 S1 O0 O1, 128 columns each
constexpr int kFlags = 16;            // items with tiles: K's warp is at most 9 ahead of a softmax group (tiles: 4 listed, 1 brought, 2 stages; 2 of the ring)

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

// A tile of codes: where its blocks are, their scales, and what the warps that turn it are to make of it.
enum { kPlainTile = 0, kMixedTile = 1, kNoMoreTiles = 2 };
struct ListedTile {
  int z[8];               // of each block: the pool's (layer, block), or past its end
  uint16_t k[8], v[8];    // for each 16 tokens: what codes are multiplied by, in f16
  float k_rest[8];        // and what K's logits are besides, where k_odd
  float k_scale, v_log, v_inv;  // of the whole tile: K's scale; V's, a power of two: its log2 (-inf: all values are 0), and 2^-kGain over it
  int row;                // of K in a block
  int what;               // V's: kPlainTile, ...
  int k_odd;
};
// Ring of them.  The warp that fills it is 4 tiles ahead of those that turn them: V of tile n + 4 is turned when the second
// product of tile n + 2 is done with the stage, so no softmax group still reads the scales of tile n when n + 8 takes its place.
constexpr int kList = 8, kListLead = 4;

template <int D, Source SRC>
struct __align__(1024) TileSmem {
  uint8_t q[2][D / 64][kRows * 128];         // [tile][64-column half][row][128 B], 128-byte swizzle
  uint8_t k[kStages][D / 64][kKeys * 128];
  uint8_t v[kStages][D / 64][kKeys * 128];
  uint8_t codes[2][4][kCodes<SRC> ? kKeys / 4 * D : 16];  // of K and V, a quarter of a tile for each warp that turns them
  uint64_t codes_full[2][4], q_turned, listed[kList], unlisted[kList];
  ListedTile list[kCodes<SRC> ? kList : 1];
  uint64_t q_full, q_empty, k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  uint64_t v_mixed[kStages], v_clean[kStages];  // in place of v_full where a tile is mixed: loaded, and looked over
  uint64_t s_full[2], p_full[2], o_full[2], o_empty[2], drain, item_full[kItems], item_empty[kItems];
  uint64_t never;                            // the test hook's, completed by nothing
  uint32_t tmem;
  int abort;
  Item items[kItems];
  int bad[kFlags], odd[kFlags];              // the last item (those with tiles, from 1) that a block id or a value marked
  int odd_lo[kFlags], odd_hi[kFlags];        // the first and last tile with such values
  int end;                                   // of what is used
};
// Bytes that a CTA asks for: any base is brought to 1024.
template <class Smem>
constexpr int used_bytes() { return static_cast<int>(offsetof(Smem, end)); }
template <int D, Source SRC>
constexpr int kSmemBytes = used_bytes<TileSmem<D, SRC>>() + 1024;


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
template <Source SRC>
__device__ __forceinline__ Raw load_raw(const AttnArgs& a, int item, int items) {
  Raw raw{0, 0, 0};
  if (item < items) {
    const int r = static_cast<int>(static_cast<uint32_t>(item) / static_cast<uint32_t>(a.splits * a.Hkv) % static_cast<uint32_t>(a.B));
    if (SRC != Source::kRows) raw.L = a.seq_lens[r];
    raw.q0 = a.q_start[r];
    raw.q1 = a.q_start[r + 1];
  }
  return raw;
}

// Items in order of queries from the last (which see the most) to the first, request, kv head,
// and part of the tiles.  False: nothing to do (`bad`: the request is reported).
template <Source SRC>
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
  w.q0 = raw.q0;
  const int64_t n = static_cast<int64_t>(raw.q1) - raw.q0;
  bad = w.q0 < 0 || n < 0 || n > a.max_q || w.q0 + n > a.T;
  w.L = SRC == Source::kRows ? static_cast<int>(n) : raw.L;
  if (SRC != Source::kRows) bad = bad || (n > 0 && (w.L < n || w.L > static_cast<int64_t>(a.max_blocks) * a.b));
  if (bad) return false;
  w.n = static_cast<int>(n);
  w.i0 = (nx - 1 - x) * 2 * qpt;
  if (w.i0 >= w.n) return false;
  w.queries = min(2 * qpt, w.n - w.i0);
  w.p0 = w.L - w.n;
  w.p_first = w.p0 + w.i0;
  w.p_last = w.p_first + w.queries - 1;
  const int bs = SRC == Source::kRows && a.b == 128 ? 7 : a.b == 16 ? 4 : 5;
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
// Whether the low or the high bf16 (or f16) of a word is not finite.
template <bool F16 = false>
__device__ __forceinline__ bool odd_lo(uint32_t x) { return (x & (F16 ? 0x7C00u : 0x7F80u)) == (F16 ? 0x7C00u : 0x7F80u); }
template <bool F16 = false>
__device__ __forceinline__ bool odd_hi(uint32_t x) { return odd_lo<F16>(x >> 16); }

// Two E4M3 codes (the low bytes) as bf16: NaN, or finite.
__device__ __forceinline__ uint32_t bf16_of_codes(uint32_t two) {
  uint32_t h;
  asm("{.reg .b16 a;\n\tcvt.u16.u32 a, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;}" : "=r"(h) : "r"(two));
  float lo, hi;
  asm("{.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;}" : "=f"(lo), "=f"(hi) : "r"(h));
  return pack_bf16x2(lo, hi);
}

// The lane's D / 32 dims of keys (kv 0) or values (1) of 8 tokens from t0 on, which stand in one block.
template <int D, Source SRC>
struct OddRows {
  static constexpr int DW = D / 64;  // words of a lane
  const uint8_t* at[2];
  int64_t step[2];                   // bytes from one token to the next
  int left;                          // tokens that there are (rows of prompts end anywhere)
  __device__ __forceinline__ OddRows(const AttnArgs& a, const Item& w, int t0, int lane) {
    left = 8;
    if constexpr (SRC == Source::kRows) {
      const int64_t t = w.q0 + t0;
      at[0] = reinterpret_cast<const uint8_t*>(a.k + t * a.k_ts + w.h * a.k_hs + lane * (2 * DW));
      at[1] = reinterpret_cast<const uint8_t*>(a.v + t * a.v_ts + w.h * a.v_hs + lane * (2 * DW));
      step[0] = a.k_ts * 2;
      step[1] = a.v_ts * 2;
      left = w.L - t0;
    } else {
      constexpr int kBytes = kCodes<SRC> ? 1 : 2;
      const int64_t tile_bytes = static_cast<int64_t>(a.b) * D * kBytes;  // of a (block, K|V, head)
      const int64_t phys = a.tables[static_cast<int64_t>(w.r) * a.max_blocks + t0 / a.b];
      const int64_t tile = (static_cast<int64_t>(a.layer) * a.num_blocks + phys) * 2 * a.Hkv + w.h;
      at[0] = a.pool + tile * tile_bytes + (t0 % a.b * D + lane * (2 * DW)) * kBytes;
      at[1] = at[0] + a.Hkv * tile_bytes;
      step[0] = step[1] = D * kBytes;
    }
  }
  // word i of token c
  __device__ __forceinline__ uint32_t word(int kv, int c, int i) const {
    const uint8_t* const p = at[kv] + c * step[kv];
    if constexpr (SRC == Source::kRows) {  // rows may start at any 2-byte address
      if (c >= left) return 0;
      const uint16_t* const x = reinterpret_cast<const uint16_t*>(p) + 2 * i;
      return static_cast<uint32_t>(x[0]) | static_cast<uint32_t>(x[1]) << 16;
    }
    if constexpr (kCodes<SRC>) return bf16_of_codes(reinterpret_cast<const uint16_t*>(p)[i]);
    return reinterpret_cast<const uint32_t*>(p)[i];
  }
};

// Adds what look_over took out of V in tiles lo to hi to the rows of one query tile that see it, whose
// results stand in memory: 32 rows a warp, D / 32 dims a lane.  Rolled and a call of its own: with its loop over
// tokens unrolled, calls that never come here took 1 % longer.
template <int D, Source SRC>
__device__ __noinline__ void add_odd_values(const AttnArgs& a, const Item& w, int lo, int hi, int t, int warp, int lane) {
  constexpr int DW = D / 64;  // words of a lane
  const int qpt = kRows / a.G;
  for (int e = lo * (kKeys / 8); e < (hi + 1) * (kKeys / 8); ++e) {
    const int j = e / (kKeys / 8), t0 = token_of(a, w, j, e % (kKeys / 8) * 8);
    if (!mixed_tile(w, j) || e * 8 >= w.blocks * a.b || whole8(a, w, t0)) continue;
    const OddRows<D, SRC> rows(a, w, t0, lane);
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
      for (int i = 0; i < DW; ++i) top = max_u16x2(top, rows.word(1, c, i) & 0x7FFF7FFFu);
    if (!__any_sync(0xffffffffu, odd_lo(top) || odd_hi(top))) continue;
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
      uint32_t x[DW];
      bool odd = false;
#pragma unroll
      for (int i = 0; i < DW; ++i) {
        x[i] = rows.word(1, c, i);
        odd |= odd_lo(x[i]) || odd_hi(x[i]);
      }
      if (!seen_by_some(a, w, t0 + c) || !__any_sync(0xffffffffu, odd)) continue;
      // A weight of 0 (a logit of -inf) makes NaN of it, and only an infinite key can give one; a key of
      // NaN has made the whole row NaN.
      uint32_t kw[DW];
      bool inf = false, nan = false;
#pragma unroll
      for (int i = 0; i < DW; ++i) {
        kw[i] = rows.word(0, c, i);
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
template <int D, bool F16>
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
  if (!__any_sync(0xffffffffu, odd_lo<F16>(top) || odd_hi<F16>(top))) return false;
  for (todo = look; todo; todo &= todo - 1) {
    const int g = __ffs(todo) - 1;
#pragma unroll 1
    for (int y = 0; y < kLoads; ++y) {
      uint32_t* const x = reinterpret_cast<uint32_t*>(v + (ch >> 3) * (kKeys * 128) + (y * kPer + sub) * 128 + (((ch & 7) ^ (y * kPer + sub)) << 4) + g * 1024);
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        uint32_t z = x[i];
        if (odd_lo<F16>(z)) z &= 0xFFFF0000u;
        if (odd_hi<F16>(z)) z &= 0x0000FFFFu;
        x[i] = z;
      }
    }
  }
  return true;
}

// Keys or values of list tile j from rows at any address (one warp), where the copies would have put them; zeros
// behind the prompt's end.
template <int D>
__device__ __forceinline__ void load_rows(const AttnArgs& a, const Item& w, int j, int kv, uint8_t* tile, int lane) {
  for (int row = lane; row < kKeys; row += 32) {
    const int tk = token_of(a, w, j, row);
    const bool have = (j * kKeys + row) < w.blocks * a.b && tk < w.L;
    const uint16_t* const x = (kv ? a.v + (w.q0 + tk) * a.v_ts + w.h * a.v_hs : a.k + (w.q0 + tk) * a.k_ts + w.h * a.k_hs);
    for (int c = 0; c < D / 8; ++c) {
      uint32_t y[4] = {0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (have) y[e] = static_cast<uint32_t>(x[c * 8 + 2 * e]) | static_cast<uint32_t>(x[c * 8 + 2 * e + 1]) << 16;
      *reinterpret_cast<uint4*>(tile + (c >> 3) * (kKeys * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// E4M3 codes of 4 bytes as two pairs of f16, which holds them (NaN too) exactly.
__device__ __forceinline__ void f16_of_codes(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;}" : "=r"(lo), "=r"(hi) : "r"(w));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Turns a quarter of a tile (32 tokens) from codes into f16(code * factor), a factor for each 16 tokens, in the place and
// order that a bf16 tile has (one warp).  `refill` starts the next copy into the codes' place: every lane has used its loads.
// What bounds it is how fast one warp gets its instructions beside the softmax groups (8 cycles each), so it is a short loop
// over 8 tokens at a time, whose code stays at hand: 2048-token chunks of 4 requests over 0 to 6144 tokens took 532 us so, 622
// unrolled, and took 740 with values turned into bf16 by 6 integer steps a pair in place of a conversion and a product.
template <int D, class Refill>
__device__ __forceinline__ void turn_quarter(uint32_t codes, uint32_t tile, const uint16_t* factors, int quarter, int lane, const Refill& refill) {
  constexpr int N = D / 64;  // 16-byte pieces of a lane, of 8 tokens
  // Which piece (row, 16 codes): 8 lanes at a time read and write every bank once.  With 8 pieces a row, lanes 4 to 7 of
  // 8 have the row whose bits 0 and 2 differ from the others'; the second piece's row differs in bit 2.
  const int sub = lane & 7, ch = D == 128 ? (sub & 3) + ((lane >> 3) & 1) * 4 : lane & 3;
  const int row = D == 128 ? ((lane >> 4) * 2) ^ ((sub >> 2) * 5) : lane >> 2;
  uint32_t from = codes + row * D + ((D == 128 ? ch ^ (row & 7) : ch ^ ((row >> 1) & 3)) << 4);
  uint32_t to = tile + (ch >> 2) * (kKeys * 128) + (quarter * 32 + row) * 128 + ((((ch & 3) * 2) ^ (row & 7)) << 4);
  constexpr uint32_t kSecond = 4 * 128 + (4 << 4);
  uint4 x[N];
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = lds16(i ? from ^ kSecond : from);
#pragma unroll 1
  for (int g = 0; g < 4; ++g) {
    const uint32_t f = factors[quarter * 2 + (g >> 1)] * 0x10001u;
    from += 8 * D;
    uint4 next[N];
    if (g < 3)
#pragma unroll
      for (int i = 0; i < N; ++i) next[i] = lds16(i ? from ^ kSecond : from);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      uint32_t y[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f16_of_codes(w[e], y[2 * e], y[2 * e + 1]);
        y[2 * e] = mul_f16x2(y[2 * e], f);
        y[2 * e + 1] = mul_f16x2(y[2 * e + 1], f);
      }
      const uint32_t at = i ? to ^ kSecond : to;
      sts16(at, make_uint4(y[0], y[1], y[2], y[3]));
      sts16(at ^ 16, make_uint4(y[4], y[5], y[6], y[7]));
    }
    to += 8 * 128;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = next[i];
  }
  refill();
}

// The part of one of the four warps that bring and turn codes: a quarter of each tile.
template <int D, class Smem>
__device__ __forceinline__ void turn_codes(Smem& s, const CUtensorMap& tm, const AttnArgs& a, int quarter, int lane, volatile int* abort) {
  const uint32_t k = smem_u32(s.k[0][0]), v = smem_u32(s.v[0][0]);
  const int bpq = kKeys / 4 / a.b;  // blocks of a quarter
  uint32_t fetched[2] = {0, 0};
  const auto listed = [&](uint32_t n) { return __all_sync(0xffffffffu, wait(&s.listed[n % kList], (n / kList) & 1, abort)) != 0; };
  const auto fetch = [&](uint32_t n, int kv) {
    const ListedTile& e = s.list[n % kList];
    if (lane == 0) mbar_arrive_expect_tx(&s.codes_full[kv][quarter], kKeys / 4 * D);
    __syncwarp();
    if (lane < bpq)
      tma_load_3d(s.codes[kv][quarter] + lane * a.b * D, &tm, &s.codes_full[kv][quarter], 0, e.row + kv * a.Hkv * a.b, e.z[quarter * bpq + lane]);
    ++fetched[kv];
  };
  bool go = listed(0);
  if (go && s.list[0].what != kNoMoreTiles) {
    fetch(0, 0);
    fetch(0, 1);
    for (uint32_t n = 0; go; ++n) {
      const uint32_t st = n % kStages, ph = (n / kStages) & 1;
      const ListedTile& e = s.list[n % kList];
      go = listed(n + 1);
      if (!go) break;
      const bool more = s.list[(n + 1) % kList].what != kNoMoreTiles;
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        uint64_t* const empty = kv ? &s.v_empty[st] : &s.k_empty[st];
        go = __all_sync(0xffffffffu, wait(&s.codes_full[kv][quarter], n & 1, abort) && (n < kStages || wait(empty, ph ^ 1, abort)));
        if (!go) break;
        turn_quarter<D>(smem_u32(s.codes[kv][quarter]), (kv ? v : k) + st * (kKeys * D * 2), kv ? e.v : e.k, quarter, lane, [&] {
          __syncwarp();
          if (more) fetch(n + 1, kv);
        });
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(!kv ? &s.k_full[st] : e.what == kMixedTile ? &s.v_mixed[st] : &s.v_full[st]);
          if (kv) mbar_arrive(&s.unlisted[n % kList]);
        }
      }
      if (!go) break;
      go = more;
    }
  }
  // copies still in flight after a give-up land before the shared memory is released
  if (lane == 0)
    for (int kv = 0; kv < 2; ++kv)
      if (fetched[kv] > 0) mbar_wait_bounded(&s.codes_full[kv][quarter], (fetched[kv] - 1) & 1, kWaitNs);
  __syncwarp();
}

// Brings a row of queries to f16 in place, by a power of two that brings its largest magnitude to [2^14, 2^15): exact for
// values down to 2^-31 of it, less than the fp32 sums hold.  Returns what the logits are then multiplied by.
template <int D>
__device__ __forceinline__ float turn_queries(uint8_t* q, int row) {  // q: [64-column half][row][128 B]
  const uint32_t at = smem_u32(q) + row * 128;
  uint32_t m = 0;
  const auto piece = [&](int c) { return at + (c >> 3) * (kRows * 128) + (((c & 7) ^ (row & 7)) << 4); };
#pragma unroll
  for (int c = 0; c < D / 8; ++c) {
    const uint4 x = lds16(piece(c));
    m = max_u16x2(max_u16x2(m, x.x & 0x7FFF7FFFu), max_u16x2(x.y & 0x7FFF7FFFu, max_u16x2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
  }
  const int ex = min(max(static_cast<int>(max(m & 0xFFFFu, m >> 16) >> 7), 15), 253);  // both powers of two are normal
  const float inv = __uint_as_float(static_cast<uint32_t>(268 - ex) << 23);
#pragma unroll 4
  for (int c = 0; c < D / 8; ++c) {
    const uint4 x = lds16(piece(c));
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = pack_f16x2(bf16x2_lo(w[e]) * inv, bf16x2_hi(w[e]) * inv);
    sts16(piece(c), make_uint4(y[0], y[1], y[2], y[3]));
  }
  return __uint_as_float(static_cast<uint32_t>(ex - 14) << 23);
}

// Q_TMA: the queries' rows are aligned and come by TMA (one box per tile and 64-column half: the
// group's heads of 128 / G tokens, which is the order of the tile's rows); else by plain loads.
// PARTS: items are split, and leave sums for the joining kernel.
// tm: the pool, or the keys of prompts; tv: the values of prompts.
template <int D, bool Q_TMA, bool PARTS, Source SRC>
__global__ void __launch_bounds__(kThreads<SRC>, 1) tile_kernel(const __grid_constant__ CUtensorMap tm, const __grid_constant__ CUtensorMap tv,
                                                                  const __grid_constant__ CUtensorMap tq, const __grid_constant__ AttnArgs a,
                                                                  int nx, int items) {
  constexpr int NH = D / 64;
  extern __shared__ uint8_t dyn[];
  using Smem = TileSmem<D, SRC>;
  Smem& s = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t(1023));
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
    mbar_init(&s.q_empty, PARTS ? 9 : 1);  // parts go out through the queries' place: the softmax groups let go of it too
    mbar_init(&s.drain, 1);
    mbar_init(&s.never, 1);
    constexpr int kFills = kCodes<SRC> ? 4 : 1;  // warps that fill a stage
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.k_full[i], kFills);
      mbar_init(&s.k_empty[i], 1);
      mbar_init(&s.v_full[i], kFills);
      mbar_init(&s.v_empty[i], 1);
      mbar_init(&s.v_mixed[i], kFills);
      mbar_init(&s.v_clean[i], 1);
    }
    if (kCodes<SRC>) {
      mbar_init(&s.q_turned, 8);
      for (int i = 0; i < 8; ++i) mbar_init(&s.codes_full[i >> 2][i & 3], 1);
      for (int i = 0; i < kList; ++i) {
        mbar_init(&s.listed[i], 1);
        mbar_init(&s.unlisted[i], 4);
      }
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
    if (SRC != Source::kRows || a.kv_tma) prefetch_tensormap(&tm);
    if (SRC == Source::kRows && a.kv_tma) prefetch_tensormap(&tv);
    if (Q_TMA) prefetch_tensormap(&tq);
  }
  // rows of the query tiles that no query has filled start as zeros
  for (int i = tid; i < static_cast<int>(sizeof(s.q) / 16); i += kThreads<SRC>)
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
  // softmax groups spill inside their loop (2048-token chunks 210 us, 200 us with 208).  With codes to turn:
  // 2 x 128 x 192 + 2 x 128 x 64 of 512 x 128 (200 with 48 for those that turn them, or 192 with 80 and 48, took 589 us where
  // this took 532: 2048-token chunks of 4 requests over 0 to 6144 tokens).  The roles of 64 registers spill 144 to 152 bytes a thread with
  // D 128 and 92 with 64, and nothing with 96.
  if (kCodes<SRC> && warp >= kTurnWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if constexpr (kCodes<SRC>) turn_codes<D>(s, tm, a, warp - kTurnWarp, lane, abort);
  } else if (warp >= 8) {
  if constexpr (kCodes<SRC>) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  Item w;
  bool bad;
  Raw raw = load_raw<SRC>(a, blockIdx.x, items);
  int count = 0;       // items with work so far
  int walked = 0;      // those of them that have tiles
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
      raw = load_raw<SRC>(a, next_item(item), items);
      if (!take_item<SRC>(a, item, nx, now, w, bad)) {
        if (bad && lane == 0) atomicCAS(a.err, 0, ZP_ERR_BAD_TABLE);
        continue;
      }
      ++count;
      walked += w.j0 < w.j1;
      const int32_t* const table = a.tables + static_cast<int64_t>(w.r) * a.max_blocks;
      const auto id_of = [&](int j) {  // block id that the lane loads for tile j
        const int e = j * bpt + lane;
        if (lane >= bpt || e >= w.blocks || j >= w.j1) return 0;
        const int block = e < w.sink_blocks ? e : w.win_block + e - w.sink_blocks;
        return SRC == Source::kRows ? block : table[block];
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
      if (kCodes<SRC> && kv) {  // V's warp brings the queries alone
        load_q();
        continue;
      }
      if (!kCodes<SRC> && !kv && w.j0 == w.j1) load_q();  // a part without tiles
      int id = id_of(w.j0);
      for (int j = w.j0; go && j < w.j1; ++j, ++done) {
        const uint32_t st = done % kStages, ph = (done / kStages) & 1;
        const int nb = min(bpt, w.blocks - j * bpt);
        // an id outside the pool: the item's rows are not written, and block 0 is read in its place
        const bool out = SRC != Source::kRows && (id < 0 || id >= a.num_blocks);
        if (SRC != Source::kRows && __any_sync(0xffffffffu, out) && lane == 0) {
          *reinterpret_cast<volatile int*>(&s.bad[walked % kFlags]) = walked;
          atomicCAS(a.err, 0, ZP_ERR_BAD_TABLE);
        }
        // blocks past the list's end have a coordinate past the tensor's: they come as zeros
        const int z = SRC == Source::kRows ? (lane < nb ? w.q0 + id * a.b : a.T)
                      : lane < nb          ? a.layer * static_cast<int>(a.num_blocks) + (out ? 0 : id)
                                           : a.layers * static_cast<int>(a.num_blocks);
        const int now_id = id;
        id = id_of(j + 1);
        if constexpr (kCodes<SRC>) {  // K's warp lists the tiles, the ones that turn them bring them
          const int64_t at = (static_cast<int64_t>(a.layer) * a.num_blocks + (out ? 0 : now_id)) * 2 * a.Hkv + w.h;
          const float k_scale = lane < nb ? a.scales[at] : 0.0f, v_scale = lane < nb ? a.scales[at + a.Hkv] : 0.0f;
          if (done >= kListLead) {
            const uint32_t before = done - kListLead;
            go = __all_sync(0xffffffffu, wait(&s.unlisted[before % kList], (before / kList) & 1, abort)) != 0;
            if (!go) break;
          }
          // The tile's own scales, and what its blocks' are of them.  K: the largest; where another is not a power of two
          // (or 0) of 2^-15 or more times it, which f16 takes exactly, the logits are scaled instead.  V: a power of two, at
          // least the largest, from 2^-104 to 2^104 (sums of weights are divided by it).
          const float k_top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(k_scale))));
          const uint32_t v_bits = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(v_scale)));
          const int v_exp = v_bits == 0 ? 0 : min(max(static_cast<int>(v_bits >> 23) - 127 + ((v_bits & 0x7FFFFFu) != 0), -104), 104);
          const float k_all = k_top > 0.0f ? k_top : 1.0f, k_of = k_scale / k_all;
          const float v_of = v_scale * __uint_as_float(static_cast<uint32_t>(127 - v_exp) << 23);
          const bool odd = __any_sync(0xffffffffu, k_of != 0.0f && ((__float_as_uint(k_of) & 0x7FFFFFu) != 0 || fabsf(k_of) < 0x1p-15f));
          ListedTile& e = s.list[done % kList];
          const int of = a.b == 16 ? lane & 7 : (lane & 7) >> 1;  // the block of 16 tokens
          const float k16 = __shfl_sync(0xffffffffu, k_of, of), v16 = __shfl_sync(0xffffffffu, v_of, of);
          if (lane < 8) {
            e.z[lane] = z;
            e.k[lane] = odd ? 0x3C00 : static_cast<uint16_t>(pack_f16x2(k16, 0.0f));
            e.v[lane] = static_cast<uint16_t>(pack_f16x2(v16, 0.0f));
            e.k_rest[lane] = k16;
          }
          if (lane == 0) {
            e.k_scale = k_all;
            e.v_log = v_bits == 0 ? -INFINITY : static_cast<float>(v_exp);
            e.v_inv = __uint_as_float(static_cast<uint32_t>(127 - v_exp - static_cast<int>(kGain)) << 23);
            e.row = w.h * a.b;
            e.what = mixed_tile(w, j) ? kMixedTile : kPlainTile;
            e.k_odd = odd;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.listed[done % kList]);
          continue;
        }
        uint64_t* full = kv ? &s.v_full[st] : &s.k_full[st];
        uint32_t* used = &used_full;
        if (kv && mixed_tile(w, j)) {
          full = &s.v_mixed[st];
          used = &used_mixed;
        }
        const bool tma = SRC != Source::kRows || a.kv_tma;
        if (lane == 0) {
          if (done >= kStages) go = wait(&empties[st], ph ^ 1, abort);
          if (go && tma) mbar_arrive_expect_tx(full, kKeys * D * 2);
        }
        go = __shfl_sync(0xffffffffu, go, 0);
        if (!go) break;
        if (!tma) {
          load_rows<D>(a, w, j, kv, kv ? s.v[st][0] : s.k[st][0], lane);
          if (lane == 0) mbar_arrive(full);
        } else if (lane < bpt) {
#pragma unroll
          for (int hd = 0; hd < NH; ++hd) {
            uint8_t* const to = (kv ? s.v[st][hd] : s.k[st][hd]) + lane * a.b * 128;
            if constexpr (SRC == Source::kRows) tma_load_3d(to, kv ? &tv : &tm, full, hd * 64, w.h, z);
            else tma_load_3d(to, &tm, full, hd * 64, (kv * a.Hkv + w.h) * a.b, z);
          }
        }
        if (!kv && j == w.j0) load_q();
        last[st] = full;
        last_parity = (last_parity & ~(1u << st)) | (*used & (1u << st));
        *used ^= 1u << st;
        __syncwarp();
      }
    }
    if (kCodes<SRC> && go && !kv && lane == 0) {  // the list's end
      const uint32_t before = done - kListLead;
      if (done < kListLead || wait(&s.unlisted[before % kList], (before / kList) & 1, abort)) {
        s.list[done % kList].what = kNoMoreTiles;
        mbar_arrive(&s.listed[done % kList]);
      }
    }
    __syncwarp();
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
      raw = load_raw<SRC>(a, next_item(item), items);
      if (!take_item<SRC>(a, item, nx, now, w, bad)) continue;
      walked += w.j0 < w.j1;
      for (int j = w.j0; j < w.j1; ++j) {
        if (!mixed_tile(w, j)) continue;
        const uint32_t st = (tiles + static_cast<uint32_t>(j - w.j0)) % kStages;
        go = __all_sync(0xffffffffu, wait(&s.v_mixed[st], (seen_mixed >> st) & 1, abort));
        if (!go) break;
        seen_mixed ^= 1u << st;
        if (look_over<D, kCodes<SRC>>(a, w, j, s.v[st][0], lane) && lane == 0) {
          const int f = walked % kFlags;
          if (s.odd[f] != walked) s.odd[f] = walked, s.odd_lo[f] = j;
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
    const uint32_t idesc_s = kCodes<SRC> ? idesc_f16_f32(kRows, kKeys) : idesc_bf16_f32(kRows, kKeys);
    const uint32_t idesc_o = (kCodes<SRC> ? idesc_f16_f32(kRows, D) : idesc_bf16_f32(kRows, D)) | kTransposeB;
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
        raw = load_raw<SRC>(a, item, items);
        have = take_item<SRC>(a, cur, nx, now, next, bad);
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
      ok = wait_all(kCodes<SRC> ? &s.q_turned : &s.q_full, count & 1);
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
    if constexpr (kCodes<SRC>) asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    int count = 0, walked = 0;  // items so far, and those with tiles
    const int t = warp >> 2, row = tid & 127;
    const int qi = row / a.G, gi = row - qi * a.G;
    const int i = t * qpt + qi;  // query of the item
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tbase + lanes + t * kKeys, to = tbase + lanes + 256 + t * 128;
    const uint64_t sl2x2 = pair2(a.sl2);
    uint32_t s_seen = 0, o_seen = 0;
    uint32_t scale_tile = 0;  // tiles of the items before, of both groups
    bool ok = true;
    while (true) {
      ok = __all_sync(0xffffffffu, wait(&s.item_full[count % kItems], (count / kItems) & 1, abort));
      if (!ok) break;
      const Item& w = s.items[count % kItems];  // stays until every warp has let go of it
      uint64_t* const let_go = &s.item_empty[count % kItems];
      if (w.r < 0) break;
      ++count;
      float gain = 1.0f;  // of the row's logits, where its queries were turned
      // Also a group without rows waits for the item's queries, which come when both groups are done with those before: what it
      // arrives at below belongs to this item then, however many it has no part in.
      if (kCodes<SRC> || (PARTS && t == 1 && !w.two)) {
        ok = __all_sync(0xffffffffu, wait(&s.q_full, (count - 1) & 1, abort));
        if (!ok) break;
      }
      if constexpr (kCodes<SRC>) {
        if (t == 0 || w.two) {
          gain = turn_queries<D>(s.q[t][0], row);
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.q_turned);
      }
      if (t == 1 && !w.two) {
        if (kCodes<SRC>) scale_tile += static_cast<uint32_t>(w.j1 - w.j0);
        __syncwarp();
        if (lane == 0) mbar_arrive(let_go);
        if (PARTS && lane == 0) mbar_arrive(&s.q_empty);
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
        float sl2 = a.sl2, v_log = 0.0f, v_inv = 0.0f;  // of the tile
        if constexpr (kCodes<SRC>) {
          const uint32_t slot = scale_tile % kList;
          ok = __all_sync(0xffffffffu, wait(&s.listed[slot], (scale_tile / kList) & 1, abort));
          if (!ok) break;
          ++scale_tile;
          const ListedTile& e = s.list[slot];
          // a normal number: 0 (queries of 0 beside small keys) or infinity would make NaN of what a row does not see, or of logits of 0
          sl2 = fminf(fmaxf(sl2 * (e.k_scale * gain), FLT_MIN), FLT_MAX);
          v_log = e.v_log;
          v_inv = e.v_inv;
          if (e.k_odd) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int f = 0; f < 32; ++f) x[c][f] = __float_as_uint(__uint_as_float(x[c][f]) * e.k_rest[2 * c + (f >> 4)]);
          }
        }
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
        const float all = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        if (kCodes<SRC> && v_log == -INFINITY) {
          // Values of 0 count in the sum of weights alone, so any power of two may stand for their scale: the row's own, that
          // which leaves its reference where it is, or the least where it has none yet.  (One of the item, or of what the CTA had
          // before, set references that the row's other values were lost beside.)
          v_log = fmaxf(fminf(floorf(m - kLazyCodes - all * sl2), 104.0f), -104.0f);
          v_inv = __uint_as_float(static_cast<uint32_t>(127 - static_cast<int>(v_log) - static_cast<int>(kGain)) << 23);
        }
        const float top = kCodes<SRC> ? fmaf(all, sl2, v_log) : all * a.sl2;
        if (__any_sync(0xffffffffu, top > m)) {
          const float mn = fmaxf(m, top + (kCodes<SRC> ? kLazyCodes : kLazy)), corr = m == -INFINITY ? 0.0f : ex2(m - mn);
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
          if constexpr (kCodes<SRC>) {
            // in two steps: behind values of 0 the reference may rise by 2^208, and what they count has to stay
            const float half = m == -INFINITY ? 0.0f : ex2(0.5f * (m - mn));
            l = l * half * half;
          } else {
            l *= corr;
          }
          m = mn;
        }
        const uint64_t ref = pair2((m == -INFINITY ? 0.0f : -m) + (kCodes<SRC> ? v_log + kGain : 0.0f));
        const uint64_t by = kCodes<SRC> ? pair2(sl2) : sl2x2;
        uint64_t sum = 0;  // a pair of +0
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const uint32_t (&src)[32] = x[2 * c + (e >> 4)];
            float y0, y1;
            unpair(fma2(pair(src[(2 * e) & 31], src[(2 * e + 1) & 31]), by, ref), y0, y1);
            y0 = ex2(y0);
            y1 = ex2(y1);
            sum = add2(sum, pair(__float_as_uint(y0), __float_as_uint(y1)));
            pk[e] = kCodes<SRC> ? pack_f16x2(y0, y1) : pack_bf16x2(y0, y1);
          }
          tmem_st32(ts + c * 32, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.p_full[t]);
        float a0, a1;
        unpair(sum, a0, a1);
        if (kCodes<SRC>) l = fmaf(a0 + a1, v_inv, l);
        else l += a0 + a1;
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
      walked += !empty;
      const bool marked = !empty && *reinterpret_cast<volatile int*>(&s.bad[walked % kFlags]) == walked;
      const bool odd = !empty && *reinterpret_cast<volatile int*>(&s.odd[walked % kFlags]) == walked;
      const bool write = have && !marked;
      if (to_row.part && (write || marked || empty)) {
        to_row.part[D] = marked ? NAN : m;  // a maximum is never NaN: marks a part with a bad block id
        to_row.part[D + 1] = l;
      }
      if (!empty) {
        // a row sees itself; logits of -inf alone give 0 / 0, as their softmax
        const float unit = kCodes<SRC> ? 0x1p-15f : 1.0f, inv = unit / l;
        static_assert(kGain == 15.0f, "unit");
        // Rolled: code that runs once an item comes from far away, and its size is time.
        if constexpr (PARTS) {
          // Through shared memory, 128 bytes of each row at a time, so that 8 lanes write one row's: in the place of the item's
          // queries, which it is done with and which the next one's take when every warp has let go (q_empty).
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
            {
              if (kCodes<SRC>)
#pragma unroll
                for (int f = 4 * e; f < 4 * e + 4; ++f) o[f] = __float_as_uint(__uint_as_float(o[f]) * unit);
              sts16(put + ((e ^ (lane & 7)) << 4), make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]));
            }
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
          const volatile int* const lo = &s.odd_lo[walked % kFlags], *const hi = &s.odd_hi[walked % kFlags];
          add_odd_values<D, SRC>(a, s.items[(count - 1) % kItems], *lo, *hi, t, warp & 3, lane);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(let_go);
      if (PARTS) {
        fence_proxy_async_smem();  // the rows that went through it, ahead of the next copy
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.q_empty);
      }
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
  const int64_t q0 = a.q_start[lo], n = a.q_start[lo + 1] - q0, L = a.seq_lens ? a.seq_lens[lo] : n;
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
    if (c == 0.0f) {  // values of 0 alone in one part, large ones in another: they count in the sum of weights
      const float half = ex2(0.5f * (ml.x - M));
      l = fmaf(ml.y * half, half, l);
    } else {
      l = fmaf(ml.y, c, l);
    }
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

static_assert(kSmemBytes<128, Source::kPaged> <= 227 * 1024 && kSmemBytes<128, Source::kPaged8> <= 227 * 1024, "shared memory of one CTA");

template <int D, bool Q_TMA, bool PARTS, Source SRC>
cudaError_t launch(const CUtensorMap& tm, const CUtensorMap& tv, const CUtensorMap& tq, const AttnArgs& a, const TilePlan& plan, cudaStream_t st) {
  const int nx = plan.nx, items = static_cast<int>(plan.items);
  constexpr int bytes = kSmemBytes<D, SRC>;
  static PerDeviceInit attrs;
  cudaError_t e = attrs.run(
      [] { return cudaFuncSetAttribute(tile_kernel<D, Q_TMA, PARTS, SRC>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); });
  if (e != cudaSuccess) return e;
  // Calls of one item a CTA come in early (64 queries over 16000 tokens 34.2 -> 33.4 us).  Longer ones do not: 2048-token
  // chunks take 192 us so and 196.6 when they come in early, for a reason that was not found.
  if (items <= plan.ctas) {
    e = launch_in_order(tile_kernel<D, Q_TMA, PARTS, SRC>, dim3(items), kThreads<SRC>, bytes, st, 1, tm, tv, tq, a, nx, items);
  } else {
    tile_kernel<D, Q_TMA, PARTS, SRC><<<plan.ctas, kThreads<SRC>, bytes, st>>>(tm, tv, tq, a, nx, items);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess || !PARTS) return e;
  const int64_t rows = static_cast<int64_t>(a.T) * a.Hkv * a.G;
  return launch_in_order(tile_join_kernel<D>, dim3(static_cast<unsigned>((rows + 3) / 4)), 128, 0, st, 1, a);
}

// Launches the kernel for keys and values that `tm` (and `tv`) describe.
template <Source SRC>
zp_status launch_tiles(AttnArgs a, const zp_params* p, const TilePlan& plan, void* workspace, cudaStream_t st, const CUtensorMap& tm,
                       const CUtensorMap& tv) {
  if (plan.items > INT_MAX / 2) return ZP_ERR_UNSUPPORTED;
  if (plan.splits > 1 && static_cast<int64_t>(a.T) * p->num_q_heads > INT_MAX) return ZP_ERR_UNSUPPORTED;  // rows to join
  a.err = static_cast<int32_t*>(workspace);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kHeader);
  a.splits = plan.splits;
  const int d = p->head_dim;
  CUtensorMap tq{};
  // the queries as {d, heads, T}; rows behind the last token come as zeros
  const bool q_tma = aligned(a.q, 16) && a.q_ts > 0 && a.q_hs > 0 && a.q_ts % 8 == 0 && a.q_hs % 8 == 0 &&
                     encode_tmap_3d_bf16(&tq, a.q, d, static_cast<uint64_t>(a.Hkv) * a.G, a.T, static_cast<uint64_t>(a.q_hs) * 2,
                                         static_cast<uint64_t>(a.q_ts) * 2, 64, a.G, kRows / a.G);
  cudaError_t e;
  const auto pick = [&](auto dim, auto tma) {
    constexpr int kD = decltype(dim)::value;
    constexpr bool kTma = decltype(tma)::value;
    return plan.splits > 1 ? launch<kD, kTma, true, SRC>(tm, tv, tq, a, plan, st) : launch<kD, kTma, false, SRC>(tm, tv, tq, a, plan, st);
  };
  using D128 = std::integral_constant<int, 128>;
  using D64 = std::integral_constant<int, 64>;
  if (d == 128) e = q_tma ? pick(D128{}, std::true_type{}) : pick(D128{}, std::false_type{});
  else e = q_tma ? pick(D64{}, std::true_type{}) : pick(D64{}, std::false_type{});
  return e == cudaSuccess ? ZP_OK : ZP_ERR_CUDA;
}

}  // namespace
}  // namespace zp
