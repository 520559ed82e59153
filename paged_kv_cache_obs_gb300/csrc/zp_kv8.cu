// zp_kv8.cu — the 8-bit pool: quantising keys and values as they enter the cache, and whole
// blocks to and from the bf16 pool; sm_103a.
//
// A tile is the b x d values of one (layer, block, K|V, head).  Its scale is a power of two,
//   s = 2^e, e = max(ceil(log2(amax / 448)), -126),
// read off the exponent and mantissa of the tile's largest finite magnitude, and a code is
// e4m3(x / s), one rounding (x / s is exact).  The power of two costs up to one bit of E4M3's
// range of 17 powers of two and none of its precision; in return dividing is exact, reading back
// to bf16 is exact, and raising a tile's scale later only moves the exponents of its codes.
//
// All kernels give a tile to one warp, which holds it in registers: values are read once, the
// maximum is a warp reduction, and nothing is staged.  They are bound by HBM (2 bytes read and
// 1 written a value, or the reverse).  Measured: 1016 blocks of 32 layers and 8 heads packed in 447 us
// (7.1 TB/s), 64 blocks of 28 layers and 4 heads read back in 27.6 us (6.4 TB/s), 8200 new tokens of 8
// heads appended in 10.7 us (4.7 TB/s: a chain of dependent loads before the values are needed, in 2176 CTAs,
// 1.43 times what the SMs hold at once), 256 single ones in 4.8 us (the same chain, with nothing behind it).
#include "zp_internal.h"
#include "zp_launch.h"
#include "zp_ptx.cuh"

namespace zp {
namespace {

constexpr int kWarpsQ = 4;
constexpr int kThreadsQ = kWarpsQ * 32;

__device__ __forceinline__ void record(int32_t* err, int code) { atomicCAS(err, 0, code); }

// ---- E4M3 ---------------------------------------------------------------------------------

// Two fp32 values to two codes (lo in the low byte), to nearest even; NaN gives 0x7F.  Values are
// at most 448 in size here, so the saturation never acts on finite ones.
__device__ __forceinline__ uint32_t enc2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two codes to two fp32 values (exact; by way of f16, which holds every E4M3 value).
__device__ __forceinline__ float2 dec2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  float lo, hi;
  asm("{.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;}" : "=f"(lo), "=f"(hi) : "r"(h));
  return make_float2(lo, hi);
}
// Largest magnitude of bf16 pairs, as two 15-bit patterns (which order like the values); inf and
// NaN come out as 0x7F80 and above.
__device__ __forceinline__ uint32_t amax2(uint32_t m, uint32_t x) {
  return max_u16x2(m, x & 0x7FFF7FFFu);
}
// The same over the finite values only.
__device__ __forceinline__ uint32_t amax2_finite(uint32_t m, uint32_t x) {
  if ((x & 0x7F80u) == 0x7F80u) x &= 0xFFFF0000u;
  if ((x & 0x7F800000u) == 0x7F800000u) x &= 0xFFFFu;
  return amax2(m, x);
}

// The scale of a tile whose largest finite magnitude has the bf16 bits `m`: with
// amax = 1.f * 2^(E - 127), amax / 448 <= 2^(E - 135) when 1.f <= 1.75 (mantissa bits <= 0x60),
// else 2^(E - 134); never below 2^-126 (biased exponent 1), so that 1/s is finite.
__device__ __forceinline__ float scale_of(uint32_t m) {
  if (m == 0) return 0.0f;
  const int e = max(static_cast<int>(m >> 7) - 8 + ((m & 0x7Fu) > 0x60u ? 1 : 0), 1);
  return __uint_as_float(static_cast<uint32_t>(e) << 23);
}
__device__ __forceinline__ float inverse(float s) { return s > 0.0f ? 1.0f / s : 0.0f; }  // exact for powers of two

// Two bf16 values to two codes.  ODD: some value of the tile is not finite; infinities become NaN
// (E4M3 has none).
template <bool ODD>
__device__ __forceinline__ uint32_t enc_pair(uint32_t x, float inv) {
  uint32_t c = enc2(bf16x2_lo(x) * inv, bf16x2_hi(x) * inv);
  if (ODD && (x & 0x7F80u) == 0x7F80u) c |= 0x7Fu;
  if (ODD && (x & 0x7F800000u) == 0x7F800000u) c |= 0x7F00u;
  return c;
}
template <bool ODD>
__device__ __forceinline__ uint2 enc8(const uint4& x, float inv) {
  return make_uint2(enc_pair<ODD>(x.x, inv) | enc_pair<ODD>(x.y, inv) << 16,
                    enc_pair<ODD>(x.z, inv) | enc_pair<ODD>(x.w, inv) << 16);
}

__device__ __forceinline__ uint32_t warp_max(uint32_t m) {
  return __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
}

// The tile's largest finite magnitude (bf16 bits) over the warp's registers; `odd`: some value is
// not finite.  Two instructions a pair of values, and a second look only for tiles that need it.
template <int NL>
__device__ __forceinline__ uint32_t tile_amax(const uint4 (&w)[NL], bool& odd) {
  uint32_t m = 0;
#pragma unroll
  for (int l = 0; l < NL; ++l) m = amax2(amax2(amax2(amax2(m, w[l].x), w[l].y), w[l].z), w[l].w);
  m = warp_max(m);
  odd = m >= 0x7F80u;
  if (odd) {
    m = 0;
#pragma unroll
    for (int l = 0; l < NL; ++l)
      m = amax2_finite(amax2_finite(amax2_finite(amax2_finite(m, w[l].x), w[l].y), w[l].z), w[l].w);
    m = warp_max(m);
  }
  return m;
}

// ---- append -------------------------------------------------------------------------------

struct AppendArgs {
  uint8_t* codes;
  float* scales;
  int64_t num_blocks;
  const uint16_t* x[2];            // k, v
  int64_t ts[2], hs[2];            // token and head strides
  const int32_t *token_start, *cached, *tables;
  int32_t* err;
  int T, B, max_blocks, layer, Hkv;
};

// Eight values of a row, from any 2-byte address or (VEC) a 16-byte one.
template <bool VEC>
__device__ __forceinline__ uint4 load8(const uint16_t* p) {
  if constexpr (VEC) {
    return *reinterpret_cast<const uint4*>(p);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = static_cast<uint32_t>(p[2 * i]) | static_cast<uint32_t>(p[2 * i + 1]) << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Work is laid out over slots, one touched block each.  Slot r < B is the first block that
// request r's tokens touch, so a decode step needs no search.  Behind them request r owns the slots
// B + token_start[r] / b + r on for its further blocks: at most token_start[r + 1] / b -
// token_start[r] / b + 1 of them, since tokens that start anywhere in a block touch at most
// n / b + 1 blocks after it.  A warp there finds its request by searching token_start, 32 probes at
// a time, and the host needs no per-request sizes: T / b + 2 B slots in all.  Grid (slot, group
// of kWarpsQ tiles); a warp takes one (K|V, head) tile of the slot's block.
// Registers are held to 10 CTAs an SM (5 with 32 x 128 tiles): the chains of dependent loads need the
// warps (8200 prompt tokens: 10.7 us so, 11.6 with the compiler's choice of 64 registers, although 6 to 12
// registers are spilled for it in the 32 x 64 and 16 x 128 forms).
template <int D, int BS, bool VEC>
__global__ void __launch_bounds__(kThreadsQ, BS * D == 4096 ? 5 : 10) append_kernel(const AppendArgs a) {
  constexpr int LPR = D / 8;                 // lanes per row (8 values each)
  constexpr int RPL = 32 / LPR;              // rows per load of the warp
  constexpr int NL = BS / RPL;               // loads per tile
  after_previous();
  next_may_start();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile = blockIdx.y * kWarpsQ + warp;

  int r = static_cast<int>(blockIdx.x);
  int s0, s1, j = 0;
  int64_t c;
  if (r < a.B) {
    s0 = a.token_start[r];
    s1 = a.token_start[r + 1];
    c = a.cached[r];
    // token_start as a whole: each request looks at its own step, the first at both ends
    if (blockIdx.y == 0 && threadIdx.x == 0 &&
        (s1 < s0 || (r == 0 && (s0 != 0 || a.token_start[a.B] > a.T))))
      record(a.err, ZP_ERR_BAD_TABLE);
  } else {
    // the last request whose first further slot is <= u
    const int64_t u = static_cast<int64_t>(blockIdx.x) - a.B;
    int lo = 0, hi = a.B, last;
    while (true) {
      const int step = (hi - lo + 31) / 32, i = lo + lane * step;
      int si = -1, ei = 0, ci = 0;
      if (i < hi) {
        si = a.token_start[i];
        ei = a.token_start[i + 1];
        ci = a.cached[i];
      }
      const uint32_t vote = __ballot_sync(0xffffffffu, si >= 0 && static_cast<int64_t>(si / BS) + i <= u);
      if (vote == 0) return;  // only when token_start[0] is not 0
      last = 31 - __clz(vote);
      lo += last * step;
      hi = min(hi, lo + step);
      if (step == 1) {
        s0 = __shfl_sync(0xffffffffu, si, last);
        s1 = __shfl_sync(0xffffffffu, ei, last);
        c = __shfl_sync(0xffffffffu, ci, last);
        break;
      }
    }
    r = lo;
    j = static_cast<int>(u - (s0 / BS + r)) + 1;
  }
  if (tile >= 2 * a.Hkv) return;
  const int64_t n = static_cast<int64_t>(s1) - s0;
  if (n <= 0) return;
  if (s0 < 0 || s1 > a.T || c < 0 || c + n > static_cast<int64_t>(a.max_blocks) * BS) {
    if (j == 0 && tile == 0 && lane == 0) record(a.err, ZP_ERR_BAD_TABLE);
    return;
  }
  const int64_t blk = c / BS + j;
  const int64_t p0 = max(c, blk * BS), p1 = min(c + n, (blk + 1) * BS);  // this block's new tokens
  if (p0 >= p1) return;
  const int64_t phys = a.tables[static_cast<int64_t>(r) * a.max_blocks + blk];
  const int kv = tile / a.Hkv, h = tile - kv * a.Hkv;
  const int first = static_cast<int>(p0 - blk * BS), end = static_cast<int>(p1 - blk * BS);  // rows [first, end)
  const int64_t ts = kv ? a.ts[1] : a.ts[0];
  const uint16_t* const x = (kv ? a.x[1] : a.x[0]) + (s0 + (p0 - c)) * ts + h * (kv ? a.hs[1] : a.hs[0]) + (lane % LPR) * 8;
  const int row = lane / LPR;
  uint4 w[NL];  // on their way while the block's id is
#pragma unroll
  for (int l = 0; l < NL; ++l) {
    const int rr = l * RPL + row;
    w[l] = make_uint4(0, 0, 0, 0);
    if (rr >= first && rr < end) w[l] = load8<VEC>(x + (rr - first) * ts);
  }
  if (phys < 0 || phys >= a.num_blocks) {
    if (tile == 0 && lane == 0) record(a.err, ZP_ERR_BAD_TABLE);
    return;
  }
  const int64_t t = ((static_cast<int64_t>(a.layer) * a.num_blocks + phys) * 2 + kv) * a.Hkv + h;
  uint8_t* const codes = a.codes + t * (BS * D) + lane * 8;  // + 256 per load
  const float old = first > 0 ? a.scales[t] : 0.0f;
  bool odd;
  const float s = fmaxf(old, scale_of(tile_amax(w, odd))), inv = inverse(s);
  if (first > 0 && s > old) {  // the rows already there, brought to the larger scale
    const float ratio = old * inv;
#pragma unroll
    for (int l = 0; l < NL; ++l) {
      if (l * RPL + row >= first) continue;
      uint2 o = *reinterpret_cast<const uint2*>(codes + l * 256);
      uint32_t v[2] = {o.x, o.y};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 y0 = dec2(v[e] & 0xFFFFu), y1 = dec2(v[e] >> 16);
        v[e] = enc2(y0.x * ratio, y0.y * ratio) | enc2(y1.x * ratio, y1.y * ratio) << 16;
      }
      *reinterpret_cast<uint2*>(codes + l * 256) = make_uint2(v[0], v[1]);
    }
  }
#pragma unroll
  for (int l = 0; l < NL; ++l) {
    const int rr = l * RPL + row;
    if (rr >= first && rr < end)
      *reinterpret_cast<uint2*>(codes + l * 256) = odd ? enc8<true>(w[l], inv) : enc8<false>(w[l], inv);
  }
  if (lane == 0 && (first == 0 || s > old)) a.scales[t] = s;
}

// ---- whole blocks -------------------------------------------------------------------------

struct BlockArgs {
  const uint8_t* src;
  uint8_t* dst;
  float* scales;                       // of the 8-bit pool
  const int32_t *src_ids, *dst_ids, *fill;
  int64_t src_blocks, dst_blocks, tiles;
  int32_t* err;
  int n, Hkv, layer_begin;
};

// The warp's tile: (layer, i, K|V, head) with the heads of a block next to one another, which is
// how the pool holds them.  False: nothing to do.
__device__ __forceinline__ bool take_tile(const BlockArgs& a, int64_t w, int bs, int64_t& src, int64_t& dst, int& fill) {
  if (w >= a.tiles) return false;
  const int per_block = 2 * a.Hkv;
  const int64_t bi = w / per_block;
  const int kvh = static_cast<int>(w - bi * per_block);
  const int64_t layer = a.layer_begin + bi / a.n;
  const int i = static_cast<int>(bi % a.n);
  const int64_t s = a.src_ids[i], d = a.dst_ids[i];
  fill = a.fill ? a.fill[i] : bs;
  if (s < 0 || s >= a.src_blocks || d < 0 || d >= a.dst_blocks || fill < 0 || fill > bs) {
    if ((threadIdx.x & 31) == 0) record(a.err, ZP_ERR_BAD_TABLE);
    return false;
  }
  src = (layer * a.src_blocks + s) * per_block + kvh;
  dst = (layer * a.dst_blocks + d) * per_block + kvh;
  return true;
}

template <int D, int BS>
__global__ void __launch_bounds__(kThreadsQ) pack_kernel(const BlockArgs a) {
  constexpr int NL = BS * D / 256;  // loads of 8 values a lane
  after_previous();
  next_may_start();
  const int lane = threadIdx.x & 31;
  int64_t src, dst;
  int fill;
  if (!take_tile(a, static_cast<int64_t>(blockIdx.x) * kWarpsQ + (threadIdx.x >> 5), BS, src, dst, fill)) return;
  const uint4* const x = reinterpret_cast<const uint4*>(a.src + src * (BS * D * 2)) + lane;
  uint2* const codes = reinterpret_cast<uint2*>(a.dst + dst * (BS * D)) + lane;
  const int nv = fill * D;  // values of the block's tokens come first
  uint4 w[NL];
#pragma unroll
  for (int l = 0; l < NL; ++l) w[l] = (l * 256 + lane * 8 < nv) ? x[l * 32] : make_uint4(0, 0, 0, 0);
  bool odd;
  const float s = scale_of(tile_amax(w, odd)), inv = inverse(s);
#pragma unroll
  for (int l = 0; l < NL; ++l)
    if (l * 256 + lane * 8 < nv) codes[l * 32] = odd ? enc8<true>(w[l], inv) : enc8<false>(w[l], inv);
  if (lane == 0) a.scales[dst] = s;
}

// WIDE: the bf16 pool stands on 32-byte boundaries, and a lane writes its 16 values at once.
template <int D, int BS, bool WIDE>
__global__ void __launch_bounds__(kThreadsQ) unpack_kernel(const BlockArgs a) {
  constexpr int NL = BS * D / 512;  // loads of 16 codes a lane
  after_previous();
  next_may_start();
  const int lane = threadIdx.x & 31;
  int64_t src, dst;
  int fill;
  if (!take_tile(a, static_cast<int64_t>(blockIdx.x) * kWarpsQ + (threadIdx.x >> 5), BS, src, dst, fill)) return;
  const uint4* const codes = reinterpret_cast<const uint4*>(a.src + src * (BS * D)) + lane;
  uint8_t* const y = a.dst + dst * (BS * D * 2) + lane * 32;
  uint4 w[NL];
#pragma unroll
  for (int l = 0; l < NL; ++l) w[l] = codes[l * 32];
  const float s = a.scales[src];
#pragma unroll
  for (int l = 0; l < NL; ++l) {
    const uint32_t c[4] = {w[l].x, w[l].y, w[l].z, w[l].w};
    uint32_t v[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 lo = dec2(c[e] & 0xFFFFu), hi = dec2(c[e] >> 16);
      v[2 * e] = pack_bf16x2(lo.x * s, lo.y * s);
      v[2 * e + 1] = pack_bf16x2(hi.x * s, hi.y * s);
    }
    if constexpr (WIDE) {
      asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(y + l * 1024), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                   "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                   : "memory");
    } else {
      *reinterpret_cast<uint4*>(y + l * 1024) = make_uint4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<uint4*>(y + l * 1024 + 16) = make_uint4(v[4], v[5], v[6], v[7]);
    }
  }
}

// Sizes that the 8-bit pool's operators share.
zp_status check_pool(const zp_kv8_pool* pool, const zp_params* p, const void* workspace, size_t bytes) {
  if (!pool || !p || !pool->codes || !pool->scales || pool->num_blocks <= 0) return ZP_ERR_INVALID_ARG;
  if (p->num_layers <= 0 || p->num_kv_heads <= 0) return ZP_ERR_INVALID_ARG;
  if (p->head_dim != 64 && p->head_dim != 128) return ZP_ERR_UNSUPPORTED;
  if (p->block_size != 16 && p->block_size != 32) return ZP_ERR_UNSUPPORTED;
  if (p->num_kv_heads > 65535) return ZP_ERR_UNSUPPORTED;
  if (!aligned(pool->codes, 16) || !aligned(pool->scales, 4)) return ZP_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || bytes < 256) return ZP_ERR_INVALID_ARG;
  return ZP_OK;
}

template <int D, int BS>
cudaError_t launch_append(const AppendArgs& a, bool vec, dim3 grid, cudaStream_t st) {
  return launch_in_order(vec ? append_kernel<D, BS, true> : append_kernel<D, BS, false>, grid, kThreadsQ, 0, st, 1, a);
}

template <int D, int BS>
cudaError_t launch_blocks(const BlockArgs& a, bool pack, unsigned grid, cudaStream_t st) {
  return launch_in_order(pack ? pack_kernel<D, BS> : aligned(a.dst, 32) ? unpack_kernel<D, BS, true> : unpack_kernel<D, BS, false>,
                         dim3(grid), kThreadsQ, 0, st, 1, a);
}

zp_status convert(const zp_kv_pool* pool, const zp_kv8_pool* kv8, bool pack, const int32_t* src_ids, const int32_t* fill,
                  const int32_t* dst_ids, int32_t n, int32_t layer_begin, int32_t layer_count, const zp_params* p,
                  void* workspace, size_t bytes, zp_stream stream) {
  const zp_status s = check_pool(kv8, p, workspace, bytes);
  if (s != ZP_OK) return s;
  if (!pool || !pool->base || pool->num_blocks <= 0 || !aligned(pool->base, 16) || n < 0) return ZP_ERR_INVALID_ARG;
  if (layer_count == 0) {
    if (layer_begin != 0) return ZP_ERR_INVALID_ARG;
    layer_count = p->num_layers;
  }
  if (layer_begin < 0 || layer_count < 0 || layer_begin > p->num_layers - layer_count) return ZP_ERR_INVALID_ARG;
  if (n == 0) return ZP_OK;
  if (!src_ids || !dst_ids) return ZP_ERR_INVALID_ARG;
  BlockArgs a{};
  a.src = static_cast<const uint8_t*>(pack ? pool->base : kv8->codes);
  a.dst = static_cast<uint8_t*>(pack ? kv8->codes : pool->base);
  a.scales = kv8->scales;
  a.src_ids = src_ids;
  a.dst_ids = dst_ids;
  a.fill = fill;
  a.src_blocks = pack ? pool->num_blocks : kv8->num_blocks;
  a.dst_blocks = pack ? kv8->num_blocks : pool->num_blocks;
  a.tiles = static_cast<int64_t>(layer_count) * n * 2 * p->num_kv_heads;
  a.err = static_cast<int32_t*>(workspace);
  a.n = n;
  a.Hkv = p->num_kv_heads;
  a.layer_begin = layer_begin;
  const int64_t ctas = (a.tiles + kWarpsQ - 1) / kWarpsQ;
  if (ctas >= (int64_t(1) << 31)) return ZP_ERR_UNSUPPORTED;
  const unsigned grid = static_cast<unsigned>(ctas);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool wide_heads = p->head_dim == 128, long_blocks = p->block_size == 32;
  const cudaError_t e = wide_heads ? (long_blocks ? launch_blocks<128, 32>(a, pack, grid, st) : launch_blocks<128, 16>(a, pack, grid, st))
                                   : (long_blocks ? launch_blocks<64, 32>(a, pack, grid, st) : launch_blocks<64, 16>(a, pack, grid, st));
  return e == cudaSuccess ? ZP_OK : ZP_ERR_CUDA;
}

}  // namespace
}  // namespace zp

using namespace zp;

extern "C" zp_status zp_kv8_append(const zp_kv8_pool* pool, int32_t layer, const zp_rows* k, const zp_rows* v, int32_t T,
                                   const int32_t* token_start, const int32_t* cached, int32_t B,
                                   const int32_t* block_tables, int32_t max_blocks, const zp_params* p, void* workspace,
                                   size_t workspace_bytes, zp_stream stream) {
  zp::NvtxRange nvtx_range("zp_kv8_append");
  const zp_status s = check_pool(pool, p, workspace, workspace_bytes);
  if (s != ZP_OK) return s;
  if (layer < 0 || layer >= p->num_layers || T < 0 || B < 0 || max_blocks < 1) return ZP_ERR_INVALID_ARG;
  if (T == 0 || B == 0) return T == 0 ? ZP_OK : ZP_ERR_INVALID_ARG;
  if (!k || !v || !k->data || !v->data || !aligned(k->data, 2) || !aligned(v->data, 2) || !token_start || !cached ||
      !block_tables)
    return ZP_ERR_INVALID_ARG;
  AppendArgs a{};
  a.codes = static_cast<uint8_t*>(pool->codes);
  a.scales = pool->scales;
  a.num_blocks = pool->num_blocks;
  a.x[0] = static_cast<const uint16_t*>(k->data);
  a.x[1] = static_cast<const uint16_t*>(v->data);
  a.ts[0] = k->token_stride, a.ts[1] = v->token_stride;
  a.hs[0] = k->head_stride, a.hs[1] = v->head_stride;
  a.token_start = token_start;
  a.cached = cached;
  a.tables = block_tables;
  a.err = static_cast<int32_t*>(workspace);
  a.T = T;
  a.B = B;
  a.max_blocks = max_blocks;
  a.layer = layer;
  a.Hkv = p->num_kv_heads;
  const int64_t slots = T / p->block_size + 2 * static_cast<int64_t>(B);
  const int groups = (2 * p->num_kv_heads + kWarpsQ - 1) / kWarpsQ;
  if (slots >= (int64_t(1) << 31) || groups > 65535) return ZP_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(slots), static_cast<unsigned>(groups));
  const bool vec = wide(k) && wide(v);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool wide_heads = p->head_dim == 128, long_blocks = p->block_size == 32;
  const cudaError_t e = wide_heads ? (long_blocks ? launch_append<128, 32>(a, vec, grid, st) : launch_append<128, 16>(a, vec, grid, st))
                                   : (long_blocks ? launch_append<64, 32>(a, vec, grid, st) : launch_append<64, 16>(a, vec, grid, st));
  return e == cudaSuccess ? ZP_OK : ZP_ERR_CUDA;
}

extern "C" zp_status zp_kv8_pack_blocks(const zp_kv_pool* pool, const int32_t* src_ids, const int32_t* fill,
                                        const zp_kv8_pool* kv8, const int32_t* dst_ids, int32_t n, int32_t layer_begin,
                                        int32_t layer_count, const zp_params* p, void* workspace, size_t workspace_bytes,
                                        zp_stream stream) {
  zp::NvtxRange nvtx_range("zp_kv8_pack_blocks");
  return convert(pool, kv8, true, src_ids, fill, dst_ids, n, layer_begin, layer_count, p, workspace, workspace_bytes, stream);
}

extern "C" zp_status zp_kv8_unpack_blocks(const zp_kv8_pool* kv8, const int32_t* src_ids, const zp_kv_pool* pool,
                                          const int32_t* dst_ids, int32_t n, int32_t layer_begin, int32_t layer_count,
                                          const zp_params* p, void* workspace, size_t workspace_bytes, zp_stream stream) {
  zp::NvtxRange nvtx_range("zp_kv8_unpack_blocks");
  return convert(pool, kv8, false, src_ids, nullptr, dst_ids, n, layer_begin, layer_count, p, workspace, workspace_bytes,
                 stream);
}
