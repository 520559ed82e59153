// zp_step.cu — the blocks, slots and positions of a step, made on the device from its requests'
// lengths; sm_103a.
//
// With c_r tokens in request r's cache, n_r new ones and b tokens a block:
//   token_start  = exclusive sums of n_r;  seq_lens[r] = c_r + n_r
//   h_r          = the blocks that the table holds: ceil(c_r / b), or more where tokens were taken back and the caller counts
//   taken_r      = exclusive sums of max(0, ceil((c_r + n_r) / b) - h_r), the blocks that the step takes
//   table[r][j]  = free[taken_r + j - h_r] for those blocks j
//   slots[t]     = table[r][p / b] * b + p % b,  p = c_r + t - token_start[r];  positions[t] = first_r + t - token_start[r]
//
// Few bytes and long chains: lengths, then the table's entry of a part-full block or the free list's, then
// the stores.  So one launch of one cluster does it all: every CTA sums over all requests by itself (1024 at a time, a warp
// scan in each warp and one more over the warps' totals), with the part-full blocks' ids and the first free ids on
// their way meanwhile, and takes its share of the tokens and of the new blocks.  The cluster's barrier stands
// between the last read of lengths and free_at and the writes, since both may be updated in place.  A row of the
// step finds its request by halving the chunk's sums in shared memory.
#include <algorithm>
#include <climits>

#include "zp_internal.h"
#include "zp_launch.h"
#include "zp_ptx.cuh"

namespace zp {
namespace {

constexpr int kThreads = 1024;   // and requests of a chunk
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kFresh = 4096;     // free ids in shared memory: the rows of a large step wait for none (49000 rows 7.5 -> 7.2 us)

struct StepArgs {
  const int32_t *cached, *new_tokens, *first, *free_ids;
  int32_t *have;  // blocks that each request's table holds, or NULL
  int32_t *free_at, *tables, *token_start, *seq_lens, *positions, *slots, *err;
  int64_t num_blocks;
  int B, T, num_free, max_blocks, bshift;
};

__device__ __forceinline__ int blocks_of(const StepArgs& a, int tokens) { return (tokens + (1 << a.bshift) - 1) >> a.bshift; }

// The tokens before and of a step of request r, the blocks that its table holds and those that the step takes; a
// request that is out of range takes part with none.
struct Lengths {
  int cached, add, before, more;
  bool bad;
};
template <bool HELD>
__device__ __forceinline__ Lengths lengths_of(const StepArgs& a, int r) {
  Lengths x{0, 0, 0, 0, false};
  if (r >= a.B) return x;
  const int most = a.max_blocks << a.bshift;  // at most 2^30
  x.cached = a.cached[r];
  x.add = a.new_tokens[r];
  const bool bad_cache = x.cached < 0 || x.cached > most;
  x.bad = bad_cache || x.add < 0 || x.add > most - x.cached;
  if (bad_cache) x.cached = 0;
  x.before = blocks_of(a, x.cached);
  if (HELD) {
    const int have = a.have[r];
    x.bad = x.bad || have < x.before || have > a.max_blocks;
    if (!x.bad) x.before = have;
  }
  if (x.bad) x.add = 0;
  x.more = max(0, blocks_of(a, x.cached + x.add) - x.before);
  return x;
}

// The last of n + 1 increasing sums that is at most x, below n.
__device__ __forceinline__ int place_of(const int* sums, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ uint64_t shfl_up64(uint64_t x, int by) { return __shfl_up_sync(0xffffffffu, static_cast<unsigned long long>(x), by); }

// HELD: how many blocks tables hold is given.  Compiled apart: in one kernel the slots of 256 requests took 3.9 us in place of 3.7.
template <bool CLUSTER, bool HELD>
__global__ void __launch_bounds__(kThreads) step_kernel(const __grid_constant__ StepArgs a) {
  __shared__ int start[kThreads + 1], taken[kThreads + 1], cached[kThreads], first[kThreads], before[HELD ? kThreads : 1], held[kThreads], fresh[kFresh];
  __shared__ uint64_t sum_t[kWarps], sum_b[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = CLUSTER ? static_cast<int>(cluster_ctarank()) : 0, ctas = CLUSTER ? static_cast<int>(cluster_nctarank()) : 1;
  const int all = ctas * kThreads, me = rank * kThreads + tid;
  after_previous();
  next_may_start();
  const auto barrier = [&] {
    if (CLUSTER) cluster_sync();
    else __syncthreads();
  };

  // what is free, and its first ids
  int at = a.free_at ? *a.free_at : 0;
  const bool bad_at = at < 0 || at > a.num_free;
  if (bad_at) at = a.num_free;
#pragma unroll
  for (int i = tid; i < kFresh; i += kThreads)
    if (i < a.num_free - at) fresh[i] = a.free_ids[at + i];

  uint64_t tokens_before = 0, blocks_before = 0, tokens_all = 0, blocks_all = 0;
  bool bad = false;
  // totals of a batch of several chunks, before any of it is written
  if (a.B > kThreads) {
    for (int r = tid; r < a.B; r += kThreads) {
      const Lengths x = lengths_of<HELD>(a, r);
      tokens_all += x.add;
      blocks_all += x.more;
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
      tokens_all += __shfl_xor_sync(0xffffffffu, static_cast<unsigned long long>(tokens_all), s);
      blocks_all += __shfl_xor_sync(0xffffffffu, static_cast<unsigned long long>(blocks_all), s);
    }
    if (lane == 0) sum_t[warp] = tokens_all, sum_b[warp] = blocks_all;
    __syncthreads();
    tokens_all = blocks_all = 0;
    for (int w = 0; w < kWarps; ++w) tokens_all += sum_t[w], blocks_all += sum_b[w];
    __syncthreads();
  }

  bool empty = false;  // the step does not fit: it is one without tokens
  for (int base = 0; base < a.B || base == 0; base += kThreads) {
    const int r = base + tid, n = min(kThreads, a.B - base);
    const Lengths x = lengths_of<HELD>(a, r);
    bad |= x.bad;
    // the id of the block that the first new token goes to, if the table holds it, is on its way during the sums
    int id = 0;
    if (x.add > 0 && (x.cached >> a.bshift) < x.before) id = a.tables[static_cast<int64_t>(r) * a.max_blocks + (x.cached >> a.bshift)];
    const int pos = r < a.B && a.first ? a.first[r] : x.cached;
    uint64_t st = x.add, sb = x.more;
#pragma unroll
    for (int s = 1; s < 32; s *= 2) {
      const uint64_t yt = shfl_up64(st, s), yb = shfl_up64(sb, s);
      if (lane >= s) st += yt, sb += yb;
    }
    if (lane == 31) sum_t[warp] = st, sum_b[warp] = sb;
    __syncthreads();
    uint64_t wt = sum_t[lane], wb = sum_b[lane];  // one warp's totals a lane, summed in every warp
    static_assert(kWarps == 32, "a lane for each warp's total");
    const uint64_t own_t = wt, own_b = wb;
#pragma unroll
    for (int s = 1; s < 32; s *= 2) {
      const uint64_t yt = shfl_up64(wt, s), yb = shfl_up64(wb, s);
      if (lane >= s) wt += yt, wb += yb;
    }
    const uint64_t chunk_t = __shfl_sync(0xffffffffu, static_cast<unsigned long long>(wt), 31);
    const uint64_t chunk_b = __shfl_sync(0xffffffffu, static_cast<unsigned long long>(wb), 31);
    const uint64_t off_t = __shfl_sync(0xffffffffu, static_cast<unsigned long long>(wt - own_t), warp);
    const uint64_t off_b = __shfl_sync(0xffffffffu, static_cast<unsigned long long>(wb - own_b), warp);
    if (a.B <= kThreads) tokens_all = chunk_t, blocks_all = chunk_b;
    const bool no_rows = tokens_all > static_cast<uint64_t>(a.T), no_blocks = blocks_all > static_cast<uint64_t>(a.num_free - at);
    empty = no_rows || no_blocks || bad_at;
    if (empty && rank == 0 && tid == 0 && base == 0) atomicCAS(a.err, 0, no_rows || bad_at ? ZP_ERR_BAD_TABLE : ZP_ERR_NO_BLOCKS);
    // sums that fit 32 bits where the step fits
    const int t0 = static_cast<int>(tokens_before + off_t + st) - x.add, b0 = static_cast<int>(blocks_before + off_b + sb) - x.more;
    start[tid] = t0;
    taken[tid] = b0;
    cached[tid] = x.cached;
    first[tid] = pos;
    if (HELD) before[tid] = x.before;
    held[tid] = id;
    if (tid == n - 1 || n <= 0) start[max(n, 0)] = t0 + x.add, taken[max(n, 0)] = b0 + x.more;
    barrier();  // every CTA has read what is updated in place
    if (rank == 0 && r < a.B) {
      a.token_start[r] = empty ? 0 : t0;
      a.seq_lens[r] = empty ? x.cached : x.cached + x.add;
      if (HELD && !empty && x.more > 0) a.have[r] = x.before + x.more;
    }
    if (!empty && n > 0) {
      // ids of the step's blocks
      const auto free_id = [&](int j) { return j < kFresh ? fresh[j] : a.free_ids[at + j]; };
      for (int j = taken[0] + me; j < taken[n]; j += all) {
        const int i = place_of(taken, n, j);
        a.tables[static_cast<int64_t>(base + i) * a.max_blocks + (HELD ? before[i] : blocks_of(a, cached[i])) + j - taken[i]] = free_id(j);
      }
      // unsigned: what comes behind the last row may pass 2^31
#pragma unroll 2
      for (uint32_t u = static_cast<uint32_t>(start[0]) + static_cast<uint32_t>(me); u < static_cast<uint32_t>(start[n]); u += static_cast<uint32_t>(all)) {
        const int t = static_cast<int>(u), i = place_of(start, n, t), k = t - start[i], p = cached[i] + k;
        const int at_block = p >> a.bshift, j = at_block - (HELD ? before[i] : blocks_of(a, cached[i]));
        int blk;
        if (j >= 0) blk = free_id(taken[i] + j);
        else if (!HELD || at_block == cached[i] >> a.bshift) blk = held[i];
        else blk = a.tables[static_cast<int64_t>(base + i) * a.max_blocks + at_block];  // begun by tokens that were taken back
        const bool out = blk < 0 || blk >= a.num_blocks;
        bad |= out;
        a.slots[t] = out ? -1 : (blk << a.bshift) + (p & ((1 << a.bshift) - 1));
        if (a.positions) a.positions[t] = static_cast<int>(static_cast<uint32_t>(first[i]) + static_cast<uint32_t>(k));
      }
    }
    tokens_before += chunk_t;
    blocks_before += chunk_b;
    if (base + kThreads < a.B) __syncthreads();  // before the next chunk's sums take the place
  }
  // rows behind the last request's
  const int rows = empty ? 0 : static_cast<int>(tokens_all);
  for (int64_t t = static_cast<int64_t>(rows) + me; t < a.T; t += all) {
    a.slots[t] = -1;
    if (a.positions) a.positions[t] = 0;
  }
  if (rank == 0 && tid == 0) {
    a.token_start[a.B] = rows;
    if (a.free_at && !empty) *a.free_at = at + static_cast<int>(blocks_all);
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) atomicCAS(a.err, 0, ZP_ERR_BAD_TABLE);
}

}  // namespace
}  // namespace zp

using namespace zp;

extern "C" zp_status zp_step_slots(const int32_t* cached, const int32_t* new_tokens, const int32_t* first_pos, int32_t B,
                                   const int32_t* free_ids, int32_t num_free, int32_t* free_at, int64_t num_blocks,
                                   int32_t* block_tables, int32_t max_blocks, int32_t* token_start, int32_t* seq_lens,
                                   int32_t* positions, int32_t* slots, int32_t T, const zp_params* p, void* workspace,
                                   size_t workspace_bytes, zp_stream stream) {
  return zp_step_slots_held(cached, new_tokens, first_pos, nullptr, B, free_ids, num_free, free_at, num_blocks, block_tables, max_blocks,
                            token_start, seq_lens, positions, slots, T, p, workspace, workspace_bytes, stream);
}

extern "C" zp_status zp_step_slots_held(const int32_t* cached, const int32_t* new_tokens, const int32_t* first_pos, int32_t* held_blocks,
                                        int32_t B, const int32_t* free_ids, int32_t num_free, int32_t* free_at, int64_t num_blocks,
                                        int32_t* block_tables, int32_t max_blocks, int32_t* token_start, int32_t* seq_lens,
                                        int32_t* positions, int32_t* slots, int32_t T, const zp_params* p, void* workspace,
                                        size_t workspace_bytes, zp_stream stream) {
  zp::NvtxRange nvtx_range("zp_step_slots");
  if (!p || B < 0 || T < 0 || num_free < 0 || num_blocks <= 0 || max_blocks < 1) return ZP_ERR_INVALID_ARG;
  if (p->block_size != 16 && p->block_size != 32) return ZP_ERR_UNSUPPORTED;
  if (B > 65535 || num_blocks > INT_MAX / p->block_size || static_cast<int64_t>(max_blocks) * p->block_size > (1 << 30))
    return ZP_ERR_UNSUPPORTED;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < 256) return ZP_ERR_INVALID_ARG;
  if (!token_start || (T > 0 && !slots) || (num_free > 0 && !free_ids)) return ZP_ERR_INVALID_ARG;
  if (B > 0 && (!cached || !new_tokens || !block_tables || !seq_lens)) return ZP_ERR_INVALID_ARG;
  StepArgs a{};
  a.cached = cached;
  a.new_tokens = new_tokens;
  a.first = first_pos;
  a.have = held_blocks;
  a.free_ids = free_ids;
  a.free_at = free_at;
  a.tables = block_tables;
  a.token_start = token_start;
  a.seq_lens = seq_lens;
  a.positions = positions;
  a.slots = slots;
  a.err = static_cast<int32_t*>(workspace);
  a.num_blocks = num_blocks;
  a.B = B;
  a.T = T;
  a.num_free = num_free;
  a.max_blocks = max_blocks;
  a.bshift = p->block_size == 16 ? 4 : 5;
  // a CTA for each 2048 rows, up to a portable cluster
  const int ctas = static_cast<int>(std::min<int64_t>(kMaxCluster, std::max<int64_t>(1, (static_cast<int64_t>(T) + 2047) / 2048)));
  int cluster = 1;
  while (cluster < ctas) cluster *= 2;
  auto* const kernel = cluster > 1 ? (a.have ? step_kernel<true, true> : step_kernel<true, false>)
                                   : (a.have ? step_kernel<false, true> : step_kernel<false, false>);
  return launch_in_order(kernel, dim3(cluster), kThreads, 0, reinterpret_cast<cudaStream_t>(stream), cluster, a) == cudaSuccess
             ? ZP_OK
             : ZP_ERR_CUDA;
}
