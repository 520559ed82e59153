// zp_attn_tile.cu — attention of many query rows over the paged bf16 pool (zp_attn_tile.cuh), and how calls of
// the tiled kernel are cut; sm_103a.
#include "zp_attn_tile.cuh"

namespace zp {

TilePlan tile_plan(const zp_params* p, int T, int B, int max_q, int max_blocks, int window, int sinks, size_t room, bool rounds) {
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
  const int64_t most_splits = std::max<int64_t>(1, std::min(tiles / 4, fit));
  plan.splits = 1;
  if (!rounds) {
    plan.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(plan.ctas / std::max<int64_t>(items, 1), most_splits)));
  } else {
    // As many as make the longest CTA's share shortest, in tiles: a part costs about 3 beside its own, and where there are
    // several 2 more for its sums.  64 items of up to 783 tiles take 547 us with 7 splits (3 parts a CTA) and 753 with 2 (one each).
    // Where items fill the SMs by themselves, the fewest that come within 5 % of it: lengths are at most the table's width, and
    // every further part's sums are written and read for the last wave's rounding alone (4 x 2048 tokens over up to 8192, 1024 items:
    // 529 us unsplit; with the 4 parts that a table for 65536 or more tokens gave, 848 us and a workspace of 554 MB).  Where lengths are the
    // table's width it can cost a little: 200 items of up to 64 tiles 222 us in 2 parts, 214 in 3.
    const int64_t most_parts = std::min<int64_t>(most_splits, 32);
    const auto cost = [&](int64_t n) {
      const int64_t parts = (std::max<int64_t>(items, 1) * n + plan.ctas - 1) / plan.ctas;  // of a CTA
      return parts * ((tiles + n - 1) / n + (n > 1 ? 5 : 3));
    };
    int64_t best = INT64_MAX;
    for (int64_t n = 1; n <= most_parts; ++n)
      if (cost(n) < best) best = cost(n), plan.splits = static_cast<int>(n);
    if (items >= plan.ctas)
      for (plan.splits = 1; 20 * cost(plan.splits) > 21 * best;) ++plan.splits;
  }
  plan.nx = static_cast<int>(std::min<int64_t>(nx, INT_MAX));
  plan.items = nx * heads * plan.splits;
  plan.bytes = kHeader;
  if (plan.splits > 1 && T > 0) plan.bytes += (plan.splits * part + 255) / 256 * 256;
  return plan;
}

zp_status tile_launch(const AttnArgs& a, const zp_params* p, const TilePlan& plan, void* workspace, cudaStream_t st) {
  const uint64_t d = p->head_dim, rows = static_cast<uint64_t>(2) * a.Hkv * a.b;
  CUtensorMap tm;
  // the pool as {d, 2*Hkv*b rows per (layer, block), layers*num_blocks}; box = one block's b rows
  // of one (K or V, head), 64 columns
  if (!encode_tmap_3d_bf16(&tm, a.pool, d, rows, static_cast<uint64_t>(a.layers) * a.num_blocks, d * 2, rows * d * 2, 64, a.b, 1)) return ZP_ERR_CUDA;
  return launch_tiles<Source::kPaged>(a, p, plan, workspace, st, tm, tm);
}

}  // namespace zp
