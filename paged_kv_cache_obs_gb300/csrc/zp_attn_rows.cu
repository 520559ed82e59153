// zp_attn_rows.cu — attention of packed prompts over their own keys and values (zp_attn_tile.cuh), which are rows
// of memory and no cache; sm_103a.
#include "zp_attn_tile.cuh"

namespace zp {

zp_status tile_rows_launch(const AttnArgs& args, const zp_params* p, const TilePlan& plan, void* workspace, cudaStream_t st) {
  AttnArgs a = args;
  CUtensorMap tk{}, tv{};
  // {d, heads, T}; box = b tokens of one head, 64 columns; rows behind the last one come as zeros
  const auto encode = [&](CUtensorMap* map, const uint16_t* x, int64_t ts, int64_t hs) {
    if (a.Hkv == 1) hs = p->head_dim;  // a stride that nothing takes
    if (a.T == 1) ts = a.Hkv * hs;
    return aligned(x, 16) && ts > 0 && hs > 0 && ts % 8 == 0 && hs % 8 == 0 &&
           encode_tmap_3d_bf16(map, x, p->head_dim, a.Hkv, a.T, static_cast<uint64_t>(hs) * 2, static_cast<uint64_t>(ts) * 2, 64, 1, a.b);
  };
  a.kv_tma = encode(&tk, a.k, a.k_ts, a.k_hs) && encode(&tv, a.v, a.v_ts, a.v_hs);
  return launch_tiles<Source::kRows>(a, p, plan, workspace, st, tk, tv);
}

}  // namespace zp
