// zp_attn_tile8.cu — attention of many query rows over the paged 8-bit pool (zp_attn_tile.cuh); sm_103a.
#include "zp_attn_tile.cuh"

namespace zp {

zp_status tile8_launch(const AttnArgs& a, const zp_params* p, const TilePlan& plan, void* workspace, cudaStream_t st) {
  const uint64_t d = p->head_dim, rows = static_cast<uint64_t>(2) * a.Hkv * a.b;
  CUtensorMap tm;
  // the codes as {d, 2*Hkv*b rows per (layer, block), layers*num_blocks}; box = one block's b rows of one (K or V, head)
  if (!encode_tmap_3d_u8(&tm, a.pool, d, rows, static_cast<uint64_t>(a.layers) * a.num_blocks, d, rows * d, d, a.b, 1, static_cast<int>(d)))
    return ZP_ERR_CUDA;
  return launch_tiles<Source::kPaged8>(a, p, plan, workspace, st, tm, tm);
}

}  // namespace zp
