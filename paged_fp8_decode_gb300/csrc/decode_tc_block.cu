// tcgen05 decode kernel instances for the block-scaled cache (e4m3 codes, head size
// 128 and 256).
#include "decode_tc_kernel.cuh"

namespace mj {

cudaError_t launch_tc_block(const CUtensorMap& mk, const CUtensorMap& mv, const DecodeParams& p, cudaStream_t stream) {
  return p.d == 256 ? launch_rows<MJ_KV_E4M3, kQBlock, 256>(mk, mv, p, stream)
                    : launch_rows<MJ_KV_E4M3, kQBlock, 128>(mk, mv, p, stream);
}

}  // namespace mj
