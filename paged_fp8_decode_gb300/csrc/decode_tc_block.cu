// tcgen05 decode kernel instances for the block-scaled cache (e4m3 codes): up to 8 query
// rows at head size 128, 16 at 256 (more go to the prompt's kernel, mj_api_block.cpp).
#include "decode_tc_kernel.cuh"

namespace mj {

cudaError_t launch_tc_block(const CUtensorMap& mk, const CUtensorMap& mv, const DecodeParams& p, cudaStream_t stream) {
  if (p.d == 128)
    return p.n_q <= 4 ? launch_tc<16, 16, 4, MJ_KV_E4M3, kQBlock, 128>(mk, mv, p, stream)
                      : launch_tc<16, 32, 8, MJ_KV_E4M3, kQBlock, 128>(mk, mv, p, stream);
  if (p.n_q <= 4) return launch_tc<16, 16, 4, MJ_KV_E4M3, kQBlock, 256>(mk, mv, p, stream);
  if (p.n_q <= 8) return launch_tc<16, 32, 8, MJ_KV_E4M3, kQBlock, 256>(mk, mv, p, stream);
  return launch_tc<32, 64, 16, MJ_KV_E4M3, kQBlock, 256>(mk, mv, p, stream);
}

}  // namespace mj
