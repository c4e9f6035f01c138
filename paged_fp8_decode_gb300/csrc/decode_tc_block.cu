// tcgen05 decode kernel instances for the block-scaled cache (e4m3 codes): up to 8 query
// rows (more go to the prompt's kernel, mj_api_block.cpp). 64 x 4096 tokens, 8 heads of 128, pages of 16: 4 rows
// 89 us (6.0 TB/s, 0.90 of a copy's rate), 8 rows 107 (103 in pages of 32); 1 x 131072 tokens 48 (5.6 TB/s, start and join).
#include "decode_tc_kernel.cuh"

namespace mj {

cudaError_t launch_tc_block(const CUtensorMap& mk, const CUtensorMap& mv, const DecodeParams& p, cudaStream_t stream) {
  if (p.d == 128)
    return p.n_q <= 4 ? launch_tc<16, 16, 4, MJ_KV_E4M3, kQBlock, 128>(mk, mv, p, stream)
                      : launch_tc<16, 32, 8, MJ_KV_E4M3, kQBlock, 128>(mk, mv, p, stream);
  return p.n_q <= 4 ? launch_tc<16, 16, 4, MJ_KV_E4M3, kQBlock, 256>(mk, mv, p, stream)
                    : launch_tc<16, 32, 8, MJ_KV_E4M3, kQBlock, 256>(mk, mv, p, stream);
}

}  // namespace mj
