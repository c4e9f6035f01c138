// Inline-PTX wrappers of the latent-attention kernel beside those of tc_ptx.cuh:
// tcgen05.mma, its commit and 3-D tensor loads issued by a converged warp, single
// TMEM columns, L2 prefetches, the float maximum of a warp.
#pragma once

#include "tc_ptx.cuh"

namespace mj {
namespace tc {

// D[tmem] (+)= A[smem desc] * B[smem desc] of kind f8f6f4, and the commit below,
// called by a whole converged warp: one elected lane issues (the same one each
// time). The warp's loop stays uniform, so the descriptors live in uniform
// registers and nothing is moved there per MMA.
__device__ __forceinline__ void umma_f8f6f4_warp(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                 uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void umma_commit_warp(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}

// One 32-bit TMEM column of this thread's lane.
__device__ __forceinline__ float tmem_ld1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
  return __uint_as_float(r);
}
__device__ __forceinline__ void tmem_st1(uint32_t taddr, float v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(__float_as_uint(v)) : "memory");
}

// Called by a whole converged warp: one elected lane issues.
__device__ __forceinline__ void tma_load_3d_warp(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                                 uint64_t policy) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy)
      : "memory");
}

// A line into L2.
__device__ __forceinline__ void prefetch_l2(const void* at) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
}

// `bytes` (a multiple of 16) from a 16-byte aligned address into L2, asynchronously.
__device__ __forceinline__ void prefetch_bulk_l2(const void* at, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at), "r"(bytes) : "memory");
}

// max over the warp, in every lane (NaN lanes do not count)
__device__ __forceinline__ float redux_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

constexpr uint32_t kSwizzle64B = 4;      // shared-memory descriptor, bits 61-63
constexpr uint32_t kFormatBE5m2 = 1u << 10;  // instruction descriptor: B holds e5m2 codes

}  // namespace tc
}  // namespace mj
