// Joins the partials of mj_latent_attention's split requests: for request b
// and row r, over its partials s (normalised output O~, max logit m in the
// log2 domain, sum l = sum 2^(t - m)):
//   M = max_s m_s,  w_s = 2^(m_s - M) l_s,  out = s0 sum w_s O~_s / sum w_s.
// A partial without a key has m = -inf and is selected off (its O~ and l were
// never written).
//
// Bound by latency: a few megabytes of partials at most. A task is 128 channels
// of one row (a float4 a lane). Few rows (a long request split over the whole
// GPU): 16 warps share a task's partials and meet in shared memory, so that
// their loads are in flight together; many rows: a warp each.
#include <atomic>

#include "mj_device.cuh"
#include "mj_internal.h"
#include "tc_ptx.cuh"

namespace mj {

namespace {

constexpr int kWarps = 16;
constexpr int kBlocks = MJ_LATENT_DIM / 128;

template <int KW>  // warps per task
__global__ void __launch_bounds__(32 * kWarps) latent_merge_kernel(LatentParams p) {
  __shared__ float4 part[KW > 1 ? KW : 1][32];
  tc::grid_launch_dependents();
  tc::grid_dependency_wait();
  const int lane = threadIdx.x & 31, wi = (threadIdx.x >> 5) % KW;
  const int64_t task = int64_t(blockIdx.x) * (kWarps / KW) + (threadIdx.x >> 5) / KW;
  const int64_t unit = task / kBlocks;
  const int ch = int(task % kBlocks) * 128 + 4 * lane;
  if (unit >= int64_t(p.num_seqs) * p.n_q) return;  // (KW > 1: the whole CTA)
  const int b = int(unit / p.n_q), row = int(unit % p.n_q);
  const int first = p.splits[2 * b], n = min(p.splits[2 * b + 1], 2 * p.slots - first);
  // an unsplit request was written by the attention kernel; a padding request is left alone
  if (n <= 0 || first < 0 || p.seq_lens[b] <= 0) return;
  const float* mp = p.m_part + int64_t(first) * p.n_q + row;
  const float* lp = p.l_part + int64_t(first) * p.n_q + row;
  const float* op = p.o_part + (int64_t(first) * p.n_q + row) * MJ_LATENT_DIM + ch;

  float M = -INFINITY;
  for (int s = lane; s < n; s += 32) M = fmaxf(M, mp[int64_t(s) * p.n_q]);
  M = warp_max(M);
  auto weight = [&](int s) {
    const float m = mp[int64_t(s) * p.n_q];
    return m == -INFINITY ? 0.f : fast_exp2(m - M) * lp[int64_t(s) * p.n_q];
  };
  float wsum = 0.f;
  for (int s = lane; s < n; s += 32) wsum += weight(s);
  wsum = warp_sum(wsum);

  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int s = wi; s < n; s += KW) {
    const float w = weight(s);
    const float4 o = *reinterpret_cast<const float4*>(op + int64_t(s) * p.n_q * MJ_LATENT_DIM);
    if (w != 0.f) {
      acc.x = fmaf(w, o.x, acc.x);
      acc.y = fmaf(w, o.y, acc.y);
      acc.z = fmaf(w, o.z, acc.z);
      acc.w = fmaf(w, o.w, acc.w);
    }
  }
  if constexpr (KW > 1) {
    part[wi][lane] = acc;
    __syncthreads();
    if (wi != 0) return;
#pragma unroll
    for (int k = 1; k < KW; ++k) {
      const float4 o = part[k][lane];
      acc.x += o.x;
      acc.y += o.y;
      acc.z += o.z;
      acc.w += o.w;
    }
  }
  const float f = M == -INFINITY ? 0.f : p.descale[0] / wsum;
  const int tq = row / p.h, h = row - tq * p.h;
  uint2 o;
  o.x = uint32_t(float_to_out_bits(acc.x * f, p.out_f16)) | (uint32_t(float_to_out_bits(acc.y * f, p.out_f16)) << 16);
  o.y = uint32_t(float_to_out_bits(acc.z * f, p.out_f16)) | (uint32_t(float_to_out_bits(acc.w * f, p.out_f16)) << 16);
  *reinterpret_cast<uint2*>(p.out + (int64_t(b) * p.q_len + tq) * p.out_ts + int64_t(h) * p.out_hs + ch) = o;
  if (p.lse && lane == 0 && ch == 0)
    p.lse[int64_t(b) * p.n_q + row] = M == -INFINITY ? -INFINITY : (M + fast_log2(wsum)) * kLn2;
}

template <int KW>
cudaError_t launch(const LatentParams& p, int64_t tasks, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  const int64_t ctas = (tasks + kWarps / KW - 1) / (kWarps / KW);
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, latent_merge_kernel<KW>, p);
}

}  // namespace

cudaError_t launch_latent_merge(const LatentParams& p, cudaStream_t stream) {
  const int64_t tasks = int64_t(p.num_seqs) * p.n_q * kBlocks;
  // 16 warps a task while that still is at most four CTAs a slot
  return tasks <= 4 * int64_t(p.slots) * p.n_row_tiles ? launch<kWarps>(p, tasks, stream) : launch<1>(p, tasks, stream);
}

}  // namespace mj
