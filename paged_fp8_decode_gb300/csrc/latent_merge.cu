// Joins the partials of mj_latent_attention's split requests: for request b
// and row r, over its partials s (unnormalised output O~, reference max m in
// the log2 domain, sum l, both scaled by 2^m):
//   M = max_s m_s,  out = s0 sum_s 2^(m_s - M) O~_s / sum_s 2^(m_s - M) l_s.
// A partial without a key has m = -inf and is selected off (its O~ and l may
// never have been written).
//
// Bound by latency and L2: tens of megabytes of partials at most, just
// written. A task is four rows of 32 channels, one 16-byte load a lane and
// partial. Many tasks: a warp each. Few (a long request split over the whole
// GPU): the 16 warps of a CTA share a task's partials and meet in shared
// memory, so that all their loads are in flight together.
#include "mj_device.cuh"
#include "mj_internal.h"
#include "tc_ptx.cuh"

namespace mj {

namespace {

constexpr int kBlocks = MJ_LATENT_DIM / 128;

__device__ __forceinline__ float4 max4(float4 a, float4 b) {
  return make_float4(fmaxf(a.x, b.x), fmaxf(a.y, b.y), fmaxf(a.z, b.z), fmaxf(a.w, b.w));
}
__device__ __forceinline__ float weight(float m, float M) { return m == -INFINITY ? 0.f : fast_exp2(m - M); }
// a + w b, w = 0 selecting b off (it may be anything then)
__device__ __forceinline__ float add_w(float a, float w, float b) { return w != 0.f ? fmaf(w, b, a) : a; }
__device__ __forceinline__ void add_w4(float4& a, float4 w, float4 b) {
  a.x = add_w(a.x, w.x, b.x);
  a.y = add_w(a.y, w.y, b.y);
  a.z = add_w(a.z, w.z, b.z);
  a.w = add_w(a.w, w.w, b.w);
}

constexpr int kWarps = 16;

template <int G>  // warps a task
__global__ void __launch_bounds__(32 * kWarps) latent_merge_kernel(LatentParams p) {
  constexpr int U = 4;  // partials in flight a warp
  __shared__ float4 acc_sh[G > 1 ? G : 1][32], sum_sh[G > 1 ? G : 1];
  tc::grid_launch_dependents();
  tc::grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, grp = warp % G;
  const int quads = p.row_tile / 4;  // row groups of a tile
  int64_t task = int64_t(blockIdx.x) * (kWarps / G) + warp / G;
  const int x = int(task & 3) * 32 + lane;  // channel of the block
  task >>= 2;
  const int quad = int(task % quads);
  task /= quads;
  const int j = int(task % kBlocks);
  task /= kBlocks;
  const int tile = int(task % p.n_row_tiles), b = int(task / p.n_row_tiles);
  if (b >= p.num_seqs) return;  // (G > 1: whole CTAs; the grid is exact)
  const int2 sp = reinterpret_cast<const int2*>(p.splits)[b];
  const int row = tile * p.row_tile + 4 * quad;
  const int n = min(sp.y, 2 * p.slots - sp.x);
  // an unsplit request was written by the attention kernel; a padding request
  // is left alone; the rows past the last are not anyone's
  if (n <= 0 || sp.x < 0 || p.seq_lens[b] <= 0 || row >= p.n_q) return;
  const int rows4 = p.n_row_tiles * quads;  // float4 per partial in m_part / l_part
  const float4* mp = reinterpret_cast<const float4*>(p.m_part) + int64_t(sp.x) * rows4 + row / 4;
  const float4* lp = reinterpret_cast<const float4*>(p.l_part) + int64_t(sp.x) * rows4 + row / 4;
  const int64_t ostep = int64_t(p.n_row_tiles) * kBlocks * quads * 128;
  const float4* op = reinterpret_cast<const float4*>(p.o_part) + int64_t(sp.x) * ostep +
                     ((int64_t(tile) * kBlocks + j) * quads + quad) * 128 + x;

  const float4 none = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
  float4 M = none, sum = make_float4(0.f, 0.f, 0.f, 0.f), acc = sum;
  float4 o[U], m[U], l[U];
  auto load = [&](int s0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = s0 + u * G;
      if (s < n) {
        m[u] = mp[int64_t(s) * rows4];
        l[u] = lp[int64_t(s) * rows4];
        o[u] = op[int64_t(s) * ostep];
      } else {
        m[u] = none;
      }
    }
  };
  load(grp);
  if (G == 1 && n <= U) {
#pragma unroll
    for (int u = 0; u < U; ++u) M = max4(M, m[u]);
  } else {
    for (int s = lane; s < n; s += 32) M = max4(M, mp[int64_t(s) * rows4]);
    M = make_float4(warp_max(M.x), warp_max(M.y), warp_max(M.z), warp_max(M.w));
  }
  for (int s0 = grp; s0 < n; s0 += U * G) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float4 w = make_float4(weight(m[u].x, M.x), weight(m[u].y, M.y), weight(m[u].z, M.z), weight(m[u].w, M.w));
      add_w4(sum, w, l[u]);
      add_w4(acc, w, o[u]);
    }
    if (s0 + U * G < n) load(s0 + U * G);
  }
  if constexpr (G > 1) {
    acc_sh[grp][lane] = acc;
    if (lane == 0) sum_sh[grp] = sum;
    __syncthreads();
    if (grp > 0) return;
    const float4 one = make_float4(1.f, 1.f, 1.f, 1.f);
#pragma unroll
    for (int k = 1; k < G; ++k) {
      add_w4(acc, one, acc_sh[k][lane]);
      add_w4(sum, one, sum_sh[k]);
    }
  }
  const float ds0 = p.descale[0];
  // a row without a key has sum 0; a NaN among the logits leaves NaN in both
  auto quotient = [&](float a, float s) { return s == 0.f ? 0.f : a * (ds0 / s); };
  const float v[4] = {quotient(acc.x, sum.x), quotient(acc.y, sum.y), quotient(acc.z, sum.z), quotient(acc.w, sum.w)};
  // two lanes trade, so that each holds two channels of one row
  const bool odd = x & 1;
#pragma unroll
  for (int k = 0; k < 4; k += 2) {
    const float other = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[k] : v[k + 1], 1);
    const float lo = odd ? other : v[k], hi = odd ? v[k + 1] : other;
    const int r = row + k + (odd ? 1 : 0);
    if (r < p.n_q) {
      const int tq = r / p.h, h = r - tq * p.h;
      *reinterpret_cast<uint32_t*>(p.out + (int64_t(b) * p.q_len + tq) * p.out_ts + int64_t(h) * p.out_hs + 128 * j +
                                   (x & ~1)) =
          uint32_t(float_to_out_bits(lo, p.out_f16)) | (uint32_t(float_to_out_bits(hi, p.out_f16)) << 16);
    }
  }
  if (p.lse && j == 0 && x == 0) {
    const float mv[4] = {M.x, M.y, M.z, M.w}, sv[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (row + k < p.n_q)
        p.lse[int64_t(b) * p.n_q + row + k] =
            sv[k] == 0.f ? -INFINITY : (mv[k] + fast_log2(sv[k])) * kLn2;
  }
}

template <int G>
cudaError_t launch(const LatentParams& p, int64_t tasks, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  const int64_t ctas = (tasks + kWarps / G - 1) / (kWarps / G);
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, latent_merge_kernel<G>, p);
}

}  // namespace

cudaError_t launch_latent_merge(const LatentParams& p, cudaStream_t stream) {
  const int64_t tasks = int64_t(p.num_seqs) * p.n_row_tiles * kBlocks * p.row_tile;  // x 4 channel quarters / 4 rows
  // a CTA a task while those CTAs are few
  return tasks <= 2 * int64_t(p.slots) * p.n_row_tiles ? launch<kWarps>(p, tasks, stream) : launch<1>(p, tasks, stream);
}

}  // namespace mj
