// Joins the partials of mj_latent_attention's split requests: for request b
// and row r, over its partials s (unnormalised output O~, reference max m in
// the log2 domain, sum l, both scaled by 2^m):
//   M = max_s m_s,  out = s0 sum_s 2^(m_s - M) O~_s / sum_s 2^(m_s - M) l_s.
// A partial without a key has m = -inf and is selected off (its O~ and l may
// never have been written). One lane a request compares its length with the
// tiles that the plan covers, and reports tokens past them: no CTA read those.
//
// Bound by latency and L2: tens of megabytes of partials at most, just
// written. Many tasks: a warp joins four rows of 128 channels, four 16-byte
// loads a lane and partial, two partials requested at a time. Few (a long
// request split over the whole GPU): four rows of 32 channels to a CTA, whose 16
// warps share the partials and meet in shared memory. Measured as a share of the
// step: 12 us of 48 requests of 128 heads (28 MB of partials, 28 us with 64-bit
// index divisions), 3 us of 64 x 4096 tokens with 16 heads, 6 us of one request
// in 147 pieces.
#include "mj_device.cuh"
#include "mj_latent.h"
#include "tc_ptx.cuh"

namespace mj {

namespace {

constexpr int kBlocks = MJ_LATENT_DIM / 128;

// One row's running join: the largest reference so far and the sum scaled to it.
struct Row {
  float top = -INFINITY, sum = 0.f;
};

// Takes a partial in; the factors of the output so far and of the partial's. A
// partial with m = -inf changes nothing (and its numbers are not used).
__device__ __forceinline__ float2 join(Row& r, float m, float l) {
  if (m == -INFINITY) return make_float2(1.f, 0.f);
  const float top = fmaxf(r.top, m);
  const float2 f = make_float2(fast_exp2(r.top - top), fast_exp2(m - top));  // (the first time r.top = -inf: 0)
  r.sum = fmaf(r.sum, f.x, f.y * l);
  r.top = top;
  return f;
}
__device__ __forceinline__ float scale_add(float acc, float2 f, float o) {
  return f.y == 0.f ? acc * f.x : fmaf(acc, f.x, f.y * o);
}

constexpr int kWarps = 4;

template <int G, int K>  // warps a task; channel quarters of a lane
__global__ void __launch_bounds__(G > 1 ? 32 * G : 32 * kWarps) latent_merge_kernel(LatentParams p) {
  constexpr int U = G > 1 ? 5 : 2;  // partials in flight a warp
  __shared__ float4 acc_sh[G > 1 ? G : 1][32], sum_sh[G > 1 ? G : 1], max_sh[G > 1 ? G : 1];
  tc::grid_launch_dependents();
  tc::grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // task = (((request, row tile), row group of the tile), block[, quarter of its channels]): 32-bit, and
  // shifts but for the row tile (64-bit divisions here took longer than the loads)
  constexpr int kQ = K == 4 ? 0 : 2;
  const int qs = p.row_tile == 16 ? 2 : (p.row_tile == 32 ? 3 : 4), quads = 1 << qs;
  const uint32_t task = G > 1 ? blockIdx.x : blockIdx.x * kWarps + uint32_t(warp);
  const int x = (K == 4 ? 0 : int(task & 3u) * 32) + lane;  // first channel of the block
  const int j = int(task >> kQ) & (kBlocks - 1), quad = int(task >> (kQ + 2)) & (quads - 1);
  const uint32_t rt = task >> (kQ + 2 + qs);
  const int b = int(rt / uint32_t(p.n_row_tiles)), tile = int(rt) - b * p.n_row_tiles;
  if (b >= p.num_seqs) return;  // (G > 1: whole CTAs; the grid is exact)
  const int2 sp = reinterpret_cast<const int2*>(p.splits)[b];
  const int len = p.seq_lens[b];
  const int row = tile * p.row_tile + 4 * quad;
  if (j == 0 && quad == 0 && tile == 0 && x == 0 && (G == 1 || warp == 0) && int64_t(len) > int64_t(p.planned[b]) * kKvTile)
    atomicOr(p.status, kStatusBadPlan);
  const int n = min(sp.y, 2 * p.slots - sp.x);
  // an unsplit request was written by the attention kernel; a padding request
  // is left alone; the rows past the last are not anyone's
  if (n <= 0 || sp.x < 0 || len <= 0 || row >= p.n_q) return;
  const int rows4 = p.n_row_tiles * quads;  // float4 per partial in m_part / l_part
  const float4* mp = reinterpret_cast<const float4*>(p.m_part) + int64_t(sp.x) * rows4 + row / 4;
  const float4* lp = reinterpret_cast<const float4*>(p.l_part) + int64_t(sp.x) * rows4 + row / 4;
  const int64_t ostep = int64_t(p.n_row_tiles) * kBlocks * quads * 128;
  const float4* op = reinterpret_cast<const float4*>(p.o_part) + int64_t(sp.x) * ostep +
                     ((int64_t(tile) * kBlocks + j) * quads + quad) * 128 + x;

  Row r[4];
  float4 acc[K];
#pragma unroll
  for (int k = 0; k < K; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  // one partial into the running join
  auto add = [&](float4 m, float4 l, const float4* o) {
    const float2 f0 = join(r[0], m.x, l.x), f1 = join(r[1], m.y, l.y), f2 = join(r[2], m.z, l.z), f3 = join(r[3], m.w, l.w);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      acc[k].x = scale_add(acc[k].x, f0, o[k].x);
      acc[k].y = scale_add(acc[k].y, f1, o[k].y);
      acc[k].z = scale_add(acc[k].z, f2, o[k].z);
      acc[k].w = scale_add(acc[k].w, f3, o[k].w);
    }
  };
  for (int s0 = G > 1 ? warp : 0; s0 < n; s0 += U * G) {
    float4 o[U][K], m[U], l[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = s0 + u * G;
      if (s < n) {
        m[u] = mp[int64_t(s) * rows4];
        l[u] = lp[int64_t(s) * rows4];
#pragma unroll
        for (int k = 0; k < K; ++k) o[u][k] = op[int64_t(s) * ostep + 32 * k];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s0 + u * G < n) add(m[u], l[u], o[u]);
  }
  if constexpr (G > 1) {
    acc_sh[warp][lane] = acc[0];
    if (lane == 0) {
      sum_sh[warp] = make_float4(r[0].sum, r[1].sum, r[2].sum, r[3].sum);
      max_sh[warp] = make_float4(r[0].top, r[1].top, r[2].top, r[3].top);
    }
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int k = 1; k < G; ++k) {
      const float4 o = acc_sh[k][lane];
      add(max_sh[k], sum_sh[k], &o);
    }
  }
  // a row without a key has sum 0; a NaN among the logits leaves NaN in both
  const float ds0 = p.descale[0];
  float f[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) f[k] = r[k].sum == 0.f ? 0.f : ds0 / r[k].sum;
  // two lanes trade, so that each holds two channels of one row
  const bool odd = lane & 1;
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const int rr = row + i + (odd ? 1 : 0);
    const int tq = rr / p.h, h = rr - tq * p.h;
    uint16_t* dst = p.out + (int64_t(b) * p.q_len + tq) * p.out_ts + int64_t(h) * p.out_hs + 128 * j + (x & ~1);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const float v[4] = {acc[k].x, acc[k].y, acc[k].z, acc[k].w};
      const float a = r[i].sum == 0.f ? 0.f : v[i] * f[i], c = r[i + 1].sum == 0.f ? 0.f : v[i + 1] * f[i + 1];
      const float other = __shfl_xor_sync(0xFFFFFFFFu, odd ? a : c, 1);
      const float lo = odd ? other : a, hi = odd ? c : other;
      if (rr < p.n_q)
        *reinterpret_cast<uint32_t*>(dst + 32 * k) =
            uint32_t(float_to_out_bits(lo, p.out_f16)) | (uint32_t(float_to_out_bits(hi, p.out_f16)) << 16);
    }
  }
  if (p.lse && j == 0 && x == 0) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (row + k < p.n_q)
        p.lse[int64_t(b) * p.n_q + row + k] = r[k].sum == 0.f ? -INFINITY : (r[k].top + fast_log2(r[k].sum)) * kLn2;
  }
}

template <int G, int K>
cudaError_t launch(const LatentParams& p, int64_t tasks, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  if (tasks > INT32_MAX - kWarps) return cudaErrorInvalidConfiguration;
  cfg.gridDim = dim3(unsigned(G > 1 ? tasks : (tasks + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(G > 1 ? 32 * G : 32 * kWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, latent_merge_kernel<G, K>, p);
}

}  // namespace

cudaError_t launch_latent_merge(const LatentParams& p, cudaStream_t stream) {
  const int64_t tasks = int64_t(p.num_seqs) * p.n_row_tiles * kBlocks * p.row_tile / 4;  // of 128 channels
  // a CTA for each quarter of a task while those CTAs are few
  return 4 * tasks <= 2 * int64_t(p.slots) * p.n_row_tiles ? launch<16, 1>(p, 4 * tasks, stream) : launch<1, 4>(p, tasks, stream);
}

}  // namespace mj
