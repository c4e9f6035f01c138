// The join of rows whose keys were attended to in pieces (mj_block_attention,
// mj_block_prompt): with a piece's output O_s (normalised), reference m_s and sum
// l_s = sum 2^(t - m_s), M = max_s m_s and w_s = 2^(m_s - M) l_s,
//   O = sum_s w_s O_s / sum_s w_s,   LSE = ln 2 (M + log2 sum_s w_s).
// Pieces are added in an order that does not depend on how they ran. A few
// long requests give few rows of many pieces: NW warps share a row then, each
// piece NW apart, and meet in shared memory; else a warp has a row to itself.
// The first pieces' outputs are requested before their weights are known.
#include <atomic>

#include "mj_block.h"
#include "mj_device.cuh"
#include "tc_ptx.cuh"

namespace mj {

namespace {

constexpr int kWarps = 8;
constexpr int U = 4;  // outputs a warp requests at once

template <int D, int NW>
__global__ void __launch_bounds__(32 * kWarps) block_join_kernel(BlockJoinParams p) {
  constexpr int V = D / 128;  // float4 a lane
  __shared__ float4 part[NW > 1 ? kWarps : 1][NW > 1 ? 32 * V : 1];
  __shared__ float psum[kWarps];
  tc::grid_launch_dependents();
  tc::grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w = NW > 1 ? warp : 0;
  const int64_t unit = NW > 1 ? int64_t(blockIdx.x) : int64_t(blockIdx.x) * kWarps + warp;
  if (unit >= p.units) return;

  // the row's pieces, and where it goes
  int n;
  int64_t first, step, at, lse_at;
  if (p.plan) {
    const int row = int(unit % p.n_q);
    const int64_t bg = unit / p.n_q;
    const int g = int(bg % p.h_k), b = int(bg / p.h_k);
    const int4 rq = p.plan[b];
    const int L = p.seq_lens[b];
    // a length past the tiles that the plan has of the request
    if (lane == 0 && row == 0 && g == 0 && int64_t(L) > int64_t(rq.w) * kKvTile) atomicOr(p.status, kStatusBadPlan);
    if (rq.y <= 1 || L <= 0) return;  // in one piece: already written
    if (!plan_entry_ok(rq.x, rq.y, rq.z, p.part_cap)) {  // not attended to
      if (lane == 0 && row == 0 && g == 0) atomicOr(p.status, kStatusBadPlan);
      return;
    }
    const int64_t span = int64_t(rq.z) * kKvTile;
    n = int(min(int64_t(rq.y), (int64_t(L) + span - 1) / span));  // pieces with a key
    step = int64_t(p.h_k) * p.n_q;
    first = (int64_t(rq.x) * p.h_k + g) * p.n_q + row;
    at = (int64_t(b) * p.q_len + row / p.h_r) * p.out_ts + (int64_t(g) * p.h_r + row % p.h_r) * p.out_hs;
    lse_at = bg * p.n_q + row;
  } else {
    const int64_t t = unit / p.h_q;
    if (t >= p.q_starts[p.num_seqs]) return;
    if (__ldcg(p.l_part + unit) < 0.f) return;  // not computed
    n = p.pieces;
    step = p.units;
    first = unit;
    at = t * p.out_ts + (unit % p.h_q) * p.out_hs;
    lse_at = unit;
  }
  auto load = [&](int s, float4 (&o)[V]) {
    const float4* src = reinterpret_cast<const float4*>(p.o_part + (first + s * step) * D) + lane;
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = s < n ? __ldcg(src + 32 * v) : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  float4 o[U][V];
#pragma unroll
  for (int u = 0; u < U; ++u) load(w + u * NW, o[u]);
  float M = -INFINITY;
  for (int s = lane; s < n; s += 32) M = fmaxf(M, __ldcg(p.m_part + first + s * step));
  M = warp_max(M);
  auto weight = [&](int s) {
    if (s >= n) return 0.f;
    const float m = __ldcg(p.m_part + first + s * step);
    return m > -INFINITY ? fast_exp2(m - M) * __ldcg(p.l_part + first + s * step) : 0.f;
  };
  float4 acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  // lane u's weight belongs to piece base + u NW
  for (int s0 = w; s0 < n; s0 += 32 * NW) {
    const float wl = weight(s0 + lane * NW);
    sum += wl;
    for (int u0 = 0; u0 < 32 && s0 + u0 * NW < n; u0 += U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float ws = __shfl_sync(~0u, wl, u0 + u);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          // a piece without a key has weight 0 and an output that nothing wrote
          acc[v].x = ws > 0.f ? fmaf(ws, o[u][v].x, acc[v].x) : acc[v].x + (ws != ws ? ws : 0.f);
          acc[v].y = ws > 0.f ? fmaf(ws, o[u][v].y, acc[v].y) : acc[v].y + (ws != ws ? ws : 0.f);
          acc[v].z = ws > 0.f ? fmaf(ws, o[u][v].z, acc[v].z) : acc[v].z + (ws != ws ? ws : 0.f);
          acc[v].w = ws > 0.f ? fmaf(ws, o[u][v].w, acc[v].w) : acc[v].w + (ws != ws ? ws : 0.f);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) load(s0 + (u0 + U + u) * NW, o[u]);
    }
  }
  sum = warp_sum(sum);
  if constexpr (NW > 1) {
    if (lane == 0) psum[warp] = sum;
#pragma unroll
    for (int v = 0; v < V; ++v) part[warp][lane + 32 * v] = acc[v];
    __syncthreads();
    if (warp >= V) return;
    // warp v: channels 128 v ..
    float4 a = part[0][lane + 32 * warp];
    sum = psum[0];
#pragma unroll
    for (int k = 1; k < kWarps; ++k) {
      const float4 b = part[k][lane + 32 * warp];
      a.x += b.x;
      a.y += b.y;
      a.z += b.z;
      a.w += b.w;
      sum += psum[k];
    }
    acc[0] = a;
  }
#pragma unroll
  for (int v = 0; v < (NW > 1 ? 1 : V); ++v) {
    const float4 a = acc[v];
    auto fin = [&](float x) { return uint32_t(float_to_out_bits(sum == 0.f ? 0.f : x / sum, p.out_f16)); };
    *reinterpret_cast<uint2*>(p.out + at + 4 * lane + 128 * (NW > 1 ? warp : v)) =
        make_uint2(fin(a.x) | fin(a.y) << 16, fin(a.z) | fin(a.w) << 16);
  }
  if (p.lse && lane == 0 && (NW == 1 || warp == 0))
    p.lse[lse_at] = sum == 0.f ? -INFINITY : (M + fast_log2(sum)) * kLn2;
}

template <int D>
cudaError_t launch(const BlockJoinParams& p, cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static std::atomic<int> sm_count[64];  // per device, looked up once (host threads may race)
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int sms = sm_count[dev].load(std::memory_order_relaxed);
  if (sms == 0) {
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    sm_count[dev].store(sms, std::memory_order_relaxed);
  }
  const bool shared = p.units < 4 * int64_t(sms);
  const int64_t ctas = shared ? p.units : (p.units + kWarps - 1) / kWarps;
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return shared ? cudaLaunchKernelEx(&cfg, block_join_kernel<D, kWarps>, p) : cudaLaunchKernelEx(&cfg, block_join_kernel<D, 1>, p);
}

}  // namespace

cudaError_t launch_block_join(const BlockJoinParams& p, cudaStream_t stream) {
  if (p.units == 0) return cudaSuccess;
  return p.d == 256 ? launch<256>(p, stream) : launch<128>(p, stream);
}

}  // namespace mj
