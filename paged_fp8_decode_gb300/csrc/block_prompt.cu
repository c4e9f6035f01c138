// mj_block_prompt: attention of ragged prompt chunks over the block-scaled cache.
//
// A CTA takes 32 query rows (tokens x heads of one KV head) of one request and
// one piece of their keys, 32 keys at a time: codes to float32 in shared memory,
// a lane to a key for the scores, a lane to channels for the output, one pass
// with the running maximum and sum of each row.
#include "mj_block.h"
#include "mj_device.cuh"
#include "tc_ptx.cuh"

namespace mj {

namespace {

constexpr int kRowsWarp = 8, kWarps = 4, kRows = kRowsWarp * kWarps, kKeys = 32;

template <int D>
__global__ void __launch_bounds__(32 * kWarps) block_prompt_kernel(BlockPromptParams p) {
  extern __shared__ float sm[];
  float* qs = sm;                       // [kRows][D]
  float* ks = qs + kRows * D;           // [kKeys][D + 1]
  float* vs = ks + kKeys * (D + 1);     // [kKeys][D]
  constexpr int C = D / 32;
  tc::grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int piece = int(blockIdx.y) % p.splits, g = int(blockIdx.y) / p.splits, b = blockIdx.z;
  const int t0 = max(0, p.q_starts[b]), n = min(p.q_starts[b + 1], p.num_tokens) - t0;
  const int L = p.seq_lens[b];
  const int r0 = int(blockIdx.x) * kRows;
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && n > p.max_q_len) atomicOr(p.status, kStatusBadPlan);
  const int rows = min(n, p.max_q_len) * p.h_r;
  if (r0 >= rows) return;
  const int nr = min(kRows, rows - r0);
  const int last = p.causal ? L - n + (r0 + nr - 1) / p.h_r : L - 1;  // the last key that any row sees
  const int tiles = max(0, min(last + 1, L) + kKeys - 1) / kKeys;
  const int each = (tiles + p.splits - 1) / p.splits;
  const int k0 = piece * each * kKeys, k1 = min(min(L, max(0, last + 1)), (piece + 1) * each * kKeys);

  for (int i = threadIdx.x; i < kRows * D; i += 32 * kWarps) {
    const int r = i / D, row = r0 + r;
    float v = 0.f;
    if (r < nr)
      v = bf16_bits_to_float(p.q[(t0 + int64_t(row / p.h_r)) * p.q_ts + (int64_t(g) * p.h_r + row % p.h_r) * p.q_hs + i % D]);
    qs[i] = v;
  }
  float m[kRowsWarp], l[kRowsWarp], acc[kRowsWarp][C];
#pragma unroll
  for (int r = 0; r < kRowsWarp; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[r][c] = 0.f;
  }
  for (int j0 = k0; j0 < k1; j0 += kKeys) {
    __syncthreads();
    for (int i = threadIdx.x; i < kKeys * (D / 4); i += 32 * kWarps) {
      const int k = i / (D / 4), c = i % (D / 4) * 4;
      float kf[4] = {0.f, 0.f, 0.f, 0.f}, vf[4] = {0.f, 0.f, 0.f, 0.f};
      if (j0 + k < k1) {
        const int64_t e = int64_t(j0 + k) >> p.page_shift;
        const int pg = e < p.bt_len ? p.block_table[b * p.bt_stride + e] : -1;
        const int row = (j0 + k) & ((1 << p.page_shift) - 1);
        if (pg >= 0 && pg < p.num_pages) {
          const BlockSide &K = p.side[0], &V = p.side[1];
          e4m3x4_to_float(*reinterpret_cast<const uint32_t*>(K.codes + pg * K.sp + row * K.st + g * K.sh + c), kf);
          e4m3x4_to_float(*reinterpret_cast<const uint32_t*>(V.codes + pg * V.sp + row * V.st + g * V.sh + c), vf);
          const float kx = __int_as_float(block_exp(K.exps[pg * K.esp + g * K.esh + (row >> p.block_shift)]) << 23);
          const float vx = __int_as_float(block_exp(V.exps[pg * V.esp + g * V.esh + (row >> p.block_shift)]) << 23);
          for (int u = 0; u < 4; ++u) kf[u] *= kx, vf[u] *= vx;
        } else if (c == 0) {
          atomicOr(p.status, kStatusBadPage);
        }
      }
      for (int u = 0; u < 4; ++u) ks[k * (D + 1) + c + u] = kf[u], vs[k * D + c + u] = vf[u];
    }
    __syncthreads();
    float s[kRowsWarp] = {};
    const float* q = qs + warp * kRowsWarp * D;
    for (int c = 0; c < D; ++c) {
      const float k = ks[lane * (D + 1) + c];
#pragma unroll
      for (int r = 0; r < kRowsWarp; ++r) s[r] = fmaf(q[r * D + c], k, s[r]);
    }
#pragma unroll
    for (int r = 0; r < kRowsWarp; ++r) {
      const int row = r0 + warp * kRowsWarp + r, j = j0 + lane;
      const bool see = j < k1 && (!p.causal || j <= L - n + row / p.h_r);
      const float t = see ? s[r] * p.scale_log2 : -INFINITY;
      const float top = fmaxf(m[r], warp_max(t));
      const float by = m[r] == -INFINITY ? 0.f : exp2f(m[r] - top);
      s[r] = see ? exp2f(t - top) : 0.f;
      l[r] = l[r] * by + warp_sum(s[r]);
      m[r] = top;
#pragma unroll
      for (int c = 0; c < C; ++c) acc[r][c] *= by;
    }
    for (int k = 0; k < kKeys; ++k) {
      float v[C];
#pragma unroll
      for (int c = 0; c < C; ++c) v[c] = vs[k * D + lane + 32 * c];
#pragma unroll
      for (int r = 0; r < kRowsWarp; ++r) {
        const float w = __shfl_sync(~0u, s[r], k);
#pragma unroll
        for (int c = 0; c < C; ++c) acc[r][c] = fmaf(w, v[c], acc[r][c]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kRowsWarp; ++r) {
    const int row = r0 + warp * kRowsWarp + r;
    if (row >= rows) break;
    const int64_t t = t0 + int64_t(row / p.h_r), h = int64_t(g) * p.h_r + row % p.h_r;
    const int64_t part = (int64_t(piece) * p.num_tokens + t) * p.h_q + h;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float o = l[r] == 0.f ? 0.f : acc[r][c] / l[r];
      if (p.splits > 1)
        p.o_part[part * D + lane + 32 * c] = o;
      else
        p.out[t * p.out_ts + h * p.out_hs + lane + 32 * c] = float_to_out_bits(o, p.out_f16);
    }
    if (lane == 0) {
      if (p.splits > 1) {
        p.m_part[part] = m[r];
        p.l_part[part] = l[r];
      } else if (p.lse) {
        p.lse[t * p.h_q + h] = l[r] == 0.f ? -INFINITY : (m[r] + log2f(l[r])) * kLn2;
      }
    }
  }
}

template <int D>
cudaError_t launch(const BlockPromptParams& p, cudaStream_t stream) {
  constexpr int bytes = (kRows * D + kKeys * (2 * D + 1)) * 4;
  cudaError_t e = cudaFuncSetAttribute(block_prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  const dim3 grid(unsigned((int64_t(p.max_q_len) * p.h_r + kRows - 1) / kRows), unsigned(p.h_k * p.splits), unsigned(p.num_seqs));
  block_prompt_kernel<D><<<grid, 32 * kWarps, bytes, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_block_prompt(const BlockPromptParams& p, cudaStream_t stream) {
  return p.d == 256 ? launch<256>(p, stream) : launch<128>(p, stream);
}

}  // namespace mj
