// mj_block_read_kv: cached tokens back as bf16 or fp16 rows.
//
// A warp takes 32 output rows of one KV head of K or V. Its lanes first find
// their row's request (a binary search in the row offsets), page and row; then
// groups of D / 8 lanes take a token each, a lane 8 channels: 8 bytes of codes
// in, 16 bytes out, so that each load and each store of a warp covers whole rows.
// HBM bounds it: 1 byte read and 2 written a channel. 12 requests of 500 to 16384
// tokens, 8 heads of 128: 108 us, 6.3 TB/s, 94% of a copy's rate. (16 bytes in and 32 out a lane, two
// stores of half-sectors: 112 us.)
#include "mj_block.h"
#include "mj_device.cuh"
#include "tc_ptx.cuh"

namespace mj {

namespace {

constexpr int kThreads = 256;

template <bool F16>
__device__ __forceinline__ uint32_t out2(float a, float b) {
  return F16 ? uint32_t(float_to_f16_bits(a)) | (uint32_t(float_to_f16_bits(b)) << 16)
             : uint32_t(float_to_bf16_bits(a)) | (uint32_t(float_to_bf16_bits(b)) << 16);
}

// Eight loads ahead in 64 registers, four CTAs an SM (same call: four ahead 119 us; sixteen
// ahead, three CTAs 117 us).
template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 4) block_read_kernel(BlockReadParams p) {
  constexpr int kLanesRow = D / 8;         // lanes a row
  constexpr int kRowsIt = 32 / kLanesRow;  // rows at once
  constexpr int kIts = 32 / kRowsIt;
  tc::grid_launch_dependents();
  tc::grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t(blockIdx.x) * kThreads + threadIdx.x) >> 5;
  const int pairs = p.h_k * p.sides;
  const int64_t t0 = unit / pairs * 32;
  if (t0 >= p.num_rows) return;
  const int c = int(unit % pairs);
  const int g = c / p.sides, v = p.side0 + c % p.sides;

  // this lane's row: its page (-1: none, zeros; -2: past the end, not written) and row there
  int page = -2, row = 0;
  const int64_t t = t0 + lane;
  if (t < p.num_rows && t < p.starts[p.num_seqs]) {
    int lo = 0, hi = p.num_seqs;  // starts[lo] <= t < starts[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.starts[mid] <= t)
        lo = mid;
      else
        hi = mid;
    }
    const int64_t tok = (p.first ? int64_t(p.first[lo]) : 0) + (t - p.starts[lo]);
    const int64_t e = tok >> p.page_shift;
    page = -1;
    row = int(tok) & ((1 << p.page_shift) - 1);
    if (tok >= 0 && e < p.bt_len) {
      const int pg = p.block_table[lo * p.bt_stride + e];
      if (pg >= 0 && pg < p.num_pages) page = pg;
    }
    if (page < 0 && p.status && c == 0) atomicOr(p.status, kStatusBadPage);
  }

  const BlockSide& sd = p.side[v];
  const int sub = lane / kLanesRow, ch = (lane % kLanesRow) * 8;
  const uint8_t* codes = sd.codes + g * sd.sh + ch;
  const uint8_t* exps = sd.exps + g * sd.esh;
  uint16_t* out = p.out[v] + t0 * p.ts[v] + g * p.hs[v] + ch;
  constexpr int U = 8;
#pragma unroll
  for (int i0 = 0; i0 < kIts; i0 += U) {
    uint2 x[U];
    int ex[U], pg[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int from = (i0 + u) * kRowsIt + sub;
      pg[u] = __shfl_sync(~0u, page, from);
      const int r = __shfl_sync(~0u, row, from);
      x[u] = make_uint2(0u, 0u);
      ex[u] = 127;
      if (pg[u] >= 0) {
        x[u] = __ldcg(reinterpret_cast<const uint2*>(codes + pg[u] * sd.sp + r * sd.st));
        ex[u] = exps[pg[u] * sd.esp + (r >> p.block_shift)];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (pg[u] < -1) continue;
      const float by = __int_as_float(block_exp(ex[u]) << 23);
      const uint32_t w[2] = {x[u].x, x[u].y};
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float f[4];
        e4m3x4_to_float(w[k], f);
        o[2 * k] = out2<F16>(f[0] * by, f[1] * by);
        o[2 * k + 1] = out2<F16>(f[2] * by, f[3] * by);
      }
      uint4* dst = reinterpret_cast<uint4*>(out + int64_t((i0 + u) * kRowsIt + sub) * p.ts[v]);
      __stcs(dst, make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
}

template <int D, bool F16>
cudaError_t launch(const BlockReadParams& p, cudaStream_t stream) {
  const int64_t units = (p.num_rows + 31) / 32 * p.h_k * p.sides;
  const int64_t ctas = (units + kThreads / 32 - 1) / (kThreads / 32);
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, block_read_kernel<D, F16>, p);
}

}  // namespace

cudaError_t launch_block_read(const BlockReadParams& p, int d, cudaStream_t stream) {
  if (d == 256) return p.out_f16 ? launch<256, true>(p, stream) : launch<256, false>(p, stream);
  return p.out_f16 ? launch<128, true>(p, stream) : launch<128, false>(p, stream);
}

}  // namespace mj
