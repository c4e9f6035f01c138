// mj_block_write_kv: quantize new keys and values into the block-scaled cache.
//
// For a block of tokens and a KV head the exponent e' is the smallest with
// amax <= 448 * 2^(e' - 127) over the call's tokens there, and not below the
// block's own where earlier tokens stay in it. From amax's float32 bits that is
// their exponent field less 8, one more where the mantissa is above 1.75 (448 =
// 1.75 * 2^8): an addition that carries. Scales are powers of two, so x * 2^(127 - e')
// is exact and the only rounding is the one to e4m3.
//
// The call's tokens of a block form a run (they follow one another, padding
// tokens aside, however many). A CTA looks through a window of tokens for runs that begin
// there; its warps then take the run's (KV head, K or V) pairs in turn, each
// warp 4 KB of the input in registers: one read of the input, one maximum
// over the warp (over the block's warps where it takes several), one
// write. It cannot do without 2 bytes read and 1 written a channel; what bounds a
// long call is how many reads are in flight (21 warps an SM of 78 registers; DRAM 38% busy in a capture),
// a short one the chain slots, rows, maximum, exponent.
#include <atomic>

#include "kv_codec.cuh"
#include "mj_block.h"
#include "mj_device.cuh"
#include "tc_ptx.cuh"

namespace mj {

namespace {

// Rows of a warp: 4 KB of input, 32 registers a thread.
__host__ __device__ constexpr int rows_warp(int d) { return 2048 / d; }
__host__ __device__ constexpr int warps_cta(int g) { return g > 8 ? g : 8; }

__device__ __forceinline__ uint4 load16(const uint16_t* at) { return __ldcg(reinterpret_cast<const uint4*>(at)); }

// largest |x| bits of the 16-bit halves of v, and 0 for infinities and NaN where FINITE
template <bool FINITE>
__device__ __forceinline__ uint32_t amax_bits(uint32_t m, const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t a = w[i] & 0x7FFF7FFFu;
    if constexpr (FINITE) {
      if ((a & 0xFFFFu) >= 0x7F80u) a &= 0xFFFF0000u;
      if ((a >> 16) >= 0x7F80u) a &= 0xFFFFu;
    }
    m = __vmaxu2(m, a);
  }
  return m;
}

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  return uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3)) |
         (uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3)) << 16);
}

// The first live token of the call at or after `from` (DIR 1) or at or before it
// (DIR -1); -1 where there is none. For a whole warp: 256 tokens a step.
template <int DIR>
__device__ __noinline__ int64_t find_live(const int64_t* slots, int64_t from, int64_t num_tokens, int64_t num_slots, int lane) {
  for (int64_t t0 = from; t0 >= 0 && t0 < num_tokens; t0 += DIR * 256) {
    int64_t s[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int64_t t = t0 + DIR * (32 * u + lane);
      s[u] = t >= 0 && t < num_tokens ? slots[t] : -1;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const unsigned m = __ballot_sync(~0u, s[u] >= 0 && s[u] < num_slots);
      if (m) return t0 + DIR * (32 * u + __ffs(m) - 1);
    }
  }
  return -1;
}

// G warps share a block of G rows_warp(D) rows. Three CTAs of 8 warps an SM, 80 registers: the
// moves of earlier codes are a loop of their own, since few runs have them. (4 x 4096 tokens of
// 8 heads of 128: 22.8 us over inputs that L2 does not hold, 4.4 TB/s. The others in graphs of the same
// inputs again and again, partly in L2: 19.8 us; two CTAs of 120 registers 21.6 us; four, or half the rows a
// warp, 18.2 us, but then 11 ragged chunks of 3..701 tokens, head size 256, which take 9.0 us
// here (12.9 where L2 does not hold them), take 10.6 and 11.3, and 64 tokens 3.3 and 3.6 us in place of 3.1.)
template <int D, int G>
__global__ void __launch_bounds__(32 * warps_cta(G), 24 / warps_cta(G)) block_write_kernel(BlockWriteParams p) {
  constexpr int kWarps = warps_cta(G), kRowsWarp = rows_warp(D);
  constexpr int kLanesRow = D / 8;             // lanes a row: 8 channels, 16 bytes of input each
  constexpr int kRowsIt = 32 / kLanesRow;      // rows a warp takes at once
  constexpr int kIts = kRowsWarp / kRowsIt;
  constexpr int kGroups = kWarps / G;
  __shared__ int map[kWarps][kRowsWarp];       // token + 1 that the call writes to each of the warp's rows; 0: none
  __shared__ uint32_t top[kWarps];
  tc::grid_launch_dependents();
  tc::grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / G, part = warp % G;  // rows 16 part .. of the block
  const int64_t T = p.num_tokens;
  const int block = 1 << p.block_shift;
  auto alive = [&](int64_t s) { return s >= 0 && s < p.num_slots; };

  const int64_t w0 = int64_t(blockIdx.x) * p.window, w1 = min(T, w0 + p.window);
  for (int64_t t0 = w0; t0 < w1; t0 += 32) {
    // lane l: token t0 + l, and whether a run begins there: the live token before it
    // is of another block
    const int64_t t = t0 + lane;
    const int64_t s = t < w1 ? p.slots[t] : -1;
    int64_t at = t0 - 1, before = t0 > 0 ? p.slots[at] : -1;  // (on its way together with s)
    const bool live = alive(s);
    if (p.status && s >= p.num_slots && blockIdx.y == 0 && warp == 0) atomicOr(p.status, kStatusBadPage);
    const unsigned mask = __ballot_sync(~0u, live);
    if (!mask) continue;
    const int64_t b = s >> p.block_shift;
    const unsigned below = mask & ((1u << lane) - 1u);
    int64_t pb = __shfl_sync(~0u, b, below ? 31 - __clz(below) : 0);
    if (lane == __ffs(mask) - 1) pb = -1;
    if (t0 > 0) {  // the window's first live token looks back past its begin
      if (!alive(before)) {
        at = find_live<-1>(p.slots, at, T, p.num_slots, lane);
        before = at >= 0 ? p.slots[at] : -1;
      }
      if (lane == __ffs(mask) - 1 && before >= 0) pb = before >> p.block_shift;
    }
    unsigned leaders = __ballot_sync(~0u, live && pb != b);

    while (leaders) {
      const int l = __ffs(leaders) - 1;
      leaders &= leaders - 1;
      const int64_t B = __shfl_sync(~0u, b, l);
      // the run's tokens, by row
      if (lane < kRowsWarp) map[warp][lane] = 0;
      __syncwarp();
      int first = block;
      for (int64_t c0 = t0 + l; c0 >= 0 && c0 < T;) {
        const int64_t c = c0 + lane;
        const int64_t cs = c < T ? p.slots[c] : -1;
        const bool cl = alive(cs), same = cl && (cs >> p.block_shift) == B;
        const unsigned other = __ballot_sync(~0u, cl && !same);
        unsigned mine = __ballot_sync(~0u, same);
        if (other) mine &= (other & (0u - other)) - 1u;  // up to the next block's first token
        if (mine >> lane & 1u) {
          const int row = int(cs) & (block - 1);
          first = min(first, row);
          if (row / kRowsWarp == part) map[warp][row & (kRowsWarp - 1)] = int(c) + 1;
        }
        if (other) break;
        c0 += 32;
        if (!mine && c0 < T) c0 = find_live<1>(p.slots, c0, T, p.num_slots, lane);
      }
      first = __reduce_min_sync(~0u, first);
      __syncwarp();

      const int64_t page = (B << p.block_shift) >> p.page_shift;
      const int row0 = int((B << p.block_shift) & ((1 << p.page_shift) - 1)) + kRowsWarp * part;
      const int sub = lane / kLanesRow, ch = (lane % kLanesRow) * 8;
      for (int c = blockIdx.y * kGroups + group; c < 2 * p.h_k; c += gridDim.y * kGroups) {
        const int g = c >> 1;
        const bool v = c & 1;
        const BlockSide& sd = p.side[v];
        uint8_t* ep = sd.exps + page * sd.esp + g * sd.esh + (row0 >> p.block_shift);
        const uint16_t* src = p.in[v] + g * p.hs[v] + ch;
        int old = 0;
        if (first > 0) old = *reinterpret_cast<volatile uint8_t*>(ep);
        uint4 x[kIts];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kIts; ++i) {
          const int tok = map[warp][i * kRowsIt + sub];
          x[i] = tok ? load16(src + (tok - 1) * p.ts[v]) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < kIts; ++i) m = amax_bits<false>(m, x[i]);
        m = __reduce_max_sync(~0u, max(m & 0xFFFFu, m >> 16));
        if (m >= 0x7F80u) {  // infinities or NaN: the finite values decide
          m = 0;
#pragma unroll
          for (int i = 0; i < kIts; ++i) m = amax_bits<true>(m, x[i]);
          m = __reduce_max_sync(~0u, max(m & 0xFFFFu, m >> 16));
        }
        if constexpr (G > 1) {
          // over the block's warps; the byte is written behind the second barrier,
          // when all of them have read it
          if (lane == 0) top[warp] = m;
          tc::named_bar_sync(1 + group, 32 * G);
#pragma unroll
          for (int k = 0; k < G; ++k) m = max(m, top[group * G + k]);
          tc::named_bar_sync(1 + group, 32 * G);
        }
        int e = block_exp(int(((m << 16) + 0x1FFFFFu) >> 23) - 8);
        old = block_exp(old);
        if (first > 0) e = max(e, old);
        __syncwarp();
        if (part == 0 && lane == 0) *ep = uint8_t(e);
        const float inv = __int_as_float((254 - e) << 23);  // 2^(127 - e)
        uint8_t* dst = sd.codes + page * sd.sp + int64_t(row0) * sd.st + g * sd.sh + ch;
#pragma unroll
        for (int i = 0; i < kIts; ++i) {
          const int r = i * kRowsIt + sub;
          if (map[warp][r]) {
            float f[8];
            bf16x8_to_float(x[i], f);
            *reinterpret_cast<uint2*>(dst + r * sd.st) =
                make_uint2(codes4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                           codes4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
          }
        }
        if (first > 0 && e > old && first > kRowsWarp * part) {
          // the earlier tokens move to the larger scale
          const float by = __int_as_float((127 + old - e) << 23);
          const int n = min(kRowsWarp, first - kRowsWarp * part);
#pragma unroll 2
          for (int r = sub; r < n; r += kRowsIt) {
            uint2* at = reinterpret_cast<uint2*>(dst + r * sd.st);
            const uint2 y = *at;
            float f[8];
            e4m3x4_to_float(y.x, f);
            e4m3x4_to_float(y.y, f + 4);
            *at = make_uint2(codes4(f[0] * by, f[1] * by, f[2] * by, f[3] * by),
                             codes4(f[4] * by, f[5] * by, f[6] * by, f[7] * by));
          }
        }
      }
      __syncwarp();  // the map is rewritten for the next run
    }
  }
}

template <int D, int G>
cudaError_t launch(BlockWriteParams p, cudaStream_t stream) {
  constexpr int kWarps = warps_cta(G), kGroups = kWarps / G;
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
  // Six CTAs an SM where the call has the work: first from the (head, side)
  // pairs, then from shorter windows; a window is never longer than a block.
  const int64_t want = 6 * int64_t(sms), pairs = (2 * int64_t(p.h_k) + kGroups - 1) / kGroups;
  const int64_t y_max = std::min<int64_t>(pairs, 65535);
  p.window = rows_warp(D) * G;
  while (p.window > 1 && (int64_t(p.num_tokens) + p.window - 1) / p.window * y_max < want) p.window /= 2;
  const int64_t ctas = (int64_t(p.num_tokens) + p.window - 1) / p.window;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas), unsigned(std::min(y_max, (want + ctas - 1) / ctas)));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, block_write_kernel<D, G>, p);
}

template <int D>
cudaError_t launch_block(const BlockWriteParams& p, cudaStream_t stream) {
  switch (p.block_shift) {
    case 4: return launch<D, 16 / rows_warp(D)>(p, stream);
    case 5: return launch<D, 32 / rows_warp(D)>(p, stream);
    case 6: return launch<D, 64 / rows_warp(D)>(p, stream);
    default: return launch<D, 128 / rows_warp(D)>(p, stream);
  }
}

}  // namespace

cudaError_t launch_block_write(BlockWriteParams p, int d, cudaStream_t stream) {
  return d == 256 ? launch_block<256>(p, stream) : launch_block<128>(p, stream);
}

}  // namespace mj
