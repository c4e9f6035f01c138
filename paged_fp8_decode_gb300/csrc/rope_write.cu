// mj_rope_write_kv and mj_latent_write: rotate the new tokens' queries and keys
// by their positions and append the keys and values to a paged cache.
//
// The rotation. Frequency i of a token turns the pair (x0, x1) by the angle
// a = position * inv_freq[i]:  (x0, x1) -> m (x0 cos a - x1 sin a, x1 cos a + x0 sin a).
// A float32 product of a position near 10^6 and a frequency near 1 is off by up
// to 0.03 rad, and float64 runs at a small fraction of the float32 rate here, so
// the angle is formed in turns, in fixed point: `turns[i]` is
// inv_freq[i] / (2 pi) as a fraction of 2^64, and position * turns[i] modulo 2^64
// is the angle modulo a full turn, off by at most position * 2^-65 of a turn. Its
// upper 32 bits, read as a signed number of 2^-31 half turns (below 1e-9 rad),
// go to sincospif. Everything after is float32, with one rounding at the end: to
// bf16 (queries) or to the cache format (keys and values, the division IEEE
// float32, as mj_write_kv does it).
//
// What bounds it: HBM for many tokens (each query, key and value element is
// read once and written once), launch and load latency for few. A token's
// cosines and sines serve all its heads, so a CTA takes whole tokens: it first
// requests the elements of up to four items a thread (an item: 16 channels as
// two 16-byte chunks, a pair's two sides in one thread), then computes the
// group's cosines and sines into shared memory while they arrive.
#include <cuda_fp8.h>

#include <algorithm>
#include <atomic>

#include "kv_codec.cuh"
#include "mj_device.cuh"
#include "mj_internal.h"
#include "tc_ptx.cuh"

namespace mj {

namespace {

constexpr int kItemsPerThread = 4;  // items whose loads are in flight together

struct RopeWriteParams {
  // rotation
  const int64_t* pos;
  int64_t pos_axis;  // element stride between the axes' position rows
  int axes;
  const uint64_t* turns;
  const uint8_t* freq_axis;
  int n;  // frequencies: rot_dim / 2
  int interleaved;
  float scale;
  // tokens
  int num_tokens, group;  // tokens per CTA
  int h_q, h_k;
  const uint16_t* q;
  uint16_t* q_out;
  int64_t q_ts, q_hs, qo_ts, qo_hs;
  const uint16_t* key;
  const uint16_t* value;
  int64_t k_ts, k_hs, v_ts, v_hs;
  const int64_t* slots;
  int page_shift;  // log2(page_size)
  int64_t num_slots;
  uint8_t* k_cache;
  uint8_t* v_cache;
  int64_t k_sp, k_st, k_sh, v_sp, v_st, v_sh;
  const float* k_scale;
  const float* v_scale;
  int scale_per_head;
  uint32_t* status;
};

// 8 values of one row, channels c .. c + 7 (c a multiple of 8), to codes.
template <int F>
__device__ __forceinline__ void encode8(const float x[8], const float* scale, uint8_t* row, int c) {
  if constexpr (F == MJ_KV_E4M3) {
    const float s = scale[0];
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(
          make_float2(__fdiv_rn(x[4 * k], s), __fdiv_rn(x[4 * k + 1], s)), __NV_SATFINITE, __NV_E4M3);
      const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(
          make_float2(__fdiv_rn(x[4 * k + 2], s), __fdiv_rn(x[4 * k + 3], s)), __NV_SATFINITE, __NV_E4M3);
      w[k] = uint32_t(lo) | (uint32_t(hi) << 16);
    }
    *reinterpret_cast<uint2*>(row + c) = make_uint2(w[0], w[1]);
  } else {
    const float4* sc = reinterpret_cast<const float4*>(scale + c);
    const float4 s0 = sc[0], s1 = sc[1];
    const float sv[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
    constexpr int kBits = F == MJ_KV_E2M1 ? 4 : 6;
    uint64_t bits = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float y = __fdiv_rn(x[k], sv[k]);
      const uint64_t code = F == MJ_KV_E2M3 ? e2m3_code(y) : (F == MJ_KV_E3M2 ? e3m2_code(y) : e2m1_code(y));
      bits |= code << (kBits * k);
    }
    if constexpr (F == MJ_KV_E2M1) {
      *reinterpret_cast<uint32_t*>(row + c / 2) = uint32_t(bits);
    } else {  // 6 bytes, 2-byte aligned
      uint16_t* o = reinterpret_cast<uint16_t*>(row + c / 8 * 6);
      o[0] = uint16_t(bits);
      o[1] = uint16_t(bits >> 16);
      o[2] = uint16_t(bits >> 32);
    }
  }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float x[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = uint32_t(float_to_bf16_bits(x[2 * i])) | (uint32_t(float_to_bf16_bits(x[2 * i + 1])) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// F: the cache format; D: channels of a rotated head (queries and keys); VD:
// channels of a value head (the latent vector of mj_latent_write).
template <int F, int D, int VD>
__global__ void __launch_bounds__(256) rope_write_kernel(RopeWriteParams p) {
  constexpr int U = kItemsPerThread;
  constexpr int kD = D / 16, kVD = VD / 16;  // items of a rotated and of a value head
  extern __shared__ float2 cs[];             // [group][n]: cos and sin, times the scale
  const int tid = threadIdx.x, threads = blockDim.x;
  const int t0 = blockIdx.x * p.group;
  const int nt = min(p.group, p.num_tokens - t0);
  const int qk_items = (p.h_q + p.h_k) * kD;
  const int per_token = qk_items + p.h_k * kVD;
  const int total = nt * per_token;

  // launched with programmatic stream serialization: everything below may be
  // the preceding kernel's output. The next kernel may launch (and waits for
  // this one where it reads).
  tc::grid_launch_dependents();
  tc::grid_dependency_wait();

  struct Item {
    int tok, head, c0, c1, f;  // f: first frequency of the chunk, -1 when it is not rotated
    int kind;                  // 0 query, 1 key, 2 value
  };
  auto item_of = [&](int i) {
    Item it;
    const int tl = p.group == 1 ? 0 : i / per_token;
    const int r = i - tl * per_token;
    it.tok = t0 + tl;
    it.f = -1;
    if (r < qk_items) {
      const int hs = r / kD, j = r % kD;
      it.kind = hs < p.h_q ? 0 : 1;
      it.head = hs < p.h_q ? hs : hs - p.h_q;
      if (8 * j < p.n) {
        it.f = 8 * j;
        it.c0 = p.interleaved ? 16 * j : 8 * j;
        it.c1 = it.c0 + (p.interleaved ? 8 : p.n);
      } else {
        it.c0 = 16 * j;  // rot_dim / 16 items lie before: channels rot_dim + 16 (j - n / 8)
        it.c1 = it.c0 + 8;
      }
    } else {
      it.kind = 2;
      it.head = (r - qk_items) / kVD;
      it.c0 = ((r - qk_items) % kVD) * 16;
      it.c1 = it.c0 + 8;
    }
    return it;
  };

  bool ready = false;  // the cosines and sines are in shared memory (the same in every thread)
  for (int base = 0; base < total; base += U * threads) {
    uint4 a[U], b[U];
    int64_t slot[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = base + u * threads + tid;
      if (i < total) {
        const Item it = item_of(i);
        const uint16_t* src = it.kind == 0   ? p.q + it.tok * p.q_ts + it.head * p.q_hs
                              : it.kind == 1 ? p.key + it.tok * p.k_ts + it.head * p.k_hs
                                             : p.value + it.tok * p.v_ts + it.head * p.v_hs;
        a[u] = *reinterpret_cast<const uint4*>(src + it.c0);
        b[u] = *reinterpret_cast<const uint4*>(src + it.c1);
        slot[u] = it.kind == 0 ? -1 : p.slots[it.tok];
      }
    }
    if (!ready) {
      for (int e = tid; e < nt * p.n; e += threads) {
        const int tl = p.group == 1 ? 0 : e / p.n, f = e - tl * p.n;
        const int ax = p.axes > 1 ? min(int(p.freq_axis[f]), p.axes - 1) : 0;
        const uint64_t turn = uint64_t(p.pos[int64_t(ax) * p.pos_axis + t0 + tl]) * p.turns[f];
        float s, c;
        sincospif(float(int32_t(turn >> 32)) * 0x1p-31f, &s, &c);
        cs[e] = make_float2(c * p.scale, s * p.scale);
      }
      __syncthreads();
      ready = true;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = base + u * threads + tid;
      if (i >= total) break;
      const Item it = item_of(i);
      if (it.kind != 0) {
        if (slot[u] < 0) continue;  // a padding token
        if (slot[u] >= p.num_slots) {
          if (p.status && it.kind == 2 && it.head == 0 && it.c0 == 0) atomicOr(p.status, kStatusBadPage);
          continue;
        }
      }
      float x[8], y[8];
      bf16x8_to_float(a[u], x);
      bf16x8_to_float(b[u], y);
      if (it.f >= 0) {
        const float2* w = cs + (it.tok - t0) * p.n + it.f;
        if (p.interleaved) {  // pairs (2k, 2k + 1): x holds the first four of them, y the others
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 wa = w[k], wb = w[k + 4];
            const float x0 = x[2 * k], x1 = x[2 * k + 1], y0 = y[2 * k], y1 = y[2 * k + 1];
            x[2 * k] = x0 * wa.x - x1 * wa.y;
            x[2 * k + 1] = x1 * wa.x + x0 * wa.y;
            y[2 * k] = y0 * wb.x - y1 * wb.y;
            y[2 * k + 1] = y1 * wb.x + y0 * wb.y;
          }
        } else {  // pairs (k, k + n)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float2 wk = w[k];
            const float x0 = x[k], y0 = y[k];
            x[k] = x0 * wk.x - y0 * wk.y;
            y[k] = y0 * wk.x + x0 * wk.y;
          }
        }
      }
      if (it.kind == 0) {
        uint16_t* dst = p.q_out + it.tok * p.qo_ts + it.head * p.qo_hs;
        *reinterpret_cast<uint4*>(dst + it.c0) = pack_bf16x8(x);
        *reinterpret_cast<uint4*>(dst + it.c1) = pack_bf16x8(y);
      } else {
        const int64_t page = slot[u] >> p.page_shift, prow = slot[u] & ((int64_t(1) << p.page_shift) - 1);
        const bool key = it.kind == 1;
        uint8_t* row = key ? p.k_cache + page * p.k_sp + prow * p.k_st + it.head * p.k_sh
                           : p.v_cache + page * p.v_sp + prow * p.v_st + it.head * p.v_sh;
        const float* scale = (key ? p.k_scale : p.v_scale) +
                             (F != MJ_KV_E4M3 ? it.head * D : (p.scale_per_head ? it.head : 0));
        encode8<F>(x, scale, row, it.c0);
        encode8<F>(y, scale, row, it.c1);
      }
    }
  }
}

template <int F, int D, int VD>
cudaError_t launch(RopeWriteParams p, cudaStream_t stream) {
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
  // Tokens per CTA: enough of them for four items a thread, as long as every SM
  // still gets two CTAs; 256 threads where one token alone has more than that.
  const int64_t per_token = int64_t(p.h_q + p.h_k) * (D / 16) + int64_t(p.h_k) * (VD / 16);
  const int threads = per_token > 128 * kItemsPerThread ? 256 : 128;
  int64_t g = std::max<int64_t>(1, threads * kItemsPerThread / per_token);
  g = std::min(g, std::max<int64_t>(1, p.num_tokens / (2 * int64_t(sms))));
  p.group = int(std::min<int64_t>(g, 16));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((int64_t(p.num_tokens) + p.group - 1) / p.group));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = size_t(p.group) * p.n * sizeof(float2);  // at most 16 x 128 x 8 bytes
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_write_kernel<F, D, VD>, p);
}

template <int D>
cudaError_t launch_format(int kv_format, const RopeWriteParams& p, cudaStream_t stream) {
  switch (kv_format) {
    case MJ_KV_E2M3: return launch<MJ_KV_E2M3, D, D>(p, stream);
    case MJ_KV_E3M2: return launch<MJ_KV_E3M2, D, D>(p, stream);
    case MJ_KV_E2M1: return launch<MJ_KV_E2M1, D, D>(p, stream);
    default: return launch<MJ_KV_E4M3, D, D>(p, stream);
  }
}

int log2_of(int page_size) { return page_size == 16 ? 4 : (page_size == 32 ? 5 : (page_size == 64 ? 6 : 7)); }

void set_rope(RopeWriteParams& p, const mj_rope& r) {
  p.pos = r.positions;
  p.pos_axis = r.axis_stride;
  p.axes = r.num_axes;
  p.turns = r.turns;
  p.freq_axis = r.freq_axis;
  p.n = r.rot_dim / 2;
  p.interleaved = r.interleaved ? 1 : 0;
  p.scale = r.scale;
}

}  // namespace

cudaError_t launch_rope_write(const mj_rope_write_kv_args& a, cudaStream_t stream) {
  const mj_write_kv_args& w = a.kv;
  if (w.num_tokens == 0) return cudaSuccess;
  RopeWriteParams p = {};
  set_rope(p, a.rope);
  p.num_tokens = w.num_tokens;
  p.h_q = a.h_q;
  p.h_k = w.h_k;
  p.q = static_cast<const uint16_t*>(a.q);
  p.q_out = static_cast<uint16_t*>(a.q_out);
  p.q_ts = a.q_tok_stride;
  p.q_hs = a.q_head_stride;
  p.qo_ts = a.q_out_tok_stride;
  p.qo_hs = a.q_out_head_stride;
  p.key = static_cast<const uint16_t*>(w.key);
  p.value = static_cast<const uint16_t*>(w.value);
  p.k_ts = w.key_tok_stride;
  p.k_hs = w.key_head_stride;
  p.v_ts = w.value_tok_stride;
  p.v_hs = w.value_head_stride;
  p.slots = w.slot_mapping;
  p.page_shift = log2_of(w.page_size);
  p.num_slots = w.num_pages * w.page_size;
  p.k_cache = static_cast<uint8_t*>(w.k_cache);
  p.v_cache = static_cast<uint8_t*>(w.v_cache);
  p.k_sp = w.k_stride_page;
  p.k_st = w.k_stride_token;
  p.k_sh = w.k_stride_head;
  p.v_sp = w.v_stride_page;
  p.v_st = w.v_stride_token;
  p.v_sh = w.v_stride_head;
  p.k_scale = w.k_scale;
  p.v_scale = w.v_scale;
  p.scale_per_head = w.scale_per_head;
  p.status = w.status;
  return w.d == 256 ? launch_format<256>(w.kv_format, p, stream) : launch_format<128>(w.kv_format, p, stream);
}

// The latent row: one "head" of 512 value channels at byte 0 (its scale is
// scale[0]) and one key head of 64 rotated channels at byte 512 (scale[1]).
cudaError_t launch_latent_write(const mj_latent_write_args& a, cudaStream_t stream) {
  if (a.num_tokens == 0) return cudaSuccess;
  RopeWriteParams p = {};
  set_rope(p, a.rope);
  p.num_tokens = a.num_tokens;
  p.h_q = a.h;
  p.h_k = 1;
  p.q = static_cast<const uint16_t*>(a.q_pe);
  p.q_out = static_cast<uint16_t*>(a.q_out);
  p.q_ts = a.q_tok_stride;
  p.q_hs = a.q_head_stride;
  p.qo_ts = a.q_out_tok_stride;
  p.qo_hs = a.q_out_head_stride;
  p.key = static_cast<const uint16_t*>(a.k_pe);
  p.value = static_cast<const uint16_t*>(a.latent);
  p.k_ts = a.k_pe_tok_stride;
  p.v_ts = a.latent_tok_stride;
  p.slots = a.slot_mapping;
  p.page_shift = log2_of(a.page_size);
  p.num_slots = a.num_pages * a.page_size;
  p.v_cache = static_cast<uint8_t*>(a.cache);
  p.k_cache = p.v_cache + MJ_LATENT_DIM;
  p.k_sp = p.v_sp = a.stride_page;
  p.k_st = p.v_st = a.stride_token;
  p.v_scale = a.scale;
  p.k_scale = a.scale + 1;
  p.status = a.status;
  return launch<MJ_KV_E4M3, MJ_LATENT_ROPE_DIM, MJ_LATENT_DIM>(p, stream);
}

}  // namespace mj
