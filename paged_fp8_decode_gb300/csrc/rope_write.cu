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
// upper 32 bits, a signed number of 2^-31 half turns, go to sincospif as a float32:
// that rounds an angle near half a turn by 2^-25 of one, 1e-7 rad, far inside the
// output's own rounding. Everything after is float32, with one rounding at the end: to
// bf16 (queries) or to the cache format (keys and values, the division IEEE
// float32, as mj_write_kv does it).
//
// What bounds it: HBM for many tokens (each query, key and value element is
// read once and written once), launch and load latency for few. A token's
// cosines and sines serve all its heads, so a CTA takes whole tokens: it first
// requests the first slots of each thread (of each 16 channels as two 16-byte
// chunks, a pair's two sides in one thread), then computes the tokens' cosines
// and sines into shared memory while they arrive.
#include <cuda_fp8.h>

#include <atomic>

#include "kv_codec.cuh"
#include "mj_device.cuh"
#include "mj_latent.h"
#include "tc_ptx.cuh"

namespace mj {

namespace {

constexpr int kThreads = 128;
// Two slots of loads in flight a thread and seven CTAs an SM: 16384 tokens of
// 32/8 heads of 128 in 62.6 us (5.9 TB/s; e2m3, e3m2, e2m1, which divide every
// element: 92, 87, 89 us, 4.0 TB/s). Three slots and five CTAs: 65.6 us, and 0.2
// us less for one token; eight CTAs: 71 us. (Seven leave 72 registers: 8 bytes
// are spilled for e4m3, 24 for the packed formats, more at eight.)
constexpr int kItemsPerThread = 2, kMinCtas = 7;
// Where the CTAs of that would not be resident at once, a thread takes up to
// six slots, so that its cosines, addresses and set-up serve more of them
// (16384 tokens: 62.8 against 70.2 us); where they are, the shorter chain counts
// (32/8 heads, 900 tokens: 5.1 against 7.2 us, 1500 tokens: 9.1 against 8.6).
constexpr int kItemsMany = 6;

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
  int num_tokens, group, lanes;  // tokens per CTA, slot lanes per token (a power of two)
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

// Two float32 products or fused multiply-adds in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t x, y, d;
  memcpy(&x, &a, 8);
  memcpy(&y, &b, 8);
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
  float2 r;
  memcpy(&r, &d, 8);
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t x, y, z, d;
  memcpy(&x, &a, 8);
  memcpy(&y, &b, 8);
  memcpy(&z, &c, 8);
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
  float2 r;
  memcpy(&r, &d, 8);
  return r;
}

// Bounds of 1 / s that hold x * lo <= x / s <= x * hi in size after rounding
// (8 units of 2^-24 either way; the reciprocal and the two products are off by
// three). A scale so large or small that the reciprocal could overflow or
// vanish gets bounds that never agree.
struct Recip {
  float lo, hi;
};
__device__ __forceinline__ Recip recip_bounds(float s) {
  const float r = __frcp_rn(s);
  const bool plain = fabsf(s) > 0x1p-100f && fabsf(s) < 0x1p100f;
  return plain ? Recip{r * (1.f - 0x1p-21f), r * (1.f + 0x1p-21f)} : Recip{0.f, INFINITY};
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return uint32_t(lo) | (uint32_t(hi) << 16);
}

// The e4m3 codes of x / s (IEEE float32 division) for four values. The rounding
// to a code is monotonic, so where both bounds of the quotient have the same
// code it is that one; the division itself is done where they differ (a
// quotient within 2^-21 of a border between codes, about one in 10^4).
__device__ __forceinline__ uint32_t quotient_codes(const float* x, float s, Recip r) {
  const float2 a = make_float2(x[0], x[1]), b = make_float2(x[2], x[3]);
  const float2 rl = make_float2(r.lo, r.lo), rh = make_float2(r.hi, r.hi);
  const float2 al = mul2(a, rl), bl = mul2(b, rl), ah = mul2(a, rh), bh = mul2(b, rh);
  const uint32_t lo = e4m3x4(al.x, al.y, bl.x, bl.y), hi = e4m3x4(ah.x, ah.y, bh.x, bh.y);
  if (lo == hi) return lo;
  return e4m3x4(__fdiv_rn(x[0], s), __fdiv_rn(x[1], s), __fdiv_rn(x[2], s), __fdiv_rn(x[3], s));
}

// 8 values of one row, channels c .. c + 7 (c a multiple of 8), to codes.
template <int F>
__device__ __forceinline__ void encode8(const float x[8], const float* scale, Recip r, uint8_t* row, int c) {
  if constexpr (F == MJ_KV_E4M3) {
    *reinterpret_cast<uint2*>(row + c) = make_uint2(quotient_codes(x, scale[0], r), quotient_codes(x + 4, scale[0], r));
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
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    memcpy(&w[i], &h, 4);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// F: the cache format; D: channels of a rotated head (queries and keys); VD:
// channels of a value head (the latent vector of mj_latent_write).
//
// A token's elements are `slots` of D channels: its query heads, its key heads
// and VD / D slots a value head. Thread (token, lane, j) takes chunk pair j
// (16 channels) of the slots lane, lane + lanes, ...: always the same eight
// frequencies, whose cosines and sines it holds in registers.
template <int F, int D, int VD>
__global__ void __launch_bounds__(kThreads, kMinCtas) rope_write_kernel(RopeWriteParams p) {
  constexpr int U = kItemsPerThread;
  constexpr int kD = D / 16;   // chunk pairs of a slot
  constexpr int kVS = VD / D;  // slots of a value head
  extern __shared__ __align__(16) float cs[];  // [tokens of the CTA][2][n]: cosines, sines, times the scale
  const int tid = threadIdx.x;
  const int j = tid % kD, lane = (tid / kD) & (p.lanes - 1), tl = tid / (kD * p.lanes);
  const int t0 = blockIdx.x * p.group;
  const int tok = t0 + tl;
  const int slots = p.h_q + p.h_k + p.h_k * kVS;
  const int n_slots = tok < p.num_tokens ? slots : 0;

  // this thread's two 8-channel chunks of a rotated slot, and of a value slot
  const bool rot = 8 * j < p.n;
  const int c0 = rot && !p.interleaved ? 8 * j : 16 * j;
  const int c1 = c0 + (rot && !p.interleaved ? p.n : 8);

  // launched with programmatic stream serialization: everything below may be
  // the preceding kernel's output. The next kernel may launch (and waits for
  // this one where it reads).
  tc::grid_launch_dependents();
  tc::grid_dependency_wait();

  // The n-th slot in the order taken: queries, keys, values; of a latent row
  // (one key, one value head) values, queries, key, as its eight value slots
  // fill a warp's lanes and the key then shares no pass with them (8191 tokens:
  // 14.7 against 16.6 us; 40 tokens of 128 heads 4.1 against 4.4).
  auto slot_at = [&](int n) { return VD == D ? n : (n < kVS ? p.h_q + 1 + n : n - kVS); };
  auto load = [&](int n, uint4& a, uint4& b) {
    const int s = slot_at(n);
    const uint16_t* src;
    int o0 = c0, o1 = c1;
    if (s < p.h_q) {
      src = p.q + tok * p.q_ts + s * p.q_hs;
    } else if (s < p.h_q + p.h_k) {
      src = p.key + tok * p.k_ts + (s - p.h_q) * p.k_hs;
    } else {
      const int v = s - p.h_q - p.h_k;
      src = p.value + tok * p.v_ts + (VD == D ? v * p.v_hs : v * D);
      o0 = 16 * j;
      o1 = o0 + 8;
    }
    a = *reinterpret_cast<const uint4*>(src + o0);
    b = *reinterpret_cast<const uint4*>(src + o1);
  };
  uint4 a[U], b[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (lane + u * p.lanes < n_slots) load(lane + u * p.lanes, a[u], b[u]);
  const int64_t slot = n_slots ? p.slots[tok] : -1;

  for (int e = tid; e < p.group * p.n; e += kThreads) {
    const int el = e / p.n, f = e - el * p.n;
    if (t0 + el >= p.num_tokens) break;
    const int ax = p.axes > 1 ? min(int(p.freq_axis[f]), p.axes - 1) : 0;
    const uint64_t turn = uint64_t(p.pos[int64_t(ax) * p.pos_axis + t0 + el]) * p.turns[f];
    float sn, cn;
    sincospif(float(int32_t(turn >> 32)) * 0x1p-31f, &sn, &cn);
    cs[el * 2 * p.n + f] = cn * p.scale;
    cs[el * 2 * p.n + p.n + f] = sn * p.scale;
  }
  __syncthreads();
  float2 wc[4], ws[4];  // cosines and sines of frequencies 8j + 2k, 8j + 2k + 1
  if (rot && n_slots) {
    const float* wp = cs + tl * 2 * p.n + 8 * j;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float4 c4 = *reinterpret_cast<const float4*>(wp + 4 * k);
      const float4 s4 = *reinterpret_cast<const float4*>(wp + p.n + 4 * k);
      wc[2 * k] = make_float2(c4.x, c4.y);
      wc[2 * k + 1] = make_float2(c4.z, c4.w);
      ws[2 * k] = make_float2(s4.x, s4.y);
      ws[2 * k + 1] = make_float2(s4.z, s4.w);
    }
  }
  if (slot >= p.num_slots && p.status && lane == 0 && j == 0) atomicOr(p.status, kStatusBadPage);
  const bool live = slot >= 0 && slot < p.num_slots;
  const int64_t page = slot >> p.page_shift, prow = slot & ((int64_t(1) << p.page_shift) - 1);

  for (int s0 = lane; s0 < n_slots; s0 += U * p.lanes) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s0 + u * p.lanes >= n_slots) break;
      const int s = slot_at(s0 + u * p.lanes);
      const bool value = s >= p.h_q + p.h_k;
      if (s >= p.h_q && !live) continue;  // a padding token, or a slot past the pool
      float x[8], y[8];
      bf16x8_to_float(a[u], x);
      bf16x8_to_float(b[u], y);
      if (rot && !value) {
        if (p.interleaved) {  // pairs (2k, 2k + 1): x holds the first four of them, y the others
          auto turn = [](float& x0, float& x1, float c, float sn) {
            const float t = x0 * c - x1 * sn;
            x1 = x1 * c + x0 * sn;
            x0 = t;
          };
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            turn(x[4 * k], x[4 * k + 1], wc[k].x, ws[k].x);
            turn(x[4 * k + 2], x[4 * k + 3], wc[k].y, ws[k].y);
            turn(y[4 * k], y[4 * k + 1], wc[k + 2].x, ws[k + 2].x);
            turn(y[4 * k + 2], y[4 * k + 3], wc[k + 2].y, ws[k + 2].y);
          }
        } else {  // pairs (k, k + n)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 x0 = make_float2(x[2 * k], x[2 * k + 1]), y0 = make_float2(y[2 * k], y[2 * k + 1]);
            const float2 xr = fma2(x0, wc[k], mul2(y0, make_float2(-ws[k].x, -ws[k].y)));
            const float2 yr = fma2(y0, wc[k], mul2(x0, ws[k]));
            x[2 * k] = xr.x;
            x[2 * k + 1] = xr.y;
            y[2 * k] = yr.x;
            y[2 * k + 1] = yr.y;
          }
        }
      }
      if (s < p.h_q) {
        uint16_t* dst = p.q_out + tok * p.qo_ts + s * p.qo_hs;
        *reinterpret_cast<uint4*>(dst + c0) = pack_bf16x8(x);
        *reinterpret_cast<uint4*>(dst + c1) = pack_bf16x8(y);
      } else if (!value) {
        const int g = VD == D ? s - p.h_q : 0;
        uint8_t* row = p.k_cache + page * p.k_sp + prow * p.k_st + g * p.k_sh;
        const float* scale = p.k_scale + (F != MJ_KV_E4M3 ? g * D : (p.scale_per_head ? g : 0));
        const Recip r = F == MJ_KV_E4M3 ? recip_bounds(scale[0]) : Recip{};
        encode8<F>(x, scale, r, row, c0);
        encode8<F>(y, scale, r, row, c1);
      } else {
        const int v = s - p.h_q - p.h_k, g = VD == D ? v : 0, c = (VD == D ? 0 : v * D) + 16 * j;
        uint8_t* row = p.v_cache + page * p.v_sp + prow * p.v_st + g * p.v_sh;
        const float* scale = p.v_scale + (F != MJ_KV_E4M3 ? g * D : (p.scale_per_head ? g : 0));
        const Recip r = F == MJ_KV_E4M3 ? recip_bounds(scale[0]) : Recip{};
        encode8<F>(x, scale, r, row, c);
        encode8<F>(y, scale, r, row, c + 8);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = s0 + (U + u) * p.lanes;
      if (s < n_slots) load(s, a[u], b[u]);
    }
  }
}

template <int F, int D, int VD>
cudaError_t launch(RopeWriteParams p, cudaStream_t stream) {
  constexpr int kLanes = kThreads / (D / 16);  // slot lanes of a CTA with one token
  const int64_t slots = int64_t(p.h_q) + p.h_k + int64_t(p.h_k) * (VD / D);
  // Lanes a token: so many that a thread has at most that many slots, up to the
  // CTA's; the CTA takes more tokens where that leaves room.
  auto lanes_for = [&](int per_thread) {
    int lanes = 1;
    while (lanes < kLanes && lanes * per_thread < slots) lanes *= 2;
    return lanes;
  };
  auto ctas = [&] { return (int64_t(p.num_tokens) + p.group - 1) / p.group; };
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
  p.lanes = lanes_for(kItemsPerThread);
  p.group = kLanes / p.lanes;
  if (ctas() > int64_t(kMinCtas) * sms) {
    p.lanes = lanes_for(kItemsMany);
    p.group = kLanes / p.lanes;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas()));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = size_t(p.group) * p.n * 2 * sizeof(float);  // at most 8 KB: 32 tokens of 32 or 8 of 128 frequencies
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
  p.page_shift = page_shift(w.page_size);
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
  p.page_shift = page_shift(a.page_size);
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
