// mj_block_prompt: attention of ragged prompt chunks over the block-scaled cache, on
// the tensor cores.
//
// A CTA takes the query rows (tokens x the heads of one KV head) of one or two
// 128-row tiles of a request and walks their keys once, BN at a time:
//   S = Q K^T     kind::f8f6f4, Q as two e4m3 terms (hi + lo, exact for bf16 down to 2^-9.8
//                 of the row's largest), K as it lies in the cache: 128-byte swizzled by TMA
//   P = 2^(u - m + 6) in fp16, u = t + ev: the weight on V's codes, t = S ck 2^ek, where
//                 2^ek and 2^ev are the scales of the key's block
//   O += P V      kind::f16, P from tensor memory (in place of S), V's codes widened to fp16
//                 (exact) by warps of their own
// so both products run at the 16-bit rate, and a block's scales cost an addition
// and a product per 16 keys and row. m is the row's running reference of u: it moves
// only where a tile's largest u is more than 8 above it (P stays below 2^14 + 1), and
// O, kept in tensor memory, is rescaled then. Weights keep 11 bits down to 20 binades
// below the reference, and lose less than 2^-31 of it each below. The sum l wants 2^t: P's float32
// times 2^-ev.
//
// Head size 128: two row tiles (256 rows), 128 keys a step; tensor memory is full (two S and two
// O), so a tile's next scores wait for its weights' product, and the other tile's
// products fill that time. One row tile (head size 256, or 128 rows and fewer): two S
// buffers, Q in tensor memory, 64 keys a step at head size 256. At most 32 rows, as a decode
// of more query rows than the decode kernel takes: SPREAD, below.
//
// What bounds it. 4096 tokens after 12288, 32/8 heads: 727 us, 1320 TFLOP/s, 67% of the
// measured bf16 rate: a row tile's chain, 3100 cycles a step where both tiles' products take
// 2050 (clock stamps: softmax 1500 - scores read 60, largest u 400, exponentials 1000 -, products of the
// weights 700, scores 580, from their end to the softmax 350). One row tile: 1400 to 1900 cycles a step where
// the products take 1024: softmax 900, and a step's barriers in the MMA warp. Short chunks (5 of 20 to 700
// tokens, head size 256: 45 us): the CTA's ends, 12000 cycles to the first scores, 5000 to write the rows.
// 64 x 4096 cached tokens, 16 and 32 rows: 134 and 136 us in pages of 32 (4.0 TB/s), 155 and 157 in pages of 16.
//
// What it took (the long chunk, us): four products at an election, their barriers waited for a step
// ahead 864 -> 808; scores read once into registers instead of twice 1040 -> 864; Q split by twelve
// warps and rows written whole 790 -> 735; one arrival a warp instead of one a thread, one
// barrier for all that a step frees 735 -> 727.
// Not kept: 64 keys a step with two S buffers a tile (980: at 64 columns the scores' operands
// bound shared memory), the same with Q in tensor memory and one buffer (977), two
// threads a row (940), a step's waits between the products (756).
//
// Warps: 0 TMA, 1 MMA, 2 the blocks' scales, then softmax (a thread a row) and the
// warps that widen V. Every wait is bounded (2 s): a timeout sets a status bit, and the CTA
// drains its copies and products, frees its tensor memory and returns.
#include <atomic>
#include <type_traits>

#include "latent_ptx.cuh"
#include "mj_block.h"
#include "mj_device.cuh"

namespace mj {

namespace {

constexpr uint64_t kWaitNs = 2000000000ull, kDrainNs = 100000000ull;
constexpr float kTau = 8.f, kLift = 6.f;  // log2 units
constexpr int kKStages = 4;              // (a multiple of V's two: the MMA loop's period)
constexpr int kTile = 16384;              // bytes: 128 rows of 128, and a K or V tile

// Row tiles of 128: head size 128 has two where a CTA has that many rows, else one.
template <int D, int NT_>
struct Cfg {
  static constexpr int NT = NT_;
  static constexpr int BN = D == 128 ? 128 : 64;
  static constexpr int DH = D / 128;
  static constexpr int NB = BN / 16;            // 16-key groups of a tile
  static constexpr int TB = 32 / NB;            // tiles a batch of scales covers
  // warps: 0 TMA, 1 MMA, 2 the blocks' scales, 4 .. softmax, then the ones that widen V
  static constexpr int kConvWarp0 = 4 + 4 * NT, kConvWarps = 16 - kConvWarp0, kThreads = 512;
  static constexpr int kRows = 128 * NT;
  // Tensor memory: S (and P) buffers of BN columns from 0; with one row tile Q's terms behind them
  // (D / 4 columns each), so that the scores' product reads shared memory for K alone; O
  static constexpr bool kQt = NT == 1;
  static constexpr uint32_t kQcol = 2 * BN, kO = NT == 1 && D == 128 ? 384 : 256;
  static_assert(!kQt || (kQcol + D / 2 <= kO && kO + D <= 512), "tensor memory");
  // widened V tiles: with one row tile there is room for four, and the warps that widen run ahead
  static constexpr int kVStages = NT == 1 ? 4 : 2;
  static constexpr int kQ = kQt ? 0 : NT * 2 * DH * kTile;
  static constexpr int kK = kQ, kVr = kK + kKStages * kTile, kVf = kVr + 2 * kTile, kCtrl = kVf + kVStages * 2 * kTile;
  static constexpr int kBytes = kCtrl + 2048;
  static_assert(NT > 1 || 4 * D * 32 * 4 + 1024 <= kCtrl, "the copies' join");
};
static_assert(Cfg<128, 2>::kBytes + 1024 <= 227 * 1024 && Cfg<256, 1>::kBytes + 1024 <= 227 * 1024 && kKStages % 2 == 0,
              "shared memory");

struct Ctrl {
  uint64_t k_full[kKStages];
  uint64_t vr_full[2], vr_empty[2], vf_full[4];
  uint64_t s_full[2], p_full[2][2];  // (P in halves of its keys)
  uint64_t done[4];  // of step i modulo 4: tile i's products on V, and tile i + 1's scores
  uint64_t e_full[2], e_empty[2];
  uint64_t q_ready, drain, o_last[2];  // o_last: a row tile's last product
  uint32_t tmem;
  int abort;
  uint8_t q_exp[256];  // the rows' exponents
  alignas(16) float4 scale[2][32];  // batches of TB tiles: 2^ek, ev, 2^-ev of each 16-key group
};
static_assert(sizeof(Ctrl) <= 2048, "control block");

// The two products, four instructions at a time, called by a converged warp: one elected
// lane issues (the same each time). A descriptor's upper half is constant; offsets are
// added here. (One election for four: elected one by one the products were issued
// 43 cycles apart, and the issue bounded the kernel.)
// D[tmem] (+)= A[smem desc] B[smem desc], e4m3: 128 channels, 32 bytes of the rows a step.
__device__ __forceinline__ void umma_qk4(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 w, x, y, z, a0, a1, a2, a3;\n\t.reg .b32 t, u, v, r, s, q;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "add.u32 t, %2, 2;\n\tadd.u32 u, %2, 4;\n\tadd.u32 v, %2, 6;\n\tadd.u32 r, %1, 2;\n\tadd.u32 s, %1, 4;\n\t"
      "add.u32 q, %1, 6;\n\tmov.b64 w, {%2, %3};\n\tmov.b64 x, {t, %3};\n\tmov.b64 y, {u, %3};\n\tmov.b64 z, {v, %3};\n\t"
      "mov.b64 a0, {%1, %3};\n\tmov.b64 a1, {r, %3};\n\tmov.b64 a2, {s, %3};\n\tmov.b64 a3, {q, %3};\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a0, w, %4, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, x, %4, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, y, %4, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, z, %4, 1;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// D[tmem] (+)= A[tmem] B[smem desc], e4m3: 128 channels, 8 columns of A and 32 bytes of B's rows a step.
__device__ __forceinline__ void umma_qk4_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 w, x, y, z;\n\t.reg .b32 t, u, v, a1, a2, a3;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "add.u32 t, %2, 2;\n\tadd.u32 u, %2, 4;\n\tadd.u32 v, %2, 6;\n\tadd.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\t"
      "add.u32 a3, %1, 24;\n\tmov.b64 w, {%2, %3};\n\tmov.b64 x, {t, %3};\n\tmov.b64 y, {u, %3};\n\tmov.b64 z, {v, %3};\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], w, %4, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [a1], x, %4, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [a2], y, %4, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [a3], z, %4, 1;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// D[tmem] (+)= A[tmem] B[smem desc], fp16: 64 keys, 8 columns of A and 16 rows of B a step.
__device__ __forceinline__ void umma_pv4(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 w, x, y, z;\n\t.reg .b32 t, u, v, a1, a2, a3;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "add.u32 t, %2, 128;\n\tadd.u32 u, %2, 256;\n\tadd.u32 v, %2, 384;\n\tadd.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\t"
      "add.u32 a3, %1, 24;\n\tmov.b64 w, {%2, %3};\n\tmov.b64 x, {t, %3};\n\tmov.b64 y, {u, %3};\n\tmov.b64 z, {v, %3};\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], w, %4, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], x, %4, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], y, %4, 1;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], z, %4, 1;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of kind::f16 with fp16 A (K-major) and B (MN-major), f32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | (1u << 16) | (uint32_t(N >> 3) << 17) | (uint32_t(M >> 4) << 24);
}

__device__ __forceinline__ void tmem_ld32(uint32_t at, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
}

__device__ __forceinline__ void tmem_ld16u(uint32_t at, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at));
}

// Wait for the thread's TMEM loads; N of the values pass through, so that nothing uses them earlier.
template <int N>
__device__ __forceinline__ void tmem_wait_ld(uint32_t* r) {
  static_assert(N == 16 || N == 32, "values");
  if constexpr (N == 32)
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                   "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                   "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
  else
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}

// The same without the wait: for loads that an earlier wait covers.
__device__ __forceinline__ void tmem_pass32(uint32_t* r) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}

template <int N>
__device__ __forceinline__ void tmem_st(uint32_t at, const uint32_t* r) {
  static_assert(N == 8 || N == 16, "columns");
  if constexpr (N == 16)
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
  else
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(at), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// As tc::mbar_wait, with naps of NAP ns between the looks: most warps here wait most of
// the time, and their polls take issue slots and shared memory from those that work.
template <int NAP>
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (tc::mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = 0;
  for (uint32_t it = 0;; ++it) {
    if constexpr (NAP > 0) __nanosleep(NAP);
    if (tc::mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) != 63u) continue;
    if (*abort) return false;
    const uint64_t now = tc::globaltimer_ns();
    if (t0 == 0) {
      t0 = now;
    } else if (now - t0 > kWaitNs) {
      *abort = 1;
      return false;
    }
  }
}

// This warpgroup's registers a thread from here on.
template <bool MORE, int N>
__device__ __forceinline__ void set_regs() {
  if constexpr (MORE)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// two float32 at once: a * b + c
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 w, x, y;\n\t"
      "mov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
// the largest of three (NaN does not count)
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// lo and hi to fp16, packed
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// lo and hi to bf16, packed
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// two e4m3 codes to fp16, exactly
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\t}" : "=r"(r) : "r"(two));
  return r;
}

// x (two fp16) = hi + lo, two e4m3 codes each
__device__ __forceinline__ void split_e4m3(uint32_t x, uint32_t& hi, uint32_t& lo) {
  asm("{\n\t.reg .b16 h, l;\n\t.reg .b32 y;\n\tcvt.rn.satfinite.e4m3x2.f16x2 h, %2;\n\tcvt.rn.f16x2.e4m3x2 y, h;\n\t"
      "sub.rn.f16x2 y, %2, y;\n\tcvt.rn.satfinite.e4m3x2.f16x2 l, y;\n\tcvt.u32.u16 %0, h;\n\tcvt.u32.u16 %1, l;\n\t}"
      : "=r"(hi), "=r"(lo)
      : "r"(x));
}

template <int D, int NT, bool SPREAD>
__global__ void __launch_bounds__(512, 1)
    block_prompt_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                        BlockPromptParams p) {
  using C = Cfg<D, NT>;
  constexpr int BN = C::BN, DH = C::DH, NB = C::NB, TB = C::TB, NV = C::kVStages;
  // With at most 32 rows (SPREAD) the row tile holds them four times, once for each softmax warp
  // (a warp reaches 32 of the tile's rows), and a copy takes a quarter of a tile's keys: its P is 0
  // for the others. Each copy has a reference, a sum and an output of its own; they are joined
  // at the end, as pieces of the keys are. (64 x 4096 tokens, 16 rows: 163 -> 139 us when it was added.)
  static_assert(!SPREAD || NT == 1, "one row tile");
  constexpr int kHalves = BN == 128 && !SPREAD ? 2 : 1;  // P is handed over in halves of its keys
  constexpr int HC = SPREAD ? BN / 4 : BN, HB = HC / 16;  // columns (keys) of a softmax thread, 16-key groups
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // (32-bit shared addresses throughout, from constants: what the products are issued with stays in uniform registers)
  const uint32_t raw = tc::smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  Ctrl& ctl = *reinterpret_cast<Ctrl*>(smem + C::kCtrl);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto bar = [&](uint64_t& b) {
    return base + uint32_t(C::kCtrl) + uint32_t(reinterpret_cast<char*>(&b) - reinterpret_cast<char*>(&ctl));
  };

  tc::grid_dependency_wait();
  // The CTA's rows r0 .. of request b and KV head g, the request's first query token t0 of n, and
  // its keys: k0 .. k_end - 1, nt tiles. parts: where the rows' partials begin (-1: there is one piece).
  int b, g, t0, n, rows, r0, L, k0, k_end;
  int64_t parts = -1;
  if (p.work) {
    // decode: work row and KV head, row tile
    g = int(blockIdx.x % unsigned(p.h_k));
    const int4 w = p.work[blockIdx.x / unsigned(p.h_k)];
    if (w.z <= w.y || w.x < 0 || w.x >= p.num_seqs) return;
    b = w.x;
    const int4 rq = p.req[b];  // first partial, pieces, tiles a piece, tiles planned
    L = p.seq_lens[b];
    const bool bad = w.y < 0 || w.w < 0 || w.w >= rq.y || !plan_entry_ok(rq.x, rq.y, rq.z, p.part_cap);
    if (tid == 0 && bad) atomicOr(p.status, kStatusBadPlan);
    n = p.max_q_len;
    t0 = b * n;
    rows = n * p.h_r;
    r0 = int(blockIdx.y) * C::kRows;
    if (bad || L <= int64_t(w.y) * kKvTile) return;  // (a piece without keys: the join does not count it)
    k0 = w.y * kKvTile;
    k_end = int(min(int64_t(L), int64_t(w.z) * kKvTile));
    if (rq.y > 1) parts = ((int64_t(rq.x) + w.w) * p.h_k + g) * rows;
  } else {
    // prompt: KV head and piece, row tiles from the last one on (with a causal limit the longest), request
    const int piece = int(blockIdx.x) % p.splits;
    g = int(blockIdx.x) / p.splits;
    b = blockIdx.z;
    t0 = max(0, p.q_starts[b]);
    n = p.q_starts[b + 1] - t0;
    const int held = max(0, min(n, p.num_tokens - t0));  // that are rows of q
    rows = min(held, p.max_q_len) * p.h_r;
    const int row_tiles = (rows + C::kRows - 1) / C::kRows;
    if (n > min(held, p.max_q_len) && blockIdx.x == 0 && blockIdx.y == 0) {
      if (tid == 0) atomicOr(p.status, kStatusBadPlan);
      if (p.splits > 1)  // the join passes these rows by
        for (int64_t i = tid; i < int64_t(held - p.max_q_len) * p.h_q; i += C::kThreads)
          p.l_part[(int64_t(t0) + p.max_q_len) * p.h_q + i] = -1.f;
    }
    if (int(blockIdx.y) >= row_tiles) return;
    r0 = (row_tiles - 1 - int(blockIdx.y)) * C::kRows;
    L = p.seq_lens[b];
    // this piece of the tiles up to the last key that any of the rows sees
    const int last = min(L - 1, p.causal ? L - n + (min(rows, r0 + C::kRows) - 1) / p.h_r : L - 1);
    const int tiles = last >= 0 ? last / BN + 1 : 0;
    const int each = (tiles + p.splits - 1) / p.splits;
    k0 = min(tiles, piece * each) * BN;
    k_end = min(L, min(tiles, (piece + 1) * each) * BN);
    if (p.splits > 1) parts = (int64_t(piece) * p.num_tokens + t0) * p.h_q;
  }
  if (r0 >= rows) return;
  if (p.causal) k_end = min(k_end, L - n + (min(rows, r0 + C::kRows) - 1) / p.h_r + 1);
  const int nt = k_end > k0 ? (k_end - k0 + BN - 1) / BN : 0;

  if (tid == 0) {
    for (int s = 0; s < kKStages; ++s) tc::mbar_init(bar(ctl.k_full[s]), 1);
    for (int s = 0; s < 4; ++s) {
      tc::mbar_init(bar(ctl.done[s]), 1);
      tc::mbar_init(bar(ctl.vf_full[s]), C::kConvWarps);
    }
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(bar(ctl.vr_full[s]), 1);
      tc::mbar_init(bar(ctl.vr_empty[s]), C::kConvWarps);
      tc::mbar_init(bar(ctl.s_full[s]), 1);
      for (int h = 0; h < 2; ++h) tc::mbar_init(bar(ctl.p_full[s][h]), 4);
      tc::mbar_init(bar(ctl.o_last[s]), 1);
      tc::mbar_init(bar(ctl.e_full[s]), 1);
      tc::mbar_init(bar(ctl.e_empty[s]), 4 * NT);
    }
    tc::mbar_init(bar(ctl.q_ready), 128 * NT);
    tc::mbar_init(bar(ctl.drain), 1);
    ctl.abort = 0;
    tc::fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tc::prefetch_tmap(&tmap_k);
    tc::prefetch_tmap(&tmap_v);
  }
  if (warp == 1) {
    tc::tmem_alloc(tc::smem_u32(&ctl.tmem), 512);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  constexpr uint32_t tmem = 0;  // all 512 columns: the allocation begins at 0
  volatile int* abort = &ctl.abort;

  // Q's rows, by the twelve warps that have nothing else to do yet, 8 channels a lane: x' = x *
  // 2^(127 - e), the row's largest finite |x'| in (224, 448]; hi = e4m3(x'), lo = e4m3(x' - hi). x' goes
  // through fp16: it keeps x' of 2^-17 and more exactly, and less gives code 0 either way. (By the softmax
  // threads, each its own row, this took 12000 cycles a CTA at head size 256, now 9000.)
  if (warp >= 4) {
    constexpr int kRowLanes = D / 8, kRowsLd = 32 / kRowLanes, kMine = SPREAD ? 32 : C::kRows;
    const int j0 = (warp - 4) * kRowsLd + lane / kRowLanes, ch = lane % kRowLanes * 8;
    // The rows as they are, all on their way at once, to where V's first tiles are widened to later; a
    // thread reads back what it copied. (Short loops: a CTA of the first wave waits for its code, too.)
    const uint32_t in = base + uint32_t(C::kVf + lane % kRowLanes * 16);
    {
      // a row's token and head, from the CTA's first row's (exact: rem + j is far below 2^21)
      const int tq = r0 / p.h_r, rem = r0 - tq * p.h_r;
      const float recip = 1.f / float(p.h_r);
#pragma unroll 4
      for (int j = j0; j < kMine; j += 12 * kRowsLd) {
        const int dt = int((float(rem + j) + 0.5f) * recip);
        const bool real = r0 + j < rows;
        const uint16_t* src = p.q + ch;
        if (real) src += int64_t(t0 + tq + dt) * p.q_ts + (int64_t(g) * p.h_r + (rem + j - dt * p.h_r)) * p.q_hs;
        tc::cp_async16(in + uint32_t(j * (2 * D)), src, real ? 16u : 0u);
      }
    }
    tc::cp_async_wait_all();
    // (four rows abreast: one row's shuffles and conversions are a chain of 600 cycles)
    constexpr int kAbreast = SPREAD ? 3 : 4;
#pragma unroll 1
    for (int jj = j0; jj < kMine; jj += 12 * kRowsLd * kAbreast) {
      uint32_t w[kAbreast][4], am[kAbreast], odd[kAbreast];
#pragma unroll
      for (int u = 0; u < kAbreast; ++u) {
        const int j = jj + u * 12 * kRowsLd < kMine ? jj + u * 12 * kRowsLd : jj;  // (past the end: not written)
        const uint4 v = *reinterpret_cast<const uint4*>(smem + C::kVf + lane % kRowLanes * 16 + j * (2 * D));
        w[u][0] = v.x;
        w[u][1] = v.y;
        w[u][2] = v.z;
        w[u][3] = v.w;
      }
      auto largest = [&] {
#pragma unroll
        for (int u = 0; u < kAbreast; ++u) {
          uint32_t m = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) m = __vmaxu2(m, w[u][k] & 0x7FFF7FFFu);
          am[u] = max(m & 0xFFFFu, m >> 16);
        }
#pragma unroll
        for (int o = kRowLanes / 2; o > 0; o >>= 1)
#pragma unroll
          for (int u = 0; u < kAbreast; ++u) am[u] = max(am[u], __shfl_xor_sync(~0u, am[u], o));
      };
      largest();
      uint32_t any = 0;
#pragma unroll
      for (int u = 0; u < kAbreast; ++u) {
        any = max(any, am[u]);
        odd[u] = 0;
      }
      if (__any_sync(~0u, any >= 0x7F80u)) {  // infinities or NaN: NaN codes; they do not count above
#pragma unroll
        for (int u = 0; u < kAbreast; ++u)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if ((w[u][k] & 0x7FFFu) >= 0x7F80u) {
              w[u][k] &= 0xFFFF0000u;
              odd[u] |= 1u << (2 * k);
            }
            if ((w[u][k] & 0x7FFF0000u) >= 0x7F800000u) {
              w[u][k] &= 0xFFFFu;
              odd[u] |= 2u << (2 * k);
            }
          }
        largest();
      }
      __syncwarp();  // (in place: the rows have been read)
#pragma unroll
      for (int u = 0; u < kAbreast; ++u) {
        const int j = jj + u * 12 * kRowsLd;
        const int e = max(1, int(((am[u] << 16) + 0x1FFFFFu) >> 23) - 8);
        const float inv = __int_as_float((254 - e) << 23);
        uint32_t hw[4], lw[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          split_e4m3(f16x2(__uint_as_float(w[u][k] << 16) * inv, __uint_as_float(w[u][k] & 0xFFFF0000u) * inv), hw[k], lw[k]);
        uint2 hi = make_uint2(__byte_perm(hw[0], hw[1], 0x5410), __byte_perm(hw[2], hw[3], 0x5410));
        const uint2 lo = make_uint2(__byte_perm(lw[0], lw[1], 0x5410), __byte_perm(lw[2], lw[3], 0x5410));
        if (odd[u]) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (odd[u] >> k & 1u) hi.x |= 0x7Fu << (8 * k);
            if (odd[u] >> (k + 4) & 1u) hi.y |= 0x7Fu << (8 * k);
          }
        }
        if (j >= kMine) break;
        // One row tile: [row][hi, lo] in place, on their way to tensor memory. 16-byte pieces
        // swizzled by the row in both places.
        uint8_t* at = smem + (C::kQt ? C::kVf + j * (2 * D) : (j >> 7) * (2 * kTile) + (j & 127) * 128) +
                      (((ch >> 4) ^ (j & 7)) << 4) + (ch & 8);
        *reinterpret_cast<uint2*>(at) = hi;
        *reinterpret_cast<uint2*>(at + (C::kQt ? D : kTile)) = lo;
        if (ch == 0) ctl.q_exp[j] = uint8_t(e);
      }
    }
    if constexpr (!C::kQt) tc::fence_async_smem();
    tc::named_bar_sync(1, 384);
  }

  // Registers: 128 a thread at launch. At head size 128 (without copies) a softmax thread keeps a row's 128
  // scores: 2 x 192 + 2 x 64, or 224 + 3 x 96, = 4 x 128 for the four warpgroups.
  if (warp >= 4 && warp < C::kConvWarp0) {
    if constexpr (D == 128 && !SPREAD) set_regs<true, NT == 2 ? 192 : 224>();
    // ======================= softmax: thread = row ============================
    const int a = (warp - 4) >> 2, quad = warp & 3;
    const int R = SPREAD ? r0 + lane : r0 + 128 * a + 32 * quad + lane;
    const int col = SPREAD ? quad * HC : 0;  // the thread's first column
    const bool real = R < rows;
    const int64_t tok = t0 + int64_t(real ? R / p.h_r : 0), head = int64_t(g) * p.h_r + (real ? R % p.h_r : 0);
    const uint32_t lanes = uint32_t(32 * quad) << 16;
    float ck;  // logits (log2 units) = S * ck * 2^ek
    {
      const uint8_t* qs = smem + C::kVf + (SPREAD ? 0 : quad * (64 * D));
      // (not below 2^-94: ck 2^ek stays above 0, and a hidden key's -inf times it -inf. |S| is below 2^26, so that
      // the logits of a smaller ck are within 2^-36 of 0 either way)
      ck = fmaxf(__int_as_float(int(ctl.q_exp[SPREAD ? lane : 32 * (warp - 4) + lane]) << 23) * p.scale_log2, 0x1p-94f);
      if constexpr (C::kQt) {
#pragma unroll 4
        for (int c = 0; c < 2 * D / 64; ++c) {  // 64 codes: of hi, then of lo
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4 u = *reinterpret_cast<const uint4*>(qs + lane * (2 * D) + (((4 * c + k) ^ (lane & 7)) << 4));
            w[4 * k] = u.x;
            w[4 * k + 1] = u.y;
            w[4 * k + 2] = u.z;
            w[4 * k + 3] = u.w;
          }
          tmem_st<16>(tmem + lanes + C::kQcol + uint32_t(16 * c), w);
        }
        tc::tmem_wait_st();
        tc::tc_fence_before();
      }
      tc::mbar_arrive(bar(ctl.q_ready));
    }
    // The last key this row sees (a row past the end computes something that nobody reads).
    // The first `open` tiles hide nothing from the warp's rows: their code has no
    // masks (as selects or predicated they would cost every tile).
    const int lim = real && p.causal ? min(k_end - 1, L - n + R / p.h_r) : k_end - 1;
    const int open = max(0, __reduce_min_sync(~0u, lim + 1 - k0)) / BN;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    // one tile; false: give up
    auto tile = [&](auto with_mask, int i) -> bool {
      constexpr bool masked = decltype(with_mask)::value;
      const int buf = NT == 2 ? a : (i & 1);
      const uint32_t tS = tmem + lanes + uint32_t(buf * BN);
      const int bat = i / TB;
      if (i % TB == 0) ok = wait_bar<0>(bar(ctl.e_full[bat & 1]), uint32_t(bat >> 1) & 1u, abort);
      // the groups' scales, before the scores are there: the products' operands keep
      // shared memory busy, and a load from it in the middle of the arithmetic would take long
      float4 sc[HB];
#pragma unroll
      for (int h = 0; h < HB; ++h) {
        sc[h] = ctl.scale[bat & 1][(i % TB) * NB + (SPREAD ? quad * HB : 0) + h];
        sc[h].x *= ck;
      }
      ok = ok && wait_bar<0>(bar(ctl.s_full[buf]), uint32_t(NT == 2 ? i : i >> 1) & 1u, abort);
      ok = __all_sync(~0u, ok);
      if (!ok) return false;
      tc::tc_fence_after();
      // column c of the thread's is hidden from c = seen on
      const int seen = lim - (k0 + i * BN + col) + 1;

      // the tile's largest u
      uint32_t r[HC];
      if constexpr (HC == 16) {
        tmem_ld16u(tS + col, r);
        tmem_wait_ld<16>(r);
      } else {
#pragma unroll
        for (int c = 0; c < HC; c += 32) tmem_ld32(tS + col + c, r + c);
        tmem_wait_ld<32>(r);
#pragma unroll
        for (int c = 32; c < HC; c += 32) tmem_pass32(r + c);
      }
      if constexpr (masked) {
#pragma unroll
        for (int k = 0; k < HC; ++k)
          if (k >= seen) r[k] = 0xFF800000u;
      }
      float t[HB];
#pragma unroll
      for (int h = 0; h < HB; ++h) {
        const uint32_t* x = r + 16 * h;
        float mx = __uint_as_float(x[0]), my = __uint_as_float(x[1]);
#pragma unroll
        for (int k = 2; k < 14; k += 4) {
          mx = max3(mx, __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
          my = max3(my, __uint_as_float(x[k + 2]), __uint_as_float(x[k + 3]));
        }
        mx = fmaxf(max3(mx, __uint_as_float(x[14]), __uint_as_float(x[15])), my);
        t[h] = fmaf(mx, sc[h].x, sc[h].y);
      }
      float top = t[0];
      if constexpr (HB == 2) top = fmaxf(t[0], t[1]);
      if constexpr (HB >= 4) top = fmaxf(max3(t[0], t[1], t[2]), t[3]);
      if constexpr (HB == 8) top = max3(top, max3(t[4], t[5], t[6]), t[7]);
      // the reference
      float by = 1.f;
      bool move = false;
      if (top > m + kTau) {
        by = fast_exp2(m - top);
        move = m != -INFINITY;
        m = top;
        l *= by;
      }
      if (__any_sync(~0u, move)) {
        // O holds the products up to tile i - 1: rescale it before this tile's. (With two row
        // tiles this tile's scores were issued behind the last of them. With one they
        // were issued before it.)
        if constexpr (NT == 1) {
          ok = __all_sync(~0u, wait_bar<0>(bar(ctl.done[(i - 1) & 3]), uint32_t((i - 1) >> 2) & 1u, abort));
          if (!ok) return false;
          tc::tc_fence_after();
        }
        const uint32_t tO = tmem + lanes + C::kO + uint32_t(a * D);
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          uint32_t v[16];
          tmem_ld16u(tO + c, v);
          tmem_wait_ld<16>(v);
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * by);
          tmem_st<16>(tO + c, v);
        }
      }
      // P in place of S, 32 keys at a time; a group's sums and stores come behind the
      // exponentials of the next, which do not wait for them
      const float lift = kLift - (m == -INFINITY ? 0.f : m);
      auto exps = [&](int h) {  // of 16 keys
        const float4 e = sc[h];
        const float2 mul = make_float2(e.x, e.x), add = make_float2(e.y + lift, e.y + lift);
#pragma unroll
        for (int k = 16 * h; k < 16 * h + 16; k += 2) {
          const float2 u = fma2(make_float2(__uint_as_float(r[k]), __uint_as_float(r[k + 1])), mul, add);
          r[k] = __float_as_uint(fast_exp2(u.x));
          r[k + 1] = __float_as_uint(fast_exp2(u.y));
        }
      };
      auto pack = [&](int h, uint32_t* w) {
        float2 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          x[k] = make_float2(__uint_as_float(r[16 * h + 2 * k]), __uint_as_float(r[16 * h + 2 * k + 1]));
          w[k] = f16x2(x[k].x, x[k].y);
        }
#pragma unroll
        for (int d = 4; d > 0; d >>= 1)
#pragma unroll
          for (int k = 0; k < d; ++k) x[k] = add2(x[k], x[k + d]);
        l = fmaf(x[0].x + x[0].y, sc[h].z, l);
      };
      auto give = [&](int h) {
        tc::tmem_wait_st();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(ctl.p_full[buf][h]));
      };
      if constexpr (SPREAD) {
        uint32_t w[HC / 2];
        uint32_t none[HC / 2];
#pragma unroll
        for (int k = 0; k < HC / 2; ++k) none[k] = 0u;
#pragma unroll
        for (int h = 0; h < HB; ++h) exps(h);
#pragma unroll
        for (int h = 0; h < HB; ++h) pack(h, w + 8 * h);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k == quad)
            tmem_st<HC / 2>(tS + k * (HC / 2), w);
          else
            tmem_st<HC / 2>(tS + k * (HC / 2), none);
        }
        give(0);
      } else {
        auto store = [&](int c) {
          uint32_t w[16];
          pack(2 * c, w);
          pack(2 * c + 1, w + 8);
          tmem_st<16>(tS + 16 * c, w);
          if constexpr (kHalves == 2) {
            if (c & 1) give(c >> 1);
          } else {
            if (c == BN / 32 - 1) give(0);
          }
        };
        exps(0);
        exps(1);
#pragma unroll
        for (int c = 1; c < BN / 32; ++c) {
          exps(2 * c);
          exps(2 * c + 1);
          store(c - 1);
        }
        store(BN / 32 - 1);
      }
      if (i % TB == TB - 1 || i == nt - 1) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(ctl.e_empty[bat & 1]));
      }
      return true;
    };
    {
      int i = 0;
      bool go = true;
      for (; i < min(open, nt) && go; ++i) go = tile(std::false_type{}, i);
      for (; i < nt && go; ++i) go = tile(std::true_type{}, i);
    }
    if (nt > 0) ok = ok && wait_bar<0>(bar(ctl.o_last[a]), 0, abort);
    ok = __all_sync(~0u, ok);
    tc::tc_fence_after();
    if constexpr (SPREAD) {
      // Join the copies in shared memory, whose tiles are consumed by now: [copy][channel][row].
      // (All four warps come here whatever happened.)
      float* all = reinterpret_cast<float*>(smem);
      float2* ml = reinterpret_cast<float2*>(all + 4 * D * 32);
      ml[32 * quad + lane] = ok ? make_float2(m, l) : make_float2(-INFINITY, 0.f);
      tc::named_bar_sync(2, 128);
      float M = -INFINITY, sum = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) M = fmaxf(M, ml[32 * k + lane].x);
      const float top = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int k = 0; k < 4; ++k) sum = fmaf(fast_exp2(ml[32 * k + lane].x - top), ml[32 * k + lane].y, sum);
      const float f = fast_exp2(m - top);
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t r[32];
        if (ok && nt > 0) {
          tmem_ld32(tmem + lanes + C::kO + uint32_t(c), r);
          tmem_wait_ld<32>(r);
        }
#pragma unroll
        for (int k = 0; k < 32; ++k) all[(quad * D + c + k) * 32 + lane] = nt > 0 ? __uint_as_float(r[k]) * f : 0.f;
      }
      tc::named_bar_sync(2, 128);
      m = M;
      l = sum;
    }
    if (ok) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const bool some = nt > 0 && !(l == 0.f);
      // the row's place in its partials and in the LSE
      const int64_t part = parts + (p.work ? R : (tok - t0) * p.h_q + head);
      auto out2 = [&](float x, float y) {  // (0 for a row that sees nothing)
        return some ? (p.out_f16 ? f16x2(x, y) : bf16x2(x, y)) : 0u;
      };
      const int64_t lse_at = p.work ? (int64_t(b) * p.h_k + g) * rows + R : tok * p.h_q + head;
      if constexpr (SPREAD) {  // each thread writes a quarter of the row
        const float* all = reinterpret_cast<const float*>(smem) + lane;
#pragma unroll 1
        for (int c = quad * (D / 4); c < (quad + 1) * (D / 4); c += 32) {
          float o[32];
#pragma unroll
          for (int k = 0; k < 32; ++k)
            o[k] = ((all[(c + k) * 32] + all[(D + c + k) * 32]) + (all[(2 * D + c + k) * 32] + all[(3 * D + c + k) * 32])) * inv;
          if (!real) continue;
          if (parts >= 0) {
            if (!some) continue;
            float4* dst = reinterpret_cast<float4*>(p.o_part + part * D + c);
#pragma unroll
            for (int k = 0; k < 32; k += 4) dst[k / 4] = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
          } else {
            uint4* dst = reinterpret_cast<uint4*>(p.out + tok * p.out_ts + head * p.out_hs + c);
#pragma unroll
            for (int k = 0; k < 32; k += 8)
              dst[k / 8] = make_uint4(out2(o[k], o[k + 1]), out2(o[k + 2], o[k + 3]), out2(o[k + 4], o[k + 5]), out2(o[k + 6], o[k + 7]));
          }
        }
      } else {
        // Through shared memory, whose tiles are consumed by now, so that a warp writes whole rows (a
        // thread writing its own, 32 lines a store, took 6500 cycles a CTA at head size 256). 512 bytes
        // of a row at most, its 16-byte pieces swizzled by the row.
        uint8_t* st = smem + C::kK + (warp - 4) * (32 * 512);
        const int64_t at = parts >= 0 ? part * D : tok * p.out_ts + head * p.out_hs;  // where the row begins
        const unsigned wanted = __ballot_sync(~0u, real && (some || parts < 0));
        auto rows_out = [&](auto partial) {
          constexpr bool f32 = decltype(partial)::value;
          constexpr int kCh = f32 ? 128 : D, kPieces = kCh * (f32 ? 4 : 2) / 16, kRowsSt = 32 / kPieces;
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += kCh) {
#pragma unroll 1
            for (int c = c0; c < c0 + kCh; c += 64) {
              uint32_t r[64];
              if (nt > 0) {
                tmem_ld32(tmem + lanes + C::kO + uint32_t(a * D + c), r);
                tmem_ld32(tmem + lanes + C::kO + uint32_t(a * D + c + 32), r + 32);
                tmem_wait_ld<32>(r);
                tmem_pass32(r + 32);
              }
              float o[64];
#pragma unroll
              for (int k = 0; k < 64; ++k) o[k] = __uint_as_float(r[k]) * inv;
              constexpr int kPer = f32 ? 4 : 8;  // channels a piece
#pragma unroll
              for (int k = 0; k < 64; k += kPer) {
                uint4 v;
                if constexpr (f32)
                  v = make_uint4(__float_as_uint(o[k]), __float_as_uint(o[k + 1]), __float_as_uint(o[k + 2]), __float_as_uint(o[k + 3]));
                else
                  v = make_uint4(out2(o[k], o[k + 1]), out2(o[k + 2], o[k + 3]), out2(o[k + 4], o[k + 5]), out2(o[k + 6], o[k + 7]));
                *reinterpret_cast<uint4*>(st + lane * 512 + ((((c - c0 + k) / kPer) ^ (lane & 7)) << 4)) = v;
              }
            }
            __syncwarp();
#pragma unroll 8
            for (int j0 = 0; j0 < 32; j0 += kRowsSt) {
              const int j = j0 + lane / kPieces, pc = lane % kPieces;
              const int64_t to = __shfl_sync(~0u, at, j) + c0;
              const uint4 v = *reinterpret_cast<const uint4*>(st + j * 512 + ((pc ^ (j & 7)) << 4));
              if (!(wanted >> j & 1u)) continue;
              if constexpr (f32)
                *reinterpret_cast<uint4*>(p.o_part + to + 4 * pc) = v;
              else
                *reinterpret_cast<uint4*>(p.out + to + 8 * pc) = v;
            }
            __syncwarp();
          }
        };
        if (parts >= 0)
          rows_out(std::true_type{});
        else
          rows_out(std::false_type{});
      }
      if (real && (!SPREAD || quad == 0)) {
        if (parts >= 0) {
          // m counts V's scales in, l does not: together 2^m l = sum 2^t
          p.m_part[part] = some ? fmaxf(m, -1e30f) - kLift : -INFINITY;
          p.l_part[part] = some ? l : 0.f;
        } else if (p.lse) {
          p.lse[lse_at] = some ? (m - kLift + fast_log2(l)) * kLn2 : -INFINITY;
        }
      }
    }
  } else if (warp >= C::kConvWarp0) {
    if constexpr (D == 128 && !SPREAD) set_regs<false, NT == 2 ? 64 : 96>();
    // ======================= V to fp16 ========================================
    // [key][128 codes] 128-byte swizzled -> [64 channels][key][64 fp16] likewise
    const int ct = tid - 32 * C::kConvWarp0;
    constexpr int RI = 4 * C::kConvWarps;  // rows the warps take at once, a thread 16 channels: row & 7 is a thread's own
    const int row0 = ct >> 3, ch = ct & 7, x7 = row0 & 7;
    // The upper 64 channels' lanes store their halves the other way round: eight
    // lanes of a row then cover all of shared memory's banks.
    const int swap = ch >> 2, q = (ch & 3) * 2;
    const uint8_t* src0 = smem + C::kVr + row0 * 128 + ((ch ^ x7) << 4);
    uint8_t* dst0 = smem + C::kVf + swap * (BN * 128) + row0 * 128;
    const int at0 = ((q + swap) ^ x7) << 4, at1 = ((q + 1 - swap) ^ x7) << 4;
    // (one row tile: Q's codes pass through here first)
    bool ok = NT == 2 || wait_bar<100>(bar(ctl.q_ready), 0, abort);
    for (int i = 0; i < nt && ok; ++i) {
      const int s = i & 1;
      const uint32_t ph = uint32_t(i >> 1) & 1u;
      ok = wait_bar<100>(bar(ctl.vr_full[s]), ph, abort) &&
           (i < NV || wait_bar<100>(bar(ctl.done[(i - NV) & 3]), uint32_t((i - NV) >> 2) & 1u, abort));
      if (!ok) break;
      const uint8_t* src = src0 + s * kTile;
      uint8_t* dst = dst0 + (i & (NV - 1)) * 2 * kTile;
      const int live = k_end - (k0 + i * BN);  // rows from here on are no key's: zeros (they may hold NaN codes)
#pragma unroll
      for (int it = 0; it < DH * BN / RI; ++it) {
        const int sub = it / (BN / RI), row = RI * (it % (BN / RI));  // 128-channel half; beside row0
        uint4 v = *reinterpret_cast<const uint4*>(src + sub * (BN * 128) + row * 128);
        if (row0 + row >= live) v = make_uint4(0u, 0u, 0u, 0u);
        const uint4 lo = make_uint4(e4m3x2_f16x2(v.x), e4m3x2_f16x2(v.x >> 16), e4m3x2_f16x2(v.y), e4m3x2_f16x2(v.y >> 16));
        const uint4 hi = make_uint4(e4m3x2_f16x2(v.z), e4m3x2_f16x2(v.z >> 16), e4m3x2_f16x2(v.w), e4m3x2_f16x2(v.w >> 16));
        uint8_t* at = dst + 2 * sub * (BN * 128) + row * 128;
        *reinterpret_cast<uint4*>(at + at0) = swap ? hi : lo;
        *reinterpret_cast<uint4*>(at + at1) = swap ? lo : hi;
      }
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(bar(ctl.vf_full[i & (NV - 1)]));
        tc::mbar_arrive(bar(ctl.vr_empty[s]));
      }
    }
  } else {
    if constexpr (D == 128 && !SPREAD) set_regs<false, NT == 2 ? 64 : 96>();
  if (warp == 0) {
    // ======================= TMA: K and V tiles ===============================
    const int box = min(BN, 1 << p.page_shift);  // rows of a copy
    const int per = BN / box;                    // copies a tile, one lane each
    const uint64_t pol = p.evict_first ? tc::l2_policy_evict_first() : tc::l2_policy_evict_normal();
    auto page_of = [&](int i) {  // of this lane's copy of tile i
      const int64_t key = int64_t(k0) + int64_t(i) * BN + lane * box;
      const int64_t e = key >> p.page_shift;
      return lane < per && key < k_end && e < p.bt_len ? p.block_table[b * p.bt_stride + e] : -1;
    };
    int pg = nt > 0 ? page_of(0) : -1;
    bool ok = true;
    int issued = 0;
    for (int i = 0; i < nt && ok; ++i) {
      const int next = i + 1 < nt ? page_of(i + 1) : -1;
      const int key0 = k0 + i * BN;
      const int valid = min(per, (k_end - key0 + box - 1) / box);
      const int row = (key0 + lane * box) & ((1 << p.page_shift) - 1);
      auto load = [&](const CUtensorMap* map, uint32_t dst, uint32_t full, bool used, uint32_t empty, uint32_t parity) {
        ok = !used || wait_bar<100>(empty, parity, abort);
        ok = __all_sync(~0u, ok);
        if (!ok) return;
        if (lane == 0) tc::mbar_arrive_expect_tx(full, uint32_t(valid * box * D));
        __syncwarp();
        if (lane < valid) {
#pragma unroll
          for (int dh = 0; dh < DH; ++dh) {
            const uint32_t at = dst + uint32_t(dh * BN * 128 + lane * box * 128);
            if (p.tma_head_inner)
              tc::tma_load_4d(at, map, full, 128 * dh, g, row, pg, pol);
            else
              tc::tma_load_4d(at, map, full, 128 * dh, row, g, pg, pol);
          }
        }
        ++issued;
      };
      const int ks = i % kKStages, vs = i & 1;
      const int kd = i == kKStages ? 0 : i - kKStages - 1;  // the step that used K's stage last
      load(&tmap_k, base + C::kK + ks * kTile, bar(ctl.k_full[ks]), i >= kKStages, bar(ctl.done[kd & 3]), uint32_t(kd >> 2) & 1u);
      if (ok)
        load(&tmap_v, base + C::kVr + vs * kTile, bar(ctl.vr_full[vs]), true, bar(ctl.vr_empty[vs]), (uint32_t(i >> 1) & 1u) ^ 1u);
      pg = next;
    }
    if (*abort && lane == 0) {
      // wait (bounded) for the copies in flight before the CTA exits: copy j of tile j / 2, K then V
      const uint64_t start = tc::globaltimer_ns();
      for (int j = max(0, issued - 2 * kKStages); j < issued; ++j) {
        const int i = j >> 1;
        const uint32_t full = (j & 1) ? bar(ctl.vr_full[i & 1]) : bar(ctl.k_full[i % kKStages]);
        const uint32_t par = (j & 1) ? uint32_t(i >> 1) & 1u : uint32_t(i / kKStages) & 1u;
        while (!tc::mbar_try_wait(full, par) && tc::globaltimer_ns() - start < kDrainNs) {
        }
      }
    }
  } else if (warp == 1) {
    // ======================= MMA ==============================================
    constexpr uint32_t idesc_qk = tc::idesc_e4m3(128, BN, false, false);
    constexpr uint32_t idesc_pv = idesc_f16(128, D);
    const uint64_t qd = tc::smem_desc(base, 16, 1024, tc::kSwizzle128B);
    const uint64_t kd = tc::smem_desc(base + C::kK, 16, 1024, tc::kSwizzle128B);
    // V: 64-channel columns of blocks BN * 128 bytes apart, 8-key groups 1024
    const uint64_t vd = tc::smem_desc(base + C::kVf, BN * 128, 1024, tc::kSwizzle128B);
    // (votes: the products below are issued by whole warps)
    bool ok = __all_sync(~0u, wait_bar<0>(bar(ctl.q_ready), 0, abort));
    tc::tc_fence_after();
    // Stages and buffers are constants at every issue (the loop runs over four tiles).
    auto qk = [&](auto a, auto buf, auto stage) {
#pragma unroll
      for (int term = 0; term < 2; ++term)
#pragma unroll
        for (int dh = 0; dh < DH; ++dh)
          if constexpr (C::kQt)
            umma_qk4_ts(tmem + uint32_t(buf * BN), tmem + C::kQcol + uint32_t(term * (D / 4) + 32 * dh),
                        uint32_t(kd) + stage * (kTile >> 4) + dh * (BN * 128 >> 4), uint32_t(kd >> 32), idesc_qk,
                        term > 0 || dh > 0);
          else
            umma_qk4(tmem + uint32_t(buf * BN), uint32_t(qd) + ((a * 2 + term) * DH + dh) * (kTile >> 4),
                     uint32_t(kd) + stage * (kTile >> 4) + dh * (BN * 128 >> 4), uint32_t(kd >> 32), idesc_qk,
                     term > 0 || dh > 0);
      tc::umma_commit_warp(bar(ctl.s_full[buf]));
    };
    auto wait_for = [&](uint64_t& barrier, int use) {
      ok = ok && __all_sync(~0u, wait_bar<0>(bar(barrier), uint32_t(use) & 1u, abort));
      return ok;
    };
    // row tile a's weights in buffer buf, on V stage vs, as the softmax hands them over
    auto weigh = [&](auto a, auto buf, auto vs, int i, int use) {
#pragma unroll
      for (int k = 0; k < NB; k += 4) {
        if (k == 0 || (kHalves == 2 && k == NB / 2)) {
          if (!wait_for(ctl.p_full[buf][k == 0 ? 0 : 1], use)) return false;
          tc::tc_fence_after();
        }
        umma_pv4(tmem + C::kO + uint32_t(a * D), tmem + uint32_t(buf * BN + 8 * k), uint32_t(vd) + vs * (2 * kTile >> 4) + 128 * k,
                 uint32_t(vd >> 32), idesc_pv, k > 0 || i > 0);
      }
      if (i == nt - 1) tc::umma_commit_warp(bar(ctl.o_last[a]));
      return true;
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    // Tile i's weights, tile i + 1's scores; U = i modulo the period. Products run in the
    // order they are issued, so a row tile's next scores may be asked for right behind
    // the product that reads its weights from the same columns. What is sure to come is
    // waited for at the end of the step before: only the softmaxes' barriers are left
    // between the products.
    auto step = [&](auto u, int i) {
      constexpr int U = decltype(u)::value;
      using Sb = std::integral_constant<int, U & 1>;
      using Vs = std::integral_constant<int, U & (NV - 1)>;
      using Ks = std::integral_constant<int, (U + 1) % kKStages>;
      const bool more = i + 1 < nt;
      if constexpr (NT == 2) {
        if (!weigh(I0{}, I0{}, Vs{}, i, i)) return;
        if (more) qk(I0{}, I0{}, Ks{});
        if (!weigh(I1{}, I1{}, Vs{}, i, i)) return;
        if (more) qk(I1{}, I1{}, Ks{});
      } else {
        if (more) qk(I0{}, std::integral_constant<int, (U + 1) & 1>{}, Ks{});
        if (!weigh(I0{}, Sb{}, Vs{}, i, i >> 1)) return;
      }
      if (!more) return;
      tc::umma_commit_warp(bar(ctl.done[U]));
      // (both at once, by different lanes)
      const bool k = (lane & 1) && i + 2 < nt;
      ok = ok && __all_sync(~0u, wait_bar<0>(k ? bar(ctl.k_full[(U + 2) % kKStages]) : bar(ctl.vf_full[(U + 1) & (NV - 1)]),
                                             uint32_t(k ? (i + 2) / kKStages : (i + 1) / NV) & 1u, abort));
      __syncwarp();  // (what one lane has seen holds for the one that issues)
    };
    if (nt > 0 && wait_for(ctl.k_full[0], 0)) {
      qk(I0{}, I0{}, I0{});
      if constexpr (NT == 2) qk(I1{}, I1{}, I0{});
      wait_for(ctl.vf_full[0], 0);
      if (nt > 1) wait_for(ctl.k_full[1], 0);
      for (int i = 0; i < nt && ok; i += kKStages) {
        step(I0{}, i);
        if (ok && i + 1 < nt) step(I1{}, i + 1);
        if (ok && i + 2 < nt) step(std::integral_constant<int, 2>{}, i + 2);
        if (ok && i + 3 < nt) step(std::integral_constant<int, 3>{}, i + 3);
      }
    }
    if (!ok) {
      // wait (bounded) until every product issued so far is done
      tc::umma_commit_warp(bar(ctl.drain));
      const uint64_t start = tc::globaltimer_ns();
      while (!tc::mbar_try_wait(bar(ctl.drain), 0) && tc::globaltimer_ns() - start < kDrainNs) {
      }
    }
  } else if (warp == 2) {
    // ======================= the blocks' scales ================================
    for (int q = 0; q * TB < nt; ++q) {
      const int64_t key = int64_t(k0) + int64_t(q) * TB * BN + lane * 16;
      const int64_t e = key >> p.page_shift;
      int ke = 127, ve = 127;
      if (key < k_end) {
        const int pg = e < p.bt_len ? p.block_table[b * p.bt_stride + e] : -1;
        if (pg >= 0 && pg < p.num_pages) {
          const int at = (int(key) & ((1 << p.page_shift) - 1)) >> p.block_shift;
          ke = block_exp(p.side[0].exps[pg * p.side[0].esp + g * p.side[0].esh + at]);
          ve = block_exp(p.side[1].exps[pg * p.side[1].esp + g * p.side[1].esh + at]);
        } else {
          atomicOr(p.status, kStatusBadPage);
        }
      }
      if (!__all_sync(~0u, wait_bar<100>(bar(ctl.e_empty[q & 1]), (uint32_t(q >> 1) & 1u) ^ 1u, abort))) break;
      ctl.scale[q & 1][lane] = make_float4(__int_as_float(ke << 23), float(ve - 127), __int_as_float((254 - ve) << 23), 0.f);
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar(ctl.e_full[q & 1]));
    }
  }
  }

  // ---- teardown ------------------------------------------------------------
  tc::tc_fence_before();
  __syncthreads();
  if (*abort && tid == 0) atomicOr(p.status, kStatusTimeout);
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

// The cache side as a 4-D byte tensor (channel, token, head, page), the smaller of
// the token and head strides first; a copy is 128 channels of `rows` tokens.
bool encode(CUtensorMap* map, const BlockSide& s, const BlockPromptParams& p, int rows) {
  auto fn = tensor_map_encode_fn();
  if (!fn) return false;
  const int page = 1 << p.page_shift;
  const bool hi = p.tma_head_inner;
  const int64_t sh = p.h_k == 1 ? (hi ? 32 : s.sp) : s.sh;
  const cuuint64_t dims[4] = {cuuint64_t(p.d), cuuint64_t(hi ? p.h_k : page), cuuint64_t(hi ? page : p.h_k),
                              cuuint64_t(p.num_pages)};
  const cuuint64_t strides[3] = {cuuint64_t(hi ? sh : s.st), cuuint64_t(hi ? s.st : sh), cuuint64_t(s.sp)};
  const cuuint32_t box[4] = {128, cuuint32_t(hi ? 1 : rows), cuuint32_t(hi ? rows : 1), 1}, one[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, s.codes, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NT, bool SPREAD>
cudaError_t launch(const CUtensorMap& mk, const CUtensorMap& mv, const BlockPromptParams& p, cudaStream_t stream) {
  using C = Cfg<D, NT>;
  constexpr int bytes = C::kBytes + 1024;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static std::atomic<int> configured[64];  // the shared-memory limit is raised once per device
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(block_prompt_kernel<D, NT, SPREAD>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    configured[dev].store(1, std::memory_order_release);
  }
  const int64_t tiles = (int64_t(p.max_q_len) * p.h_r + C::kRows - 1) / C::kRows;
  const int64_t x = p.work ? int64_t(p.num_work) * p.h_k : int64_t(p.h_k) * p.splits;
  if (tiles > 65535 || x > INT32_MAX) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(x), unsigned(tiles), p.work ? 1u : unsigned(p.num_seqs));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, block_prompt_kernel<D, NT, SPREAD>, mk, mv, p);
}

}  // namespace

int block_prompt_rows(int d, int64_t rows) { return d == 128 && rows > 128 ? 256 : 128; }

cudaError_t launch_block_prompt(BlockPromptParams p, cudaStream_t stream, bool* unsupported) {
  const BlockSide &k = p.side[0], &v = p.side[1];
  p.tma_head_inner = k.sh < k.st ? 1 : 0;
  const int rows = std::min(p.d == 256 ? Cfg<256, 1>::BN : Cfg<128, 2>::BN, 1 << p.page_shift);
  CUtensorMap mk, mv;
  *unsupported = k.sp == 0 || v.sp == 0 || (v.sh < v.st) != (k.sh < k.st) || !encode(&mk, k, p, rows) || !encode(&mv, v, p, rows);
  if (*unsupported) return cudaSuccess;
  const int64_t n = int64_t(p.max_q_len) * p.h_r;
  if (p.d == 256) return n <= 32 ? launch<256, 1, true>(mk, mv, p, stream) : launch<256, 1, false>(mk, mv, p, stream);
  if (n <= 32) return launch<128, 1, true>(mk, mv, p, stream);
  return block_prompt_rows(p.d, n) == 256 ? launch<128, 2, false>(mk, mv, p, stream) : launch<128, 1, false>(mk, mv, p, stream);
}

}  // namespace mj
