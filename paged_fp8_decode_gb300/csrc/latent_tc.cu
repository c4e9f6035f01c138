// mj_latent_attention: decode attention over a paged cache of latent rows
// (512 latent and 64 rotary e4m3 codes a token), in the absorbed form. All
// query heads of a request read the same key row, and the row's first 512
// channels are the value:
//
//   t[r][j] = softmax_scale (s0 q[r][:512] . c[j] + s1 q[r][512:] . c'[j])
//   out[r]  = sum_j softmax_j(t[r]) s0 c[j]
//
// One persistent CTA per (plan slot, row tile): it runs through its slot's
// work rows (request, tile range), so that every CTA streams the same number
// of tiles whatever the lengths. The rows of a request (query tokens x heads)
// are tiled by NR = 16, 32 or 64. Keys are the M = 128 side of both products,
// so a few rows still fill the tensor core, and a cache byte loaded once
// serves both:
//
//   S^T[key][row]  = K[key][:576] . Q[row][:576]    A = the tile (K-major),  B = Q
//   O^T[ch][row]  += C^T[ch][key] . P^T[key][row]   A = the tile (MN-major), B = P
//
// kind::f8f6f4 multiplies 8-bit floats, so the bf16 queries and the softmax
// weights enter as two terms each. A query row is scaled by the power of two that
// puts its largest value between 224 and 448 and split into hi = e4m3(x) and
// lo = e4m3(x - hi), two rows of the Q tile, their products added when S is read.
// bf16 has 8 bits and the terms 4 each, so a latent channel from 1/4 on is exact,
// a smaller one within 2^-10; s0 goes into the row's logit scale, and the rotary
// channels, which take s1 / s0, are within 2^-8 of themselves. (By s0 448 / amax,
// no power of two, all were within 2^-8 only: logits of 6 nats off by 0.01.)
// A weight p is split into hi = e4m3(p) and lo, the rest in e5m2: two products
// into one accumulator. From 2^-6 on that is within 2^-7.8 of p, 0.15% rms, about
// bf16's own. Below 2^-6 hi is on a fixed step and lo alone has two bits, so that
// many equal small weights, all off alike, would change their share of a row
// (131071 keys 16.8 binades below one: the output by 2% of max|V|); there lo is
// rounded up or down by a dither, 8 bits of a hash of the key's index, and the
// errors cancel (0.01%). The row sums add the p themselves in float32.
//
// Warps: 0, 2, 3 the TMA producers, 1 the MMA issuer, 4.. one or two softmax
// warpgroups (thread x of a group: key x of S, channel x of each of the four
// 128-channel blocks of O; a group owns RW = NR / groups rows).
//
// Shared memory: a ring of latent sub-tiles (128 keys x 128 channels, 128-byte
// swizzled as tcgen05.mma reads them) and of rotary sub-tiles (128 keys x 64
// channels, 64-byte swizzled); a latent entry is released when the PV product
// of its channels is done, a rotary one after QK.
//
// What bounds it (GB300, one launch and the merge; DRAM reads are the cache's
// bytes, 152.3 MB for 151.0 MB of 64 x 4096 tokens):
//   16 rows: HBM. 64 x 4096 tokens, 16 heads: 34.7 us, 4.4 TB/s in all; once it
//   streams, a tile takes 3400 cycles an SM, 6.3 TB/s. The rest is the start
//   (7500 cycles to the first scores), the last tile and the merge (3 us).
//   64 rows: the chain load, QK, softmax, PV of a ring that holds two tiles
//   beside the 72 KB of Q's two terms, 4400 cycles a tile; the products alone
//   take 3055 (18 MMAs of N = 128 at 65 cycles and 32 of N = 64 at 49 + issue),
//   and at N = 64 both operands' reads fill the shared memory's 128 bytes a
//   cycle. 48 ragged requests of 128 heads: 119.5 us, 900 TFLOP/s counted once.
//   A change of work row there is serial: after a row's last tile the softmax
//   warps stage the next row's queries and write the row's output while the
//   tensor pipe idles, so many short requests are slowest (128 of 1024 tokens,
//   128 heads: 64 us for 19 of operations).
//   Short requests: code that runs once comes from L2, 10 of the 23 cycles
//   between two instructions of a warp are waits for it; hence the rolled loops.

#include <atomic>
#include <climits>

#include "latent_ptx.cuh"
#include "mj_device.cuh"
#include "mj_latent.h"

namespace mj {

namespace {

constexpr int kSub = 16384;       // latent sub-tile: 128 keys x 128 bytes
constexpr int kRopeSub = 8192;    // rotary sub-tile: 128 keys x 64 bytes
constexpr int kRow = MJ_LATENT_ROW_BYTES;
constexpr int kLat = MJ_LATENT_DIM;
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr uint64_t kDrainLimitNs = 100000000ull;
constexpr int kMaxDynSmem = 227 * 1024;

// A weight is 2^e, e = t + c8 with a constant c8 per row (minus the reference)
// that moves when some e of a tile exceeds kTop (2^8.5 < 448). At the row's first
// tile the largest e is put at kBase, so that later tiles seldom exceed kTop
// (moving costs about as much as a tile's softmax: with a base of 6 every
// second tile of 64 rows of normal logits moved one); where it stands out by
// more than kStandsOut from the smallest of the four warps' maxima (a sink), at
// kBaseSink, which leaves more binades below it. A later move also puts it there.
constexpr float kTop = 8.5f, kBase = 4.f, kBaseSink = 6.f, kStandsOut = 8.f;
constexpr float kFar = 100.f;  // binades: a longer move starts again from the row maxima

template <int NR>
struct Cfg {
  static constexpr int kGroups = NR == 16 ? 1 : 2;  // softmax warpgroups
  static constexpr int kRw = NR / kGroups;          // rows of a group
  static constexpr int kThreads = 128 + 128 * kGroups;
  static constexpr int kRing = NR == 64 ? 8 : (NR == 32 ? 9 : 11);  // latent entries
  static constexpr int kRopeRing = NR == 64 ? 1 : 2;
  static constexpr int kPBufs = NR == 64 ? 1 : 2;
  static constexpr int kPrefetchTiles = 2;      // before the wait for the preceding kernel; at most 4 (32 pages)
  static constexpr int kPBytes = 2 * NR * 128;  // hi and lo
  static constexpr int kQSub = 2 * NR * 128;    // hi and lo rows of one 128-channel sub-tile
  static constexpr int kQBytes = 4 * kQSub + 2 * NR * 64;
  static constexpr int kOffRope = kRing * kSub;
  static constexpr int kOffQ = kOffRope + kRopeRing * kRopeSub;
  static constexpr int kOffP = kOffQ + kQBytes;
  static constexpr int kOffCtrl = kOffP + kPBufs * kPBytes;
  static constexpr int kSCols = 2 * NR;           // hi and lo columns of one S buffer
  static constexpr int kCols = 2 * kSCols + 4 * NR;  // two S buffers, four O blocks
  static constexpr uint32_t kTmemCols = kCols <= 128 ? 128 : (kCols <= 256 ? 256 : 512);
};

template <int NR>
struct Ctrl {
  uint64_t full[Cfg<NR>::kRing], empty[Cfg<NR>::kRing];
  uint64_t rfull[Cfg<NR>::kRopeRing], rempty[Cfg<NR>::kRopeRing];
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t q_ready;
  uint64_t bound_bar[2][2];  // [group][exchange & 1]: the group's warps have posted their rows
  uint64_t row_bar[2];       // ... their row maxima
  uint64_t sum_bar[2];       // ... their row sums
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  alignas(16) uint32_t above[2][2][4];  // [group][exchange & 1]: per warp, the rows whose reference it asks to move
  alignas(16) uint8_t by[2][2][4][NR == 64 ? 32 : 16];  // ... and by how many binades
  alignas(16) float red[2][4][NR == 64 ? 32 : 16];      // per warp: row maxima, at the end row sums
  alignas(16) float scale[NR];  // logit (log2 units) per unit of S
  alignas(16) float c8[NR];     // minus the reference
  alignas(16) float move[NR];   // first tile of a work row: the reference's move; later ones: 2^-move; at the end:
                                // the output's factor
  alignas(16) int lim[NR];      // last visible key
};

template <int NR>
constexpr int smem_bytes() {
  return Cfg<NR>::kOffCtrl + int(sizeof(Ctrl<NR>));
}
static_assert(smem_bytes<64>() <= kMaxDynSmem && smem_bytes<32>() <= kMaxDynSmem && smem_bytes<16>() <= kMaxDynSmem,
              "shared memory");

// Bounded wait, the loop out of line: the kernel has some twenty of them, and
// code that runs once is bound by its fetch from L2.
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* abort) {
  return tc::mbar_wait(bar, parity, abort, kWaitLimitNs);
}
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  return tc::mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort);
}

// Reduce N per-lane values over the warp's lanes: row r ends up in lanes
// r * (32 / N) .. + 32 / N - 1 (halve the rows a lane keeps, exchange the rest).
template <int N, bool MAX>
__device__ __forceinline__ float reduce_rows(float (&v)[N], int lane) {
#pragma unroll
  for (int c = N, m = 16; c > 1; c >>= 1, m >>= 1) {
    const bool upper = (lane & m) != 0;
#pragma unroll
    for (int j = 0; j < c / 2; ++j) {
      const float send = upper ? v[j] : v[c / 2 + j];
      const float keep = upper ? v[c / 2 + j] : v[j];
      const float recv = __shfl_xor_sync(0xFFFFFFFFu, send, m);
      v[j] = MAX ? fmaxf(keep, recv) : keep + recv;
    }
  }
  float r = v[0];
#pragma unroll
  for (int m = 16 / N; m > 0; m >>= 1) {
    const float o = __shfl_xor_sync(0xFFFFFFFFu, r, m);
    r = MAX ? fmaxf(r, o) : r + o;
  }
  return r;
}

// The e4m3 codes of two values and what they leave, as float16 pairs. By way of
// f16, whose 2^-11 is far inside the terms' own steps and whose range holds every
// value here (weights and scaled queries are at most 448; below 2^-14 it keeps
// 2^-25), because the difference (exact) and the conversions take both values at
// once there.
__device__ __forceinline__ uint32_t split2(float a, float b, __half2& h, uint32_t& rest) {
  h = __floats2half2_rn(a, b);
  uint32_t hb, back;
  uint16_t hc;
  memcpy(&hb, &h, 4);
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(hc) : "r"(hb));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(hc));
  asm("sub.f16x2 %0, %1, %2;" : "=r"(rest) : "r"(hb), "r"(back));
  return hc;
}

// Two query values: hi = e4m3(v), lo = e4m3(v - hi).
__device__ __forceinline__ void query_terms(float a, float b, uint32_t& hi, uint32_t& lo) {
  __half2 h;
  uint32_t rest;
  uint16_t lc;
  hi = split2(a, b, h, rest);
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(lc) : "r"(rest));
  lo = lc;
}

// Four weights: hi = e4m3(p), lo = e5m2(p - hi). An e5m2 code is the upper byte of
// a float16, so lo is rounded by adding to the lower byte: 0x80, to nearest, from
// 2^-6 on; `dither` (the key's 8 bits, in both halves) below, where over its 256
// values the two terms add up to the float16 weight on average. A weight of 0
// stays 0. (A NaN's hi is NaN whatever becomes of lo.)
__device__ __forceinline__ void weight_terms(const float* p, uint32_t dither, uint32_t& hi, uint32_t& lo) {
  uint32_t hc[2], rest[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    __half2 h;
    hc[k] = split2(p[2 * k], p[2 * k + 1], h, rest[k]);
    const uint32_t small = __hlt2_mask(h, __float2half2_rn(0x1p-6f));
    rest[k] += (dither & small) | (0x00800080u & ~small);
  }
  hi = __byte_perm(hc[0], hc[1], 0x5410);
  lo = __byte_perm(rest[0], rest[1], 0x7531);
}

// 8 bits of a key's index, in both halves: the dither of its weights. A hash, so
// that every 2nd, 16th, ... key takes all values about alike often too.
__device__ __forceinline__ uint32_t key_dither(uint32_t key) {
  uint32_t u = key * 0x9E3779B1u;  // 2^32 / golden ratio
  u ^= u >> 16;
  return (u * 0x9E3779B1u >> 24) * 0x00010001u;
}

// The larger magnitudes of two bf16 pairs, as bit patterns (a NaN counts as above infinity).
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
  return __vmaxu2(a & 0x7FFF7FFFu, b & 0x7FFF7FFFu);
}

// One work row: keys [tb * 128, min(te * 128, L)) of request b.
struct Work {
  int b, part, L, ntiles;
  int64_t k0, k1;
};

__device__ __forceinline__ int seq_len(const LatentParams& p, int b) {
  return b >= 0 && b < p.num_seqs ? p.seq_lens[b] : 0;
}

// b0, L0: the slot's first request and its length, read beside the work row
// instead of after it.
__device__ __forceinline__ Work load_work(const LatentParams& p, int row, int b0, int L0) {
  const int4 w = reinterpret_cast<const int4*>(p.work)[row];
  Work k;
  k.b = w.x;
  k.part = w.w;
  k.L = w.x == b0 ? L0 : seq_len(p, w.x);
  k.k0 = int64_t(w.y) * kKvTile;
  k.k1 = min(int64_t(w.z) * kKvTile, int64_t(k.L));
  k.ntiles = w.y >= 0 && k.k1 > k.k0 && w.w < 2 * p.slots ? int((k.k1 - k.k0 + kKvTile - 1) / kKvTile) : 0;
  return k;
}

template <int NR>
__global__ void __launch_bounds__(Cfg<NR>::kThreads, 1)
    latent_kernel(const __grid_constant__ CUtensorMap tmap_lat, const __grid_constant__ CUtensorMap tmap_rope,
                  LatentParams p) {
  using C = Cfg<NR>;
  constexpr int RW = C::kRw, G = C::kGroups;
  extern __shared__ __align__(1024) uint8_t smem[];
  Ctrl<NR>& ctl = *reinterpret_cast<Ctrl<NR>*>(smem + C::kOffCtrl);
  const uint32_t base = tc::smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (base & 1023u) {  // the swizzled layouts need it; a block without static shared memory starts so
    if (tid == 0) atomicOr(p.status, kStatusBadPlan);
    return;
  }

  // The queries of rows r_from .. r_to - 1 of the tile, of request b, into L2
  // (n threads, this one the t-th).
  auto prefetch_rows = [&](int b, int t, int n, int r_from, int r_to) {
    constexpr int kLines = kRow * 2 / 128;
    const int tile0 = (int(blockIdx.x) % p.n_row_tiles) * NR;
#pragma unroll 1
    for (int k = t; k < (r_to - r_from) * kLines; k += n) {
      const int r = tile0 + r_from + k / kLines, tq = r / p.h, h = r - tq * p.h;
      if (r < p.n_q)
        tc::prefetch_l2(p.q + (int64_t(b) * p.q_len + tq) * p.q_ts + int64_t(h) * p.q_hs + (k % kLines) * 64);
    }
  };

  if (tid == 0) {
    for (int s = 0; s < C::kRing; ++s) {
      tc::mbar_init(tc::smem_u32(&ctl.full[s]), 1);
      tc::mbar_init(tc::smem_u32(&ctl.empty[s]), 1);
    }
    for (int s = 0; s < C::kRopeRing; ++s) {
      tc::mbar_init(tc::smem_u32(&ctl.rfull[s]), 1);
      tc::mbar_init(tc::smem_u32(&ctl.rempty[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(tc::smem_u32(&ctl.s_full[s]), 1);
      tc::mbar_init(tc::smem_u32(&ctl.p_full[s]), 128 * G);
      tc::mbar_init(tc::smem_u32(&ctl.o_full[s]), 1);
      for (int x = 0; x < 2; ++x) tc::mbar_init(tc::smem_u32(&ctl.bound_bar[s][x]), 4);
      tc::mbar_init(tc::smem_u32(&ctl.row_bar[s]), 4);
      tc::mbar_init(tc::smem_u32(&ctl.sum_bar[s]), 4);
    }
    tc::mbar_init(tc::smem_u32(&ctl.q_ready), 128 * G);
    tc::mbar_init(tc::smem_u32(&ctl.drain), 1);
    ctl.abort = 0;
    tc::fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tc::prefetch_tmap(&tmap_lat);
    tc::prefetch_tmap(&tmap_rope);
  }
  if (warp == 1) {
    tc::tmem_alloc(tc::smem_u32(&ctl.tmem_base), C::kTmemCols);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;
  volatile int* abort = &ctl.abort;

  const int slot = int(blockIdx.x) / p.n_row_tiles;
  const int r0 = (int(blockIdx.x) % p.n_row_tiles) * NR;
  const int nr = min(NR, p.n_q - r0);  // real rows of this tile

  // Programmatic dependent launch: the set-up above reads nothing that the
  // preceding kernel on the stream may write; everything after the wait may.
  // Before it, L2 is asked for the pages of the first kPrefetchTiles tiles and
  // the queries of the first row, so that the memory streams them while the
  // preceding kernel finishes. A prefetch returns no data, and that kernel's
  // writes land in L2: the plan and block table that it is aimed with are only a
  // guess (bounds-checked), and all of it is read again after the wait.
  if (warp == 3 || warp >= 4) {
    const int4 f = reinterpret_cast<const int4*>(p.slot_table)[slot];
    if (f.y > f.x && f.x >= 0 && f.x < p.max_work && f.z >= 0 && f.z < p.num_seqs && f.w >= 0) {
      if (warp == 3 && r0 == 0) {
        const int4 w = reinterpret_cast<const int4*>(p.work)[f.x];
        const int64_t page = (int64_t(f.w) << (7 - p.page_shift)) + lane;
        const int64_t end = int64_t(min(w.z, f.w + C::kPrefetchTiles)) << (7 - p.page_shift);
        if (p.page_span && page < end && page < p.bt_len) {
          const int pg = p.block_table[int64_t(f.z) * p.bt_stride + page];
          if (pg >= 0 && pg < p.num_pages) tc::prefetch_bulk_l2(p.cache + int64_t(pg) * p.stride_page, p.page_span);
        }
      } else if (warp >= 4) {
        prefetch_rows(f.z, tid - 128, 128 * G, 0, NR);
      }
    }
  }
  tc::grid_dependency_wait();

  const int4 first = reinterpret_cast<const int4*>(p.slot_table)[slot];  // rows, first request, its first tile
  const int w_begin = max(0, first.x), w_end = min(first.y, p.max_work);
  const int b0 = first.z, L0 = seq_len(p, b0);
  const uint32_t tO = tmem + uint32_t(2 * C::kSCols);

  if (warp == 0 || warp == 2 || warp == 3) {
    // ======================= TMA producers =====================================
    // Issuing a tensor load takes a warp 110 to 200 cycles (280 where one lane
    // of a diverged warp issues), and a tile is 5 sub-tiles of 1 to 8 pages: one
    // warp's issue alone held the stream at 20 bytes a cycle. Three warps share
    // a tile's sub-tiles: 0 and 3, 1 and the rotary one, 2.
    const int j_first = warp == 0 ? 0 : warp - 1;
    const uint64_t pol = p.evict_first ? tc::l2_policy_evict_first() : tc::l2_policy_evict_normal();
    const int ps = p.page_size, shift = p.page_shift, ppt = kKvTile >> shift;
    int gt = 0;      // tiles so far
    int issued = 0;  // sub-tiles this warp has begun to load, in order of (tile, sub-tile)
    bool ok = true;
    auto table_entry = [&](int b, int64_t page) {  // -1 past the request's entries
      return page < p.bt_len ? p.block_table[int64_t(b) * p.bt_stride + page] : -1;
    };
    // the first row's first entries, read beside its work row and length
    const int64_t page0 = int64_t(max(0, first.w)) * ppt + lane;
    const int entry0 = w_begin < w_end && b0 >= 0 && b0 < p.num_seqs ? table_entry(b0, page0) : -1;
    for (int row = w_begin; row < w_end && ok; ++row) {
      const Work w = load_work(p, row, b0, L0);
      const int64_t first_page = w.k0 >> shift, npages = ((w.k1 + ps - 1) >> shift) - first_page;
      const bool known = row == w_begin && w.b == b0 && first_page + lane == page0;
      int64_t batch = __all_sync(0xFFFFFFFFu, known) ? 0 : -1;
      int entry = entry0;
      for (int i = 0; i < w.ntiles && ok; ++i, ++gt) {
        const int nvalid = int(min(int64_t(ppt), npages - int64_t(i) * ppt));
        const int64_t e0 = int64_t(i) * ppt;
        if (batch < 0 || e0 + nvalid > batch + 32) {
          batch = e0;
          entry = e0 + lane < npages ? table_entry(w.b, first_page + e0 + lane) : -1;
        }
        const int at = int(e0 - batch);
        const int mine = __shfl_sync(0xFFFFFFFFu, entry, at + (lane & 7));
        if (warp == 0 && lane < nvalid && (mine < 0 || int64_t(mine) >= p.num_pages)) atomicOr(p.status, kStatusBadPage);
#pragma unroll 1
        for (int j = j_first; j < 5 && ok; j += 3) {
          const bool rope = j == 4;
          const int u = rope ? gt : 4 * gt + j;
          const int s = rope ? u % C::kRopeRing : u % C::kRing;
          const uint32_t round = uint32_t(rope ? u / C::kRopeRing : u / C::kRing);
          const uint32_t full = tc::smem_u32(rope ? &ctl.rfull[s] : &ctl.full[s]);
          const uint32_t empty = tc::smem_u32(rope ? &ctl.rempty[s] : &ctl.empty[s]);
          const uint32_t page_bytes = uint32_t(ps) * (rope ? 64u : 128u);
          uint32_t dst = base + (rope ? uint32_t(C::kOffRope + s * kRopeSub) : uint32_t(s * kSub));
          // (with a ring that is no multiple of four, another warp may have
          // loaded the entry before; this warp's own wait four sub-tiles ago
          // was for a later release than the one before that, so the parity
          // cannot be mistaken)
          ok = __all_sync(0xFFFFFFFFu, wait(empty, (round & 1u) ^ 1u, abort));
          if (!ok) break;
          if (lane == 0) tc::mbar_arrive_expect_tx(full, uint32_t(nvalid) * page_bytes);
          __syncwarp();
#pragma unroll 1
          for (int k = 0; k < nvalid; ++k, dst += page_bytes)
            tc::tma_load_3d_warp(dst, rope ? &tmap_rope : &tmap_lat, full, 128 * j, 0,
                             __shfl_sync(0xFFFFFFFFu, entry, at + k), pol);
          ++issued;
        }
      }
    }
    if (!ok && lane == 0) {
      // abort: wait (bounded) for this warp's loads still in flight before the CTA exits
      const uint64_t t0 = tc::globaltimer_ns();
      const int per = j_first == 2 ? 1 : 2;  // sub-tiles of a tile that are this warp's
      for (int n = max(0, issued - C::kRing); n < issued; ++n) {
        const int t = n / per, j = j_first + 3 * (n % per);
        uint64_t* bar = j == 4 ? &ctl.rfull[t % C::kRopeRing] : &ctl.full[(4 * t + j) % C::kRing];
        const uint32_t round = uint32_t(j == 4 ? t / C::kRopeRing : (4 * t + j) / C::kRing);
        while (!tc::mbar_try_wait(tc::smem_u32(bar), round & 1u) && tc::globaltimer_ns() - t0 < kDrainLimitNs) {
        }
      }
    }
  } else if (warp == 1) {
    // ======================= MMA issuer ========================================
    // The whole warp runs the loop and one elected lane issues: with a single
    // thread's loop the descriptors had to be moved to uniform registers for
    // every MMA, and issuing a tile's 50 took 5000 cycles instead of 2050.
    constexpr uint32_t idesc_qk = tc::idesc_e4m3(128, 2 * NR, false, false);
    constexpr uint32_t idesc_pv = tc::idesc_e4m3(128, NR, true, true);
    const uint64_t kd0 = tc::smem_desc(base, 16, 1024, tc::kSwizzle128B);
    const uint64_t qd0 = tc::smem_desc(base + uint32_t(C::kOffQ), 16, 1024, tc::kSwizzle128B);
    const uint64_t krd0 = tc::smem_desc(base + uint32_t(C::kOffRope), 16, 512, tc::kSwizzle64B);
    const uint64_t qrd = tc::smem_desc(base + uint32_t(C::kOffQ + 4 * C::kQSub), 16, 512, tc::kSwizzle64B);
    const uint64_t vd0 = tc::smem_desc(base, kSub, 1024, tc::kSwizzle128B);
    // P, MN-major without swizzle: 8-key core groups 128 B apart, 16-row blocks
    // 2 KB apart; lo after hi
    const uint64_t pd0 = tc::smem_desc(base + uint32_t(C::kOffP), 128, 2048, 0);
    auto ready = [&](uint64_t& bar, uint32_t parity) {
      return __all_sync(0xFFFFFFFFu, tc::mbar_test_wait(tc::smem_u32(&bar), parity)) != 0;
    };
    int sk = 0, sr = 0, sv = 0;           // ring entries QK (latent, rotary) and PV take next
    uint32_t fk = 0, fr = 0;              // and their phases
    int g0 = 0, nrow = 0;                 // tiles of the rows before; rows with tiles so far
    bool ok = true;
    for (int row = w_begin; row < w_end && ok; ++row) {
      const int ntiles = __shfl_sync(0xFFFFFFFFu, load_work(p, row, b0, L0).ntiles, 0);
      if (ntiles == 0) continue;
      ok = __all_sync(0xFFFFFFFFu, wait(tc::smem_u32(&ctl.q_ready), uint32_t(nrow) & 1u, abort));
      ++nrow;
      int nq = 0, jq = 0, np = 0;
      uint64_t t_idle = 0;
      while (ok && np < ntiles) {
        bool progressed = false;
        if (nq < ntiles && nq <= np + 1) {
          // QK of tile nq, sub-tile by sub-tile as they land (the S buffer is
          // free: the softmax read tile nq - 2 before it released P of it)
          const uint32_t d = tmem + uint32_t(((g0 + nq) & 1) * C::kSCols);
          while (jq < 4 && ready(ctl.full[sk], fk)) {
            tc::tc_fence_after();
            const uint64_t kd = kd0 + uint64_t(sk * (kSub >> 4)), qd = qd0 + uint64_t(jq * (C::kQSub >> 4));
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc::umma_f8f6f4_warp(d, kd + uint64_t(2 * k), qd + uint64_t(2 * k), idesc_qk, jq > 0 || k > 0);
            if (++sk == C::kRing) {
              sk = 0;
              fk ^= 1u;
            }
            ++jq;
            progressed = true;
          }
          if (jq == 4 && ready(ctl.rfull[sr], fr)) {
            tc::tc_fence_after();
            const uint64_t kd = krd0 + uint64_t(sr * (kRopeSub >> 4));
#pragma unroll
            for (int k = 0; k < 2; ++k) tc::umma_f8f6f4_warp(d, kd + uint64_t(2 * k), qrd + uint64_t(2 * k), idesc_qk, 1);
            tc::umma_commit_warp(tc::smem_u32(&ctl.s_full[(g0 + nq) & 1]));
            tc::umma_commit_warp(tc::smem_u32(&ctl.rempty[sr]));
            if (++sr == C::kRopeRing) {
              sr = 0;
              fr ^= 1u;
            }
            ++nq;
            jq = 0;
            progressed = true;
          }
        }
        if (np < nq) {
          const int gi = g0 + np;
          if (ready(ctl.p_full[gi & 1], uint32_t(gi >> 1) & 1u)) {
            tc::tc_fence_after();
            const uint64_t pd = pd0 + uint64_t((gi % C::kPBufs) * (C::kPBytes >> 4));
            const uint32_t acc = np > 0;
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
              const uint64_t vd = vd0 + uint64_t(sv * (kSub >> 4));
#pragma unroll
              for (int k = 0; k < 4; ++k) {  // 32 keys a step
                tc::umma_f8f6f4_warp(tO + uint32_t(j * NR), vd + uint64_t(256 * k), pd + uint64_t(32 * k), idesc_pv,
                                     k > 0 ? 1u : acc);
                tc::umma_f8f6f4_warp(tO + uint32_t(j * NR), vd + uint64_t(256 * k), pd + uint64_t(NR * 8 + 32 * k),
                                     idesc_pv | tc::kFormatBE5m2, 1);
              }
              tc::umma_commit_warp(tc::smem_u32(&ctl.empty[sv]));
              if (++sv == C::kRing) sv = 0;
            }
            tc::umma_commit_warp(tc::smem_u32(&ctl.o_full[gi & 1]));
            ++np;
            progressed = true;
          }
        }
        if (progressed) {
          t_idle = 0;
        } else {
          const uint64_t now = tc::globaltimer_ns();
          if (t_idle == 0) {
            t_idle = now;
          } else if (__any_sync(0xFFFFFFFFu, now - t_idle > kWaitLimitNs || *abort)) {
            *abort = 1;
            ok = false;
          }
          __nanosleep(32);
        }
      }
      g0 += ntiles;
    }
    if (!ok) {
      // abort: wait (bounded) until every MMA issued so far has completed
      tc::umma_commit_warp(tc::smem_u32(&ctl.drain));
      const uint64_t t0 = tc::globaltimer_ns();
      while (!tc::mbar_try_wait(tc::smem_u32(&ctl.drain), 0) && tc::globaltimer_ns() - t0 < kDrainLimitNs) {
      }
    }
  } else if (warp >= 4) {
    // ======================= softmax warpgroups ================================
    const int grp = (warp - 4) >> 2, qd = warp & 3;
    const int x = qd * 32 + lane;  // key of the tile (S), channel of a block (O)
    const uint32_t lane_off = uint32_t(qd * 32) << 16;
    const int rg = grp * RW;       // the group's first row in the tile
    constexpr int kShare = 32 / RW;  // lanes that share a row after reduce_rows
    const float ds0 = p.descale[0], ds1 = p.descale[1];
    // Queries enter in units of one descale: the latent channels', unless it is 0
    // or far below the other (2^16 times a row's factor, 2^108 at most, is finite).
    const float unit = ds0 != 0.f && fabsf(ds1) <= fabsf(ds0) * 0x1p16f ? ds0 : (ds1 != 0.f ? ds1 : 1.f);
    const float rel0 = ds0 / unit, rel1 = ds1 / unit;
    const float qk_log2 = p.softmax_scale * kLog2e * unit;
    const int rows_pad = p.n_row_tiles * NR;  // rows of a partial
    int g0 = 0;           // tiles of the rows before
    int xb = 0, xr = 0, xs = 0;  // bound, row and sum exchanges so far (the same in every thread of the group)
    bool ok = true;
    int row = w_begin;
    // The next work row that holds keys; empty partials are written on the way.
    auto next_row = [&](Work& w) {
      for (; row < w_end; ++row) {
        w = load_work(p, row, b0, L0);
        if (w.ntiles > 0) {
          ++row;
          return true;
        }
        // no key of this range is held any more
        if (w.part >= 0 && w.part < 2 * p.slots && x < RW) p.m_part[int64_t(w.part) * rows_pad + r0 + rg + x] = -INFINITY;
        if (w.part >= 2 * p.slots && x == 0) atomicOr(p.status, kStatusBadPlan);
      }
      return false;
    };
    Work w = {}, wn = {};
    bool have = false;            // w's tiles are done
    bool more = next_row(wn);     // wn is the row after it
    float l_part[RW];
    float c8_row = 0.f;      // lane r < RW: row r's c8
    bool empty_row = true;   // lane r < RW: row r has seen no key
    // One turn: post w's sums, stage the next row's queries (the tensor core
    // still works on w's last product), then w's output (it already works on
    // the next row's first scores), then the next row's tiles.
    for (;;) {
      if (have) {
        // (every warp has read the last tile's row maxima, whose place the sums
        // take, and the row constants, which the next row's replace)
        ok = wait(tc::smem_u32(&ctl.p_full[(g0 - 1) & 1]), uint32_t((g0 - 1) >> 1) & 1u, abort);
        if (!ok) break;
        const float ws = reduce_rows<RW, false>(l_part, lane);
        if (lane % kShare == 0) ctl.red[grp][qd][lane / kShare] = ws;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::smem_u32(&ctl.sum_bar[grp]));
      }
      if (more) {
        // ---- Q: RW rows by 128 threads, kTpr threads a row --------------------
        {
          constexpr int kTpr = 128 / RW;
          const int r = x / kTpr, part = x % kTpr;
          const int gr = r0 + rg + r;  // row of the request
          const bool live = rg + r < nr;
          const int tq = live ? gr / p.h : 0, h = live ? gr - tq * p.h : 0;
          const uint16_t* src = p.q + (int64_t(wn.b) * p.q_len + tq) * p.q_ts + int64_t(h) * p.q_hs;
          // The 8 bytes of a chunk's hi codes: row tr of its sub-tile of the Q
          // tile; the lo codes NR rows on (a multiple of 8, so swizzled alike).
          const int tr = rg + r;
          auto hi_at = [&](int c) {
            const int ch = c * 8;
            return ch < kLat ? uint32_t(C::kOffQ + (ch >> 7) * C::kQSub + tr * 128 + ((((ch & 127) >> 4) ^ (tr & 7)) << 4) + (ch & 8))
                             : uint32_t(C::kOffQ + 4 * C::kQSub + tr * 64 + ((((ch - kLat) >> 4) ^ ((tr >> 1) & 3)) << 4) + (ch & 8));
          };
          auto lo_step = [&](int c) { return uint32_t(NR * (c < kLat / 8 ? 128 : 64)); };
          constexpr int kCh = kRow / 8 / kTpr;  // 8-channel chunks of a thread, requested at once
          uint4 qv[kCh];
#pragma unroll
          for (int c = 0; c < kCh; ++c)
            qv[c] = live ? *reinterpret_cast<const uint4*>(src + (part + c * kTpr) * 8) : make_uint4(0u, 0u, 0u, 0u);
          // the raw chunks wait in the places of their codes, so that the
          // conversion can be a rolled loop (a thread's registers could not be
          // indexed, and there is no L1 to speak of beside this shared memory)
#pragma unroll
          for (int ci = 0; ci < kCh; ++ci) {
            const int c = part + ci * kTpr;
            *reinterpret_cast<uint2*>(smem + hi_at(c)) = make_uint2(qv[ci].x, qv[ci].y);
            *reinterpret_cast<uint2*>(smem + hi_at(c) + lo_step(c)) = make_uint2(qv[ci].z, qv[ci].w);
          }
          // |q| of two channels as bf16 bit patterns, which order like the values
          uint32_t am_lat = 0, am_rope = 0;
#pragma unroll
          for (int c = 0; c < kCh; ++c) {
            const uint32_t m = max_abs_bf16x2(max_abs_bf16x2(qv[c].x, qv[c].y), max_abs_bf16x2(qv[c].z, qv[c].w));
            if (part + c * kTpr < kLat / 8)
              am_lat = max_abs_bf16x2(am_lat, m);
            else
              am_rope = max_abs_bf16x2(am_rope, m);
          }
          float am = fmaxf(fmaxf(__uint_as_float(am_lat << 16), __uint_as_float(am_lat & 0xFFFF0000u)) * fabsf(rel0),
                           fmaxf(__uint_as_float(am_rope << 16), __uint_as_float(am_rope & 0xFFFF0000u)) * fabsf(rel1));
#pragma unroll
          for (int m = 1; m < kTpr; m <<= 1) am = fmaxf(am, __shfl_xor_sync(0xFFFFFFFFu, am, m));
          am = fmaxf(am, 1e-30f);
          // 2^(8 - k), 2^k the power below am 8/7: am goes to [224, 448]
          const uint32_t k2 = __float_as_uint(am * (8.f / 7.f)) & 0x7F800000u;
          const float up = __uint_as_float((262u << 23) - k2);
#pragma unroll 1
          for (int c = part; c < kRow / 8; c += 3 * kTpr) {  // three chunks at a time
            uint2 q0[3], q1[3];
#pragma unroll
            for (int t = 0; t < 3; ++t) {
              q0[t] = *reinterpret_cast<const uint2*>(smem + hi_at(c + t * kTpr));
              q1[t] = *reinterpret_cast<const uint2*>(smem + hi_at(c + t * kTpr) + lo_step(c + t * kTpr));
            }
#pragma unroll
            for (int t = 0; t < 3; ++t) {
              const float f = (c + t * kTpr < kLat / 8 ? rel0 : rel1) * up;
              const uint32_t q4[4] = {q0[t].x, q0[t].y, q1[t].x, q1[t].y};
              uint32_t h[4], l[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                query_terms(__uint_as_float(q4[k] << 16) * f, __uint_as_float(q4[k] & 0xFFFF0000u) * f, h[k], l[k]);
              q0[t] = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
              q1[t] = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
            }
#pragma unroll
            for (int t = 0; t < 3; ++t) {
              *reinterpret_cast<uint2*>(smem + hi_at(c + t * kTpr)) = q0[t];
              *reinterpret_cast<uint2*>(smem + hi_at(c + t * kTpr) + lo_step(c + t * kTpr)) = q1[t];
            }
          }
          if (part == 0) {
            // (NaN for a row with an infinity)
            ctl.scale[rg + r] = __uint_as_float(k2 - (8u << 23)) * qk_log2 + (am - am);
            ctl.c8[rg + r] = 0.f;
            ctl.lim[rg + r] = !live ? -1 : (p.causal ? wn.L - p.q_len + tq : INT_MAX);
          }
        }
      }
      if (have) {
        ok = wait(tc::smem_u32(&ctl.sum_bar[grp]), uint32_t(xs) & 1u, abort);
        if (!ok) break;
        ++xs;
        if (lane < RW) {
          const float l = (ctl.red[grp][0][lane] + ctl.red[grp][1][lane]) + (ctl.red[grp][2][lane] + ctl.red[grp][3][lane]);
          const int gr = r0 + rg + lane;
          // the output's factor: a partial stays as it is, an empty row becomes 0 (the same in the four warps)
          ctl.move[rg + lane] = w.part >= 0 ? 1.f : (empty_row ? 0.f : ds0 / l);
          if (qd == 0) {
            const float m = -c8_row;  // l = sum of 2^(t - m)
            if (w.part >= 0) {
              p.m_part[int64_t(w.part) * rows_pad + gr] = empty_row ? -INFINITY : m;
              p.l_part[int64_t(w.part) * rows_pad + gr] = l;
            } else if (p.lse && rg + lane < nr) {
              p.lse[int64_t(w.b) * p.n_q + gr] = empty_row ? -INFINITY : (m + fast_log2(l)) * kLn2;
            }
          }
        }
        __syncwarp();
      }
      if (more) {
        // (after the sums are read: the next row's first maxima take their place)
        tc::fence_async_smem();
        tc::mbar_arrive(tc::smem_u32(&ctl.q_ready));
      }
      if (have) {
        ok = wait(tc::smem_u32(&ctl.o_full[(g0 - 1) & 1]), uint32_t((g0 - 1) >> 1) & 1u, abort);
        if (!ok) break;
        tc::tc_fence_after();
        if (w.part >= 0) {
          // a partial: four rows of a channel are one 16-byte store, a warp's 512 bytes in a row
          float4* dst = reinterpret_cast<float4*>(p.o_part) +
                        ((int64_t(w.part) * p.n_row_tiles + r0 / NR) * 4 * (NR / 4) + rg / 4) * 128 + x;
#pragma unroll 1
          for (int k = 0; k < 4 * (RW / 16); ++k) {  // 16 rows of a channel block
            const int j = k / (RW / 16), c = k % (RW / 16) * 16;
            float v[16];
            tc::tmem_ld16(tO + uint32_t(j * NR + rg + c) + lane_off, v);
            tc::tmem_wait_ld();
#pragma unroll
            for (int q = 0; q < 4; ++q)
              dst[(j * (NR / 4) + c / 4 + q) * 128] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
          }
        } else {
          // the output: two lanes trade, so that each holds two channels of one
          // row (even lanes the even rows) and a store is 4 bytes
          const bool odd = lane & 1;
          uint16_t* dst = p.out + int64_t(w.b) * p.q_len * p.out_ts + (x & ~1);
          const int rows = min(RW, nr - rg);
          int gr = r0 + rg + (odd ? 1 : 0);
          int tq = gr / p.h, h = gr - tq * p.h;
#pragma unroll 1
          for (int c = 0; c < rows; c += 2) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              v[2 * j] = tc::tmem_ld1(tO + uint32_t(j * NR + rg + c) + lane_off);
              v[2 * j + 1] = tc::tmem_ld1(tO + uint32_t(j * NR + rg + c + 1) + lane_off);
            }
            tc::tmem_wait_ld();
            const float2 f = *reinterpret_cast<const float2*>(&ctl.move[rg + c]);
            uint16_t* at = dst + int64_t(tq) * p.out_ts + int64_t(h) * p.out_hs;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float a = f.x == 0.f ? 0.f : v[2 * j] * f.x, b = f.y == 0.f ? 0.f : v[2 * j + 1] * f.y;
              const float other = __shfl_xor_sync(0xFFFFFFFFu, odd ? a : b, 1);
              const float lo_c = odd ? other : a, hi_c = odd ? b : other;
              if (c + (odd ? 1 : 0) < rows)
                *reinterpret_cast<uint32_t*>(at + 128 * j) =
                    uint32_t(float_to_out_bits(lo_c, p.out_f16)) | (uint32_t(float_to_out_bits(hi_c, p.out_f16)) << 16);
            }
            h += 2;
            while (h >= p.h) {
              h -= p.h;
              ++tq;
            }
          }
        }
        tc::tc_fence_before();
        __syncwarp();
      }
      if (!more) break;
      w = wn;
      have = true;
      more = next_row(wn);
      if (more) {
        // its queries, into L2: they are staged right after this row's last tile
        prefetch_rows(wn.b, x, 128, rg, rg + RW);
      }
      c8_row = 0.f;
      empty_row = true;
#pragma unroll
      for (int r = 0; r < RW; ++r) l_part[r] = 0.f;
      const int lim_min = p.causal ? w.L - p.q_len + r0 / p.h : INT_MAX;  // the tile's first row sees least
      for (int i = 0; i < w.ntiles; ++i) {
        const int gi = g0 + i;
        ok = wait(tc::smem_u32(&ctl.s_full[gi & 1]), uint32_t(gi >> 1) & 1u, abort);
        if (!ok) break;
        tc::tc_fence_after();
        const int64_t t_end = w.k0 + int64_t(i + 1) * kKvTile;
        const bool dead = t_end - kKvTile + x >= w.k1;  // this key is past the end
        const bool masked = t_end > w.k1 || t_end - 1 > int64_t(lim_min);
        float e[RW];
        uint32_t hi[RW / 4], lo[RW / 4];
        // e = t + c8, in log2 units; -inf where the row does not see the key
        auto logits = [&] {
          float s_lo[RW];
          const uint32_t ts = tmem + uint32_t((gi & 1) * C::kSCols + rg) + lane_off;
          tc::tmem_ld_cols<RW>(ts, e);
          tc::tmem_ld_cols<RW>(ts + uint32_t(NR), s_lo);
          tc::tmem_wait_ld();
#pragma unroll
          for (int r = 0; r < RW; r += 4) {
            const float4 sc = *reinterpret_cast<const float4*>(&ctl.scale[rg + r]);
            const float4 c8 = *reinterpret_cast<const float4*>(&ctl.c8[rg + r]);
            e[r] = fmaf(e[r] + s_lo[r], sc.x, c8.x);
            e[r + 1] = fmaf(e[r + 1] + s_lo[r + 1], sc.y, c8.y);
            e[r + 2] = fmaf(e[r + 2] + s_lo[r + 2], sc.z, c8.z);
            e[r + 3] = fmaf(e[r + 3] + s_lo[r + 3], sc.w, c8.w);
          }
          if (masked) {
            const int key = int(t_end) - kKvTile + x;
#pragma unroll
            for (int r = 0; r < RW; ++r)
              if (dead || key > ctl.lim[rg + r]) e[r] = -INFINITY;
          }
        };
        auto exps = [&] {
#pragma unroll
          for (int r = 0; r < RW; ++r) e[r] = fast_exp2(e[r]);
        };
        auto terms = [&] {  // of p = e
          const uint32_t dither = key_dither(uint32_t(t_end) - kKvTile + x);
#pragma unroll
          for (int r = 0; r < RW; r += 4) weight_terms(e + r, dither, hi[r / 4], lo[r / 4]);
        };
        // Rows whose reference moves (bits; the same in every thread of the
        // group). A later tile's weights are formed from the references as they
        // stand while the warps exchange which rows have weights above the limit
        // and by how many binades; where some do (few tiles), the references move
        // and the tile is done once more. A first tile, and a move too far for a
        // byte, start from the rows' maxima. (One copy of the code for all: code
        // that is seldom run comes from L2, some 25 cycles an instruction.)
        uint32_t moving = 0;
        enum { kCheck, kMaxima, kDone } phase = i == 0 ? kMaxima : kCheck;
#pragma unroll 1
        for (;;) {
          logits();
          if (phase == kCheck) {
            float m = e[0];
#pragma unroll
            for (int r = 1; r < RW; ++r) m = fmaxf(m, e[r]);
            uint32_t above = 0;
            if (__any_sync(0xFFFFFFFFu, m > kTop)) {
#pragma unroll
              for (int r = 0; r < RW; ++r) above |= e[r] > kTop ? 1u << r : 0u;
              above = __reduce_or_sync(0xFFFFFFFFu, above);
              const uint32_t ts = tmem + uint32_t((gi & 1) * C::kSCols + rg) + lane_off;
#pragma unroll 1
              for (uint32_t left = above; left; left &= left - 1) {
                const int r = __ffs(int(left)) - 1;
                const float s0 = tc::tmem_ld1(ts + uint32_t(r)), s1 = tc::tmem_ld1(ts + uint32_t(NR + r));
                tc::tmem_wait_ld();
                float v = fmaf(s0 + s1, ctl.scale[rg + r], ctl.c8[rg + r]);
                if (masked && (dead || int(t_end) - kKvTile + x > ctl.lim[rg + r])) v = -INFINITY;
                v = tc::redux_max(v) - kBaseSink;
                if (lane == 0) ctl.by[grp][xb & 1][qd][r] = uint8_t(fminf(ceilf(v), kFar));
              }
            }
            if (lane == 0) ctl.above[grp][xb & 1][qd] = above;
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(tc::smem_u32(&ctl.bound_bar[grp][xb & 1]));
          } else if (phase == kMaxima) {
            float tmp[RW];
#pragma unroll
            for (int r = 0; r < RW; ++r) tmp[r] = e[r];
            const float wm = reduce_rows<RW, true>(tmp, lane);
            if (lane % kShare == 0) ctl.red[grp][qd][lane / kShare] = wm;
            __syncwarp();
            const uint32_t bar = tc::smem_u32(&ctl.row_bar[grp]);
            if (lane == 0) tc::mbar_arrive(bar);
            ok = wait(bar, uint32_t(xr) & 1u, abort);
            if (!ok) break;
            ++xr;
            // lane r moves row r's reference (the four warps compute and store
            // the same values)
            bool moved = false;
            if (lane < RW) {
              const float m0 = ctl.red[grp][0][lane], m1 = ctl.red[grp][1][lane];
              const float m2 = ctl.red[grp][2][lane], m3 = ctl.red[grp][3][lane];
              const float em = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)), least = fminf(fminf(m0, m1), fminf(m2, m3));
              moved = em != -INFINITY && (i == 0 || em > kTop);
              const float d = moved ? em - (i == 0 && em - least <= kStandsOut ? kBase : kBaseSink) : 0.f;
              // (by the mask, not by em: NaN logits beside masked keys leave em at -inf too)
              if (i == 0) empty_row = int64_t(ctl.lim[rg + lane]) < w.k0;
              c8_row -= d;
              ctl.c8[rg + lane] = c8_row;
              ctl.move[rg + lane] = i == 0 ? d : fast_exp2(-d);
            }
            moving = __ballot_sync(0xFFFFFFFFu, moved);
            __syncwarp();
            phase = kDone;
            if (i > 0) continue;
#pragma unroll
            for (int r = 0; r < RW; r += 4) {
              const float4 sh = *reinterpret_cast<const float4*>(&ctl.move[rg + r]);
              e[r] -= sh.x;
              e[r + 1] -= sh.y;
              e[r + 2] -= sh.z;
              e[r + 3] -= sh.w;
            }
          }
          exps();
          terms();
          if (phase == kDone) break;
          ok = wait(tc::smem_u32(&ctl.bound_bar[grp][xb & 1]), uint32_t(xb >> 1) & 1u, abort);
          if (!ok) break;
          const uint4 b = *reinterpret_cast<const uint4*>(&ctl.above[grp][xb & 1][0]);
          moving = (b.x | b.y) | (b.z | b.w);
          if (!moving) {
            ++xb;
            break;
          }
          int d = 0;
          if (lane < RW) {
            if (b.x >> lane & 1u) d = max(d, int(ctl.by[grp][xb & 1][0][lane]));
            if (b.y >> lane & 1u) d = max(d, int(ctl.by[grp][xb & 1][1][lane]));
            if (b.z >> lane & 1u) d = max(d, int(ctl.by[grp][xb & 1][2][lane]));
            if (b.w >> lane & 1u) d = max(d, int(ctl.by[grp][xb & 1][3][lane]));
          }
          ++xb;
          phase = kDone;
          if (__any_sync(0xFFFFFFFFu, d >= int(kFar))) {
            phase = kMaxima;
          } else {
            if (lane < RW) {
              c8_row -= float(d);
              ctl.c8[rg + lane] = c8_row;
              ctl.move[rg + lane] = __int_as_float((127 - d) << 23);  // 2^-d
            }
            __syncwarp();
          }
        }
        if (!ok) break;
        const bool rescale = i > 0 && moving != 0;
        if (rescale) {
#pragma unroll
          for (int r = 0; r < RW; ++r) l_part[r] *= ctl.move[rg + r];
        }
#pragma unroll
        for (int r = 0; r < RW; ++r) l_part[r] += e[r];
        // the P buffer is free, and O complete up to the tile before, once
        // that product is done
        if (gi >= C::kPBufs) {
          const int pi = rescale ? gi - 1 : gi - C::kPBufs;
          ok = wait(tc::smem_u32(&ctl.o_full[pi & 1]), uint32_t(pi >> 1) & 1u, abort);
          if (!ok) break;
        } else if (rescale) {
          ok = wait(tc::smem_u32(&ctl.o_full[(gi - 1) & 1]), uint32_t((gi - 1) >> 1) & 1u, abort);
          if (!ok) break;
        }
        uint8_t* pt = smem + C::kOffP + (gi % C::kPBufs) * C::kPBytes + x * 16;
#pragma unroll
        for (int k = 0; k < RW / 16; ++k) {
          const int blk = (rg / 16 + k) * 2048;
          *reinterpret_cast<uint4*>(pt + blk) = make_uint4(hi[4 * k], hi[4 * k + 1], hi[4 * k + 2], hi[4 * k + 3]);
          *reinterpret_cast<uint4*>(pt + NR * 128 + blk) = make_uint4(lo[4 * k], lo[4 * k + 1], lo[4 * k + 2], lo[4 * k + 3]);
        }
        if (dead) {
          // value rows past the end: their weights are 0, but the bytes may be
          // NaN codes. QK has read the tile (s_full), PV waits for p_full.
#pragma unroll
          for (int j = 0; j < 4 / G; ++j) {
            const int s = (4 * gi + grp * (4 / G) + j) % C::kRing;
            uint4* z = reinterpret_cast<uint4*>(smem + s * kSub + x * 128);
#pragma unroll
            for (int k = 0; k < 8; ++k) z[k] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        if (rescale) {
          tc::tc_fence_after();
          for (uint32_t left = moving; left; left &= left - 1) {
            const int r = __ffs(int(left)) - 1;
            const uint32_t at = tO + uint32_t(rg + r) + lane_off;
            const float f = ctl.move[rg + r];
            float v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = tc::tmem_ld1(at + uint32_t(j * NR));
            tc::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 4; ++j) tc::tmem_st1(at + uint32_t(j * NR), v[j] * f);
          }
          tc::tmem_wait_st();
        }
        tc::fence_async_smem();
        tc::tc_fence_before();
        tc::mbar_arrive(tc::smem_u32(&ctl.p_full[gi & 1]));
      }
      if (!ok) break;
      g0 += w.ntiles;
    }
  }

  // ---- teardown ----------------------------------------------------------------
  __syncthreads();
  if (*abort && tid == 0) atomicOr(p.status, kStatusTimeout);
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, C::kTmemCols);
  }
}

// 3-D byte tensor (row, token, page) of the cache; a box is `width` bytes of a page's tokens.
bool encode_map(CUtensorMap* map, const LatentParams& p, int width, CUtensorMapSwizzle swizzle) {
  auto fn = tensor_map_encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {cuuint64_t(kRow), cuuint64_t(p.page_size), cuuint64_t(p.num_pages)};
  const cuuint64_t strides[2] = {cuuint64_t(p.stride_token), cuuint64_t(p.stride_page)};
  const cuuint32_t box[3] = {cuuint32_t(width), cuuint32_t(p.page_size), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(p.cache), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NR>
cudaError_t launch(const CUtensorMap& ml, const CUtensorMap& mr, const LatentParams& p, cudaStream_t stream) {
  constexpr int bytes = smem_bytes<NR>();
  static std::atomic<bool> configured[64];  // the shared-memory limit is raised once per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(latent_kernel<NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    configured[dev].store(true, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(p.slots) * unsigned(p.n_row_tiles));
  cfg.blockDim = dim3(Cfg<NR>::kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, latent_kernel<NR>, ml, mr, p);
}

}  // namespace

cudaError_t launch_latent(const LatentParams& p, cudaStream_t stream) {
  CUtensorMap ml, mr;
  if (!encode_map(&ml, p, 128, CU_TENSOR_MAP_SWIZZLE_128B) || !encode_map(&mr, p, 64, CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  switch (p.row_tile) {
    case 16: return launch<16>(ml, mr, p, stream);
    case 32: return launch<32>(ml, mr, p, stream);
    default: return launch<64>(ml, mr, p, stream);
  }
}

}  // namespace mj
