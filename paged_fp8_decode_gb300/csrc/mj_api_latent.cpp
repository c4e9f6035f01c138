// Host side of the rotated cache writes and the latent-cache attention
// (include/mj.h): argument checks, the rotation's turns, the latent plan, the
// workspace layout and the launches. Nothing here allocates, synchronises or
// reads device memory.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "mj_latent.h"

namespace {

using mj::rows_apart;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int status_of(cudaError_t e) { return e == cudaSuccess ? MJ_OK : MJ_ERR_CUDA; }

bool page_size_ok(int ps) { return ps == 16 || ps == 32 || ps == 64 || ps == 128; }

// A plan's cost of a work row beside its tiles, in tiles: staging the queries,
// refilling the pipeline, writing the rows out and joining them (a row of an
// unsplit request has no partial to join, but is charged alike). Fitted, each to
// one batch, not derived; in us:
// 64 x 4096 tokens, 16 heads: 35.8, 34.5, 35.7 at 0, 1, 2; 96 requests of 300 to
// 5000 tokens, 32 heads: 55.2, 49.8, 48.8, 50.6 at 1, 2, 3, 6; 48 of 1024 to
// 16384, 128 heads: 136, 125, 116, 121 at 1, 2, 5, 9.
constexpr int kCost16 = 1, kCost32 = 3, kCost64 = 5;

// The writes' kernel indexes tokens, rounded up to whole CTAs, with 32 bits.
constexpr int kMaxTokens = 1 << 30;

// Query rows of a request (its partials' sizes stay far inside 64 bits).
constexpr int64_t kMaxRows = 1 << 20;

int latent_row_tile(int64_t n_q) { return n_q <= 16 ? 16 : (n_q <= 32 ? 32 : 64); }

int check_rope(const mj_rope& r, int d) {
  if (r.num_axes < 1 || r.num_axes > 4 || r.axis_stride < 0) return MJ_ERR_INVALID_ARG;
  if (r.rot_dim < 16 || r.rot_dim > d || r.rot_dim % 16) return MJ_ERR_UNSUPPORTED;
  if (!std::isfinite(r.scale)) return MJ_ERR_INVALID_ARG;
  if (!r.positions || !r.turns || (r.num_axes > 1 && !r.freq_axis)) return MJ_ERR_INVALID_ARG;
  if (!aligned(r.positions, 8) || !aligned(r.turns, 8)) return MJ_ERR_ALIGNMENT;
  return MJ_OK;
}

// The query part of a write: h heads of d channels in, h heads out.
int check_query(int T, int h, int d, const void* q, const void* q_out, int64_t ts, int64_t hs, int64_t ots, int64_t ohs) {
  if (h < 0) return MJ_ERR_INVALID_ARG;
  if (h == 0) return MJ_OK;
  if (!q || !q_out || ts < 0 || hs < 0 || ots < 0 || ohs < 0) return MJ_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(q_out, 16) || ts % 8 || hs % 8 || ots % 8 || ohs % 8) return MJ_ERR_ALIGNMENT;
  if (!rows_apart(d, {{ots, T}, {ohs, h}})) return MJ_ERR_INVALID_ARG;
  if (q == q_out && ((T > 1 && ts != ots) || (h > 1 && hs != ohs))) return MJ_ERR_INVALID_ARG;
  return MJ_OK;
}

}  // namespace

extern "C" {

int mj_rope_turns(const double* inv_freq, int n, uint64_t* turns) {
  if (n < 0 || (n > 0 && (!inv_freq || !turns))) return MJ_ERR_INVALID_ARG;
  // 1 / (2 pi) = 0.1591549430918953357688837633725143620344596457404564...,
  // its first 192 fraction bits, highest word first
  const uint64_t r[3] = {0x28be60db9391054aull, 0x7f09d5f47d4d3770ull, 0x36d8a5664f10e410ull};
  for (int i = 0; i < n; ++i)
    if (!std::isfinite(inv_freq[i]) || std::fabs(inv_freq[i]) > 1048576.0) return MJ_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    int e = 0;
    const double f = std::frexp(std::fabs(inv_freq[i]), &e);  // |inv_freq| = f 2^e, f in [1/2, 1)
    const uint64_t m = uint64_t(std::ldexp(f, 53));           // = m 2^(e - 53), exactly
    // the product m * r as 256 bits, lowest word first: |inv_freq| / (2 pi) = P 2^(e - 53 - 192)
    uint64_t P[4];
    unsigned __int128 c = 0;
    for (int k = 0; k < 3; ++k) {
      c += static_cast<unsigned __int128>(m) * r[2 - k];
      P[k] = uint64_t(c);
      c >>= 64;
    }
    P[3] = uint64_t(c);
    // turns = round(P 2^(e - 53 - 192 + 64)) modulo 2^64: a right shift by s bits
    const int s = 181 - e;  // e <= 21, so at least 160
    uint64_t t = 0;
    if (s <= 256) {
      auto bits = [&](int at) -> uint64_t {  // 64 bits of P from bit `at` up (zeros above 255)
        const int w = at >> 6, sh = at & 63;
        const uint64_t lo = w < 4 ? P[w] >> sh : 0;
        const uint64_t hi = sh && w + 1 < 4 ? P[w + 1] << (64 - sh) : 0;
        return lo | hi;
      };
      t = bits(s) + ((bits(s - 1)) & 1u);  // to nearest, halves up
    }
    turns[i] = std::signbit(inv_freq[i]) ? 0 - t : t;
  }
  return MJ_OK;
}

int mj_rope_write_kv(const mj_rope_write_kv_args* a, void* stream) {
  const mj::NvtxRange range("mj_rope_write_kv");
  if (!a) return MJ_ERR_INVALID_ARG;
  if (a->kv.num_tokens > kMaxTokens) return MJ_ERR_CAPACITY;
  int st = mj::check_write_kv(&a->kv);
  if (st != MJ_OK || a->kv.num_tokens == 0) return st;
  st = check_rope(a->rope, a->kv.d);
  if (st != MJ_OK) return st;
  st = check_query(a->kv.num_tokens, a->h_q, a->kv.d, a->q, a->q_out, a->q_tok_stride, a->q_head_stride,
                   a->q_out_tok_stride, a->q_out_head_stride);
  if (st != MJ_OK) return st;
  const mj_write_kv_args& w = a->kv;
  if ((int64_t(a->h_q) + 2 * int64_t(w.h_k)) * w.d > (int64_t(1) << 24)) return MJ_ERR_INVALID_ARG;
  const int64_t row = mj::kv_row_bytes(w.kv_format, w.d);
  if (!rows_apart(row, {{w.k_stride_page, w.num_pages}, {w.k_stride_token, w.page_size}, {w.k_stride_head, w.h_k}}) ||
      !rows_apart(row, {{w.v_stride_page, w.num_pages}, {w.v_stride_token, w.page_size}, {w.v_stride_head, w.h_k}}))
    return MJ_ERR_INVALID_ARG;
  return status_of(mj::launch_rope_write(*a, static_cast<cudaStream_t>(stream)));
}

int mj_latent_write(const mj_latent_write_args* a, void* stream) {
  const mj::NvtxRange range("mj_latent_write");
  if (!a) return MJ_ERR_INVALID_ARG;
  if (a->num_tokens < 0 || a->num_pages < 0) return MJ_ERR_INVALID_ARG;
  if (a->num_tokens > kMaxTokens) return MJ_ERR_CAPACITY;
  if (!page_size_ok(a->page_size)) return MJ_ERR_UNSUPPORTED;
  if (a->num_tokens == 0) return MJ_OK;
  int st = check_rope(a->rope, MJ_LATENT_ROPE_DIM);
  if (st != MJ_OK) return st;
  st = check_query(a->num_tokens, a->h, MJ_LATENT_ROPE_DIM, a->q_pe, a->q_out, a->q_tok_stride, a->q_head_stride,
                   a->q_out_tok_stride, a->q_out_head_stride);
  if (st != MJ_OK) return st;
  if (a->h > (1 << 16)) return MJ_ERR_INVALID_ARG;
  if (!a->latent || !a->k_pe || !a->slot_mapping || !a->cache || !a->scale) return MJ_ERR_INVALID_ARG;
  if (a->latent_tok_stride < 0 || a->k_pe_tok_stride < 0 || a->stride_page < MJ_LATENT_ROW_BYTES ||
      a->stride_token < MJ_LATENT_ROW_BYTES)
    return MJ_ERR_INVALID_ARG;
  if (!aligned(a->latent, 16) || !aligned(a->k_pe, 16) || !aligned(a->cache, 16) || !aligned(a->slot_mapping, 8) ||
      !aligned(a->scale, 4) || (a->status && !aligned(a->status, 4)))
    return MJ_ERR_ALIGNMENT;
  if (a->latent_tok_stride % 8 || a->k_pe_tok_stride % 8 || a->stride_page % 16 || a->stride_token % 16)
    return MJ_ERR_ALIGNMENT;
  if (!rows_apart(MJ_LATENT_ROW_BYTES, {{a->stride_page, a->num_pages}, {a->stride_token, a->page_size}}))
    return MJ_ERR_INVALID_ARG;
  return status_of(mj::launch_latent_write(*a, static_cast<cudaStream_t>(stream)));
}

int mj_latent_slots(int sm_count, int q_len, int h) {
  if (sm_count < 1 || q_len < 1 || h < 1) return 1;
  const int64_t n_q = int64_t(q_len) * h;
  const int64_t tile = latent_row_tile(n_q);
  return int(std::max<int64_t>(1, sm_count / ((n_q + tile - 1) / tile)));
}

int mj_latent_plan_size(int slots, int max_num_seqs, size_t* words) {
  if (!words || slots < 1 || max_num_seqs < 0) return MJ_ERR_INVALID_ARG;
  *words = size_t(mj::latent_plan_slot_words(slots) + mj::latent_plan_split_words(max_num_seqs) +
                  4 * mj::latent_plan_max_work(slots, max_num_seqs) + mj::latent_plan_tile_words(max_num_seqs));
  return MJ_OK;
}

int mj_latent_plan(const int32_t* seq_lens_host, int num_seqs, int max_num_seqs, int slots, int q_len, int h,
                   int margin, int32_t* plan_host, size_t plan_words) {
  const mj::NvtxRange range("mj_latent_plan");
  if (num_seqs < 0 || max_num_seqs < num_seqs || slots < 1 || q_len < 1 || h < 1 || margin < 0 || !plan_host ||
      (num_seqs > 0 && !seq_lens_host))
    return MJ_ERR_INVALID_ARG;
  size_t need = 0;
  const int st = mj_latent_plan_size(slots, max_num_seqs, &need);
  if (st != MJ_OK) return st;
  if (plan_words < need) return MJ_ERR_CAPACITY;
  const int tile = latent_row_tile(int64_t(q_len) * h);
  const int row_cost = tile == 16 ? kCost16 : (tile == 32 ? kCost32 : kCost64), least = std::min(row_cost, 3);
  int64_t total = 0;
  for (int b = 0; b < num_seqs; ++b) {
    if (seq_lens_host[b] < 0 || int64_t(seq_lens_host[b]) + margin > INT32_MAX) return MJ_ERR_INVALID_ARG;
    total += (int64_t(seq_lens_host[b]) + margin + mj::kKvTile - 1) / mj::kKvTile + row_cost;
  }
  auto tiles = [&](int b) -> int64_t {  // a padding request has none
    return seq_lens_host[b] > 0 ? (int64_t(seq_lens_host[b]) + margin + mj::kKvTile - 1) / mj::kKvTile : 0;
  };
  std::memset(plan_host, 0, need * sizeof(int32_t));
  int32_t* table = plan_host;
  int32_t* splits = table + mj::latent_plan_slot_words(slots);
  int32_t* work = splits + mj::latent_plan_split_words(max_num_seqs);
  int32_t* planned = work + 4 * mj::latent_plan_max_work(slots, max_num_seqs);
  for (int b = 0; b < num_seqs; ++b) planned[b] = int32_t(tiles(b));

  // The requests' tiles in order, cut so that no slot's cost (its tiles, and
  // row_cost for each of its rows) exceeds `limit`; false when that takes more
  // slots than there are. With `write`, the plan.
  auto cut = [&](int64_t limit, bool write) {
    int slot = 0, rows = 0, parts = 0;
    int64_t used = 0;
    for (int b = 0; b < num_seqs; ++b) {
      const int64_t t = tiles(b);
      int64_t at = 0;
      const int first_row = rows, first_part = parts;
      while (at < t) {
        // no room for a row here, or for so few tiles only that starting it costs more
        if (used > 0 && used + row_cost + std::min<int64_t>(t - at, least) > limit) {
          if (++slot >= slots) return false;
          used = 0;
        }
        const int64_t take = std::min(t - at, limit - used - row_cost);
        if (write) {
          int32_t* w = work + 4 * int64_t(rows);
          w[0] = b;
          w[1] = int32_t(at);
          w[2] = int32_t(at + take);
          w[3] = -1;
          int32_t* e = table + 4 * int64_t(slot);
          if (used == 0) {  // the slot's first row
            e[0] = rows;
            e[2] = w[0];
            e[3] = w[1];
          }
          e[1] = rows + 1;
        }
        ++rows;
        at += take;
        used += take + row_cost;
      }
      if (rows - first_row > 1) {
        if (write) {
          for (int r = first_row; r < rows; ++r) work[4 * int64_t(r) + 3] = first_part + (r - first_row);
          splits[2 * int64_t(b)] = first_part;
          splits[2 * int64_t(b) + 1] = rows - first_row;
        }
        parts += rows - first_row;
      }
    }
    return true;
  };
  int64_t lo = row_cost + 1, hi = std::max<int64_t>(lo, total);  // one slot holds everything at `total`
  while (lo < hi) {
    const int64_t mid = lo + (hi - lo) / 2;
    if (cut(mid, false))
      hi = mid;
    else
      lo = mid + 1;
  }
  cut(lo, true);
  return MJ_OK;
}

int mj_latent_workspace_size(int slots, int q_len, int h, size_t* bytes) {
  if (!bytes || slots < 1 || q_len < 1 || h < 1 || int64_t(q_len) * h > kMaxRows) return MJ_ERR_INVALID_ARG;
  const int64_t tile = latent_row_tile(int64_t(q_len) * h);
  const int64_t rows = (int64_t(q_len) * h + tile - 1) / tile * tile;
  *bytes = mj::kWsHeader + size_t(2) * slots * size_t(rows) * (MJ_LATENT_DIM + 2) * sizeof(float);
  return MJ_OK;
}

int mj_latent_attention(const mj_latent_args* a, void* stream) {
  const mj::NvtxRange range("mj_latent_attention");
  if (!a) return MJ_ERR_INVALID_ARG;
  if (a->num_seqs < 0 || a->max_num_seqs < a->num_seqs || a->q_len < 1 || a->h < 1 || a->slots < 1)
    return MJ_ERR_INVALID_ARG;
  if (!page_size_ok(a->page_size)) return MJ_ERR_UNSUPPORTED;
  if (a->num_pages < 1 || a->num_pages > INT32_MAX || a->block_table_stride < 0 || a->block_table_len < 0)
    return MJ_ERR_INVALID_ARG;
  if (!(a->softmax_scale > 0.f) || !std::isfinite(a->softmax_scale)) return MJ_ERR_INVALID_ARG;
  if (a->out_dtype != MJ_OUT_BF16 && a->out_dtype != MJ_OUT_F16) return MJ_ERR_UNSUPPORTED;
  const int64_t n_q = int64_t(a->q_len) * a->h;
  if (n_q > kMaxRows) return MJ_ERR_INVALID_ARG;
  const void* need[] = {a->q, a->cache, a->descale, a->block_table, a->seq_lens, a->plan, a->out, a->workspace};
  for (const void* ptr : need)
    if (!ptr) return MJ_ERR_INVALID_ARG;
  const int64_t strides[] = {a->q_tok_stride, a->q_head_stride, a->out_tok_stride, a->out_head_stride,
                             a->stride_page, a->stride_token};
  for (int64_t s : strides)
    if (s < 0) return MJ_ERR_INVALID_ARG;
  if (a->stride_token < MJ_LATENT_ROW_BYTES || a->stride_page < MJ_LATENT_ROW_BYTES) return MJ_ERR_INVALID_ARG;
  const void* a16[] = {a->q, a->cache, a->block_table, a->seq_lens, a->plan, a->out, a->workspace};
  for (const void* ptr : a16)
    if (!aligned(ptr, 16)) return MJ_ERR_ALIGNMENT;
  if (!aligned(a->descale, 4) || (a->lse && !aligned(a->lse, 4))) return MJ_ERR_ALIGNMENT;
  for (int k = 0; k < 4; ++k)
    if (strides[k] % 8) return MJ_ERR_ALIGNMENT;
  if (a->stride_page % 16 || a->stride_token % 16) return MJ_ERR_ALIGNMENT;
  if (!rows_apart(MJ_LATENT_DIM, {{a->out_tok_stride, int64_t(a->num_seqs) * a->q_len}, {a->out_head_stride, a->h}}))
    return MJ_ERR_INVALID_ARG;
  size_t bytes = 0;
  const int st = mj_latent_workspace_size(a->slots, a->q_len, a->h, &bytes);
  if (st != MJ_OK) return st;
  if (a->workspace_bytes < bytes) return MJ_ERR_CAPACITY;

  mj::LatentParams p = {};
  p.num_seqs = a->num_seqs;
  p.q_len = a->q_len;
  p.h = a->h;
  p.n_q = int(n_q);
  p.causal = a->causal ? 1 : 0;
  p.row_tile = latent_row_tile(n_q);
  p.n_row_tiles = int((n_q + p.row_tile - 1) / p.row_tile);
  if (int64_t(a->slots) * p.n_row_tiles > INT32_MAX) return MJ_ERR_INVALID_ARG;
  p.softmax_scale = a->softmax_scale;
  p.q = static_cast<const uint16_t*>(a->q);
  p.q_ts = a->q_tok_stride;
  p.q_hs = a->q_head_stride;
  p.cache = static_cast<const uint8_t*>(a->cache);
  p.stride_page = a->stride_page;
  p.stride_token = a->stride_token;
  p.page_size = a->page_size;
  p.page_shift = mj::page_shift(a->page_size);
  p.page_span = a->stride_token <= 2 * MJ_LATENT_ROW_BYTES
                    ? uint32_t((a->page_size - 1) * a->stride_token + MJ_LATENT_ROW_BYTES)
                    : 0;
  p.num_pages = a->num_pages;
  p.descale = a->descale;
  p.block_table = a->block_table;
  p.bt_stride = a->block_table_stride;
  p.bt_len = a->block_table_len;
  p.seq_lens = a->seq_lens;
  p.slots = a->slots;
  const int64_t max_work = mj::latent_plan_max_work(a->slots, a->max_num_seqs);
  if (max_work > INT32_MAX) return MJ_ERR_INVALID_ARG;
  p.max_work = int(max_work);
  p.slot_table = a->plan;
  p.splits = p.slot_table + mj::latent_plan_slot_words(a->slots);
  p.work = p.splits + mj::latent_plan_split_words(a->max_num_seqs);
  p.planned = p.work + 4 * max_work;
  p.out = static_cast<uint16_t*>(a->out);
  p.out_f16 = a->out_dtype == MJ_OUT_F16 ? 1 : 0;
  p.out_ts = a->out_tok_stride;
  p.out_hs = a->out_head_stride;
  p.lse = a->lse;
  char* ws = static_cast<char*>(a->workspace);
  p.status = reinterpret_cast<uint32_t*>(ws);
  const int64_t rows = 2 * int64_t(a->slots) * p.n_row_tiles * p.row_tile;
  p.o_part = reinterpret_cast<float*>(ws + mj::kWsHeader);
  p.m_part = p.o_part + rows * MJ_LATENT_DIM;
  p.l_part = p.m_part + rows;
  // with several row tiles the tiles' CTAs read the same cache rows: keep them in L2
  p.evict_first = a->evict_first && p.n_row_tiles == 1 ? 1 : 0;
  if (a->num_seqs == 0) return MJ_OK;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int e = status_of(mj::launch_latent(p, s));
  return e != MJ_OK ? e : status_of(mj::launch_latent_merge(p, s));
}

}  // extern "C"
