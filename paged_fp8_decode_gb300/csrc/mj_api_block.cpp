// Host side of the block-scaled cache's calls (include/mj.h): argument checks,
// the plan, the workspace layouts and the launches. Nothing here allocates,
// synchronises or reads device memory.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "mj_block.h"
#include "mj_latent.h"

namespace {

using mj::rows_apart;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int status_of(cudaError_t e) { return e == cudaSuccess ? MJ_OK : MJ_ERR_CUDA; }

bool size_ok(int n) { return n == 16 || n == 32 || n == 64 || n == 128; }

constexpr int kMaxTokens = 1 << 30;
// The least keys of a prompt's piece worth a CTA of its own. (64 tokens after 2000, 32/8 heads of 128: 1024
// 28.7 us, 512 23.0, 320 19.8, 192 19.5; 4 chunks of 20 after 500: 12.3, 12.3, 12.6, 16.3.)
constexpr int64_t kPromptMinKeys = 320;
constexpr int64_t kMaxRows = 1 << 20;  // query rows of a request and KV head; of a prompt, heads of a KV head

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The cache of a call. written: its rows and exponent bytes must lie apart.
int check_cache(const mj_block_cache& c, bool written) {
  if (c.h_k < 1 || c.num_pages < 1) return MJ_ERR_INVALID_ARG;
  if (!mj::head_dim_ok(c.d) || !size_ok(c.page_size) || !size_ok(c.block)) return MJ_ERR_UNSUPPORTED;
  if (c.block > c.page_size) return MJ_ERR_INVALID_ARG;
  if (c.h_k > 65535 || c.num_pages > INT32_MAX) return MJ_ERR_UNSUPPORTED;
  if (!c.k_cache || !c.v_cache || !c.k_exp || !c.v_exp) return MJ_ERR_INVALID_ARG;
  const int64_t st[] = {c.k_stride_page, c.k_stride_token, c.k_stride_head, c.v_stride_page, c.v_stride_token, c.v_stride_head};
  for (int64_t s : st)
    if (s < 0) return MJ_ERR_INVALID_ARG;
  if (c.k_exp_stride_page < 0 || c.k_exp_stride_head < 0 || c.v_exp_stride_page < 0 || c.v_exp_stride_head < 0)
    return MJ_ERR_INVALID_ARG;
  for (int64_t s : st)
    if (s % 16) return MJ_ERR_ALIGNMENT;
  if (!aligned(c.k_cache, 16) || !aligned(c.v_cache, 16)) return MJ_ERR_ALIGNMENT;
  if (written) {
    const int64_t blocks = c.page_size / c.block;
    if (!rows_apart(c.d, {{c.k_stride_page, c.num_pages}, {c.k_stride_token, c.page_size}, {c.k_stride_head, c.h_k}}) ||
        !rows_apart(c.d, {{c.v_stride_page, c.num_pages}, {c.v_stride_token, c.page_size}, {c.v_stride_head, c.h_k}}) ||
        !rows_apart(blocks, {{c.k_exp_stride_page, c.num_pages}, {c.k_exp_stride_head, c.h_k}}) ||
        !rows_apart(blocks, {{c.v_exp_stride_page, c.num_pages}, {c.v_exp_stride_head, c.h_k}}))
      return MJ_ERR_INVALID_ARG;
  }
  return MJ_OK;
}

// bf16 rows of d channels at element strides: (t, h, c) for T tokens and H heads.
int check_rows(const void* p, int64_t ts, int64_t hs) {
  if (!p || ts < 0 || hs < 0) return MJ_ERR_INVALID_ARG;
  return !aligned(p, 16) || ts % 8 || hs % 8 ? MJ_ERR_ALIGNMENT : MJ_OK;
}

int check_table(const int32_t* table, int64_t stride, int64_t len) {
  return !table || stride < 0 || len < 0 ? MJ_ERR_INVALID_ARG : (aligned(table, 4) ? MJ_OK : MJ_ERR_ALIGNMENT);
}

// The two sides. (One head's own stride is of no use: K's and V's may differ in it, and stand in any order to
// their tokens' strides, which the attentions want alike.)
void sides(const mj_block_cache& c, mj::BlockSide (&s)[2]) {
  s[0] = {static_cast<uint8_t*>(c.k_cache), c.k_stride_page, c.k_stride_token, c.k_stride_head, c.k_exp, c.k_exp_stride_page,
          c.k_exp_stride_head};
  s[1] = {static_cast<uint8_t*>(c.v_cache), c.v_stride_page, c.v_stride_token, c.v_stride_head, c.v_exp, c.v_exp_stride_page,
          c.v_exp_stride_head};
  for (mj::BlockSide& x : s)
    if (c.h_k == 1) x.sh = x.st;
}

// A plan has at most a piece a slot and one a request (each launch has a CTA for every
// row that there could be), and a piece at least half a slot's share of all tiles: of
// split requests, over one piece each, at most four a slot.
int64_t work_rows(int slots, int max_num_seqs) { return int64_t(slots) + max_num_seqs; }
int64_t part_cap(int slots) { return 4 * int64_t(slots); }

// What starting, ending and joining a piece costs, in tiles, and how much of the
// longest piece the slots that end early wait for the last one. Of 16 batches (1 to 100
// requests, ragged and equal, 4 to 32 query rows, both head sizes) none is slower at 4 to 6 and 0.3 to
// 0.5; at (4, 0.2) 13 requests of 1000 to 60000 tokens take 197 us in place of 157, at (2, 0.2) 20 of
// 100 to 20000 108 in place of 84, at (4, 0.6) 100 of 100 to 3000 66 in place of 59.
constexpr double kPieceTiles = 5, kTail = 0.4;

// Which kernel attends: the decode kernel (keys on the tensor cores' rows, so that a few
// query rows fill them) or the prompt's (query rows there, up to 32 of them four times over). In us, the decode
// kernel's time first, where both were built, pages of 32: head size 128, 64 x 4096 tokens, 8 KV heads: 8 rows 103 and
// 133, 16 rows 184 and 133; head size 256, 4 KV heads: 8 rows 95 and 125, 12 rows 125 and 125, 16 rows 137
// and 126; 16 rows, 1 x 65536 tokens, 37 and 21, 40 ragged requests 181 and 133.
bool by_rows(int64_t n_q) { return n_q > 8; }

bool slots_ok(int slots) { return slots >= 1 && slots <= (1 << 20); }

}  // namespace

extern "C" {

int mj_block_write_kv(const mj_block_write_args* a, void* stream) {
  const mj::NvtxRange range("mj_block_write_kv");
  if (!a || a->num_tokens < 0) return MJ_ERR_INVALID_ARG;
  if (a->num_tokens > kMaxTokens) return MJ_ERR_CAPACITY;
  int st = check_cache(a->cache, true);
  if (st != MJ_OK || a->num_tokens == 0) return st;
  st = check_rows(a->key, a->key_tok_stride, a->key_head_stride);
  if (st == MJ_OK) st = check_rows(a->value, a->value_tok_stride, a->value_head_stride);
  if (st != MJ_OK) return st;
  if (!a->slot_mapping) return MJ_ERR_INVALID_ARG;
  if (!aligned(a->slot_mapping, 8) || !aligned(a->status, 4)) return MJ_ERR_ALIGNMENT;
  mj::BlockWriteParams p = {};
  p.num_tokens = a->num_tokens;
  p.h_k = a->cache.h_k;
  p.in[0] = static_cast<const uint16_t*>(a->key);
  p.in[1] = static_cast<const uint16_t*>(a->value);
  p.ts[0] = a->key_tok_stride;
  p.hs[0] = a->key_head_stride;
  p.ts[1] = a->value_tok_stride;
  p.hs[1] = a->value_head_stride;
  p.slots = a->slot_mapping;
  p.num_slots = a->cache.num_pages * a->cache.page_size;
  p.page_shift = mj::page_shift(a->cache.page_size);
  p.block_shift = mj::page_shift(a->cache.block);
  sides(a->cache, p.side);
  p.status = a->status;
  return status_of(mj::launch_block_write(p, a->cache.d, static_cast<cudaStream_t>(stream)));
}

int mj_block_read_kv(const mj_block_read_args* a, void* stream) {
  const mj::NvtxRange range("mj_block_read_kv");
  if (!a || a->num_seqs < 0 || a->num_rows < 0) return MJ_ERR_INVALID_ARG;
  if (a->num_rows > kMaxTokens) return MJ_ERR_CAPACITY;
  int st = check_cache(a->cache, false);
  if (st != MJ_OK) return st;
  if (a->out_dtype != MJ_OUT_BF16 && a->out_dtype != MJ_OUT_F16) return MJ_ERR_UNSUPPORTED;
  if (a->num_rows == 0 || a->num_seqs == 0) return MJ_OK;
  if (!a->starts || (!a->k_out && !a->v_out)) return MJ_ERR_INVALID_ARG;
  st = check_table(a->block_table, a->block_table_stride, a->block_table_len);
  const mj_block_cache& c = a->cache;
  if (st == MJ_OK && a->k_out) st = check_rows(a->k_out, a->k_tok_stride, a->k_head_stride);
  if (st == MJ_OK && a->v_out) st = check_rows(a->v_out, a->v_tok_stride, a->v_head_stride);
  if (st != MJ_OK) return st;
  if ((a->k_out && !rows_apart(c.d, {{a->k_tok_stride, a->num_rows}, {a->k_head_stride, c.h_k}})) ||
      (a->v_out && !rows_apart(c.d, {{a->v_tok_stride, a->num_rows}, {a->v_head_stride, c.h_k}})))
    return MJ_ERR_INVALID_ARG;
  if (!aligned(a->starts, 4) || !aligned(a->first, 4) || !aligned(a->status, 4)) return MJ_ERR_ALIGNMENT;
  mj::BlockReadParams p = {};
  p.num_seqs = a->num_seqs;
  p.num_rows = a->num_rows;
  p.h_k = c.h_k;
  p.page_shift = mj::page_shift(c.page_size);
  p.block_shift = mj::page_shift(c.block);
  p.num_pages = c.num_pages;
  sides(c, p.side);
  p.block_table = a->block_table;
  p.bt_stride = a->block_table_stride;
  p.bt_len = a->block_table_len;
  p.starts = a->starts;
  p.first = a->first;
  p.out[0] = static_cast<uint16_t*>(a->k_out);
  p.out[1] = static_cast<uint16_t*>(a->v_out);
  p.ts[0] = a->k_tok_stride;
  p.hs[0] = a->k_head_stride;
  p.ts[1] = a->v_tok_stride;
  p.hs[1] = a->v_head_stride;
  p.out_f16 = a->out_dtype == MJ_OUT_F16 ? 1 : 0;
  p.sides = (a->k_out ? 1 : 0) + (a->v_out ? 1 : 0);
  p.side0 = a->k_out ? 0 : 1;
  p.status = a->status;
  return status_of(mj::launch_block_read(p, c.d, static_cast<cudaStream_t>(stream)));
}

int mj_block_slots(int sm_count, int q_len, int h_q, int h_k, int d) {
  if (sm_count < 1 || q_len < 1 || h_k < 1 || h_q < h_k || h_q % h_k || !mj::head_dim_ok(d)) return 1;
  const int64_t n_q = int64_t(q_len) * (h_q / h_k);
  if (!by_rows(n_q)) return mj_slots(sm_count, 2, h_k, q_len, h_q);
  const int64_t tiles = ceil_div(n_q, mj::block_prompt_rows(d, n_q));
  return int(std::max<int64_t>(1, sm_count / (h_k * tiles)));
}

int mj_block_plan_size(int slots, int max_num_seqs, size_t* words) {
  if (!words || !slots_ok(slots) || max_num_seqs < 0 || max_num_seqs > (1 << 24)) return MJ_ERR_INVALID_ARG;
  *words = size_t(4 * (work_rows(slots, max_num_seqs) + max_num_seqs));
  return MJ_OK;
}

int mj_block_plan(const int32_t* seq_lens_host, int num_seqs, int max_num_seqs, int slots, int margin, int32_t* plan_host,
                  size_t plan_words) {
  const mj::NvtxRange range("mj_block_plan");
  if (num_seqs < 0 || num_seqs > max_num_seqs || margin < 0 || (num_seqs > 0 && !seq_lens_host) || !plan_host)
    return MJ_ERR_INVALID_ARG;
  size_t words = 0;
  const int st = mj_block_plan_size(slots, max_num_seqs, &words);
  if (st != MJ_OK) return st;
  if (plan_words < words) return MJ_ERR_CAPACITY;
  for (int b = 0; b < num_seqs; ++b)
    if (seq_lens_host[b] < 0) return MJ_ERR_INVALID_ARG;
  auto tiles = [&](int b) -> int64_t {
    return seq_lens_host[b] > 0 ? ceil_div(int64_t(seq_lens_host[b]) + margin, mj::kKvTile) : 0;
  };
  int64_t total = 0, longest = 1;
  for (int b = 0; b < num_seqs; ++b) {
    const int64_t t = tiles(b);
    total += t;
    longest = std::max(longest, t);
  }
  // Tiles a piece has at most: between half a slot's share of all and the longest
  // request, where the last slot is expected to end first. If all pieces run at once (one a
  // slot), that is the longest piece; else the slots' common load and part of the longest. Few or equal requests
  // stay in one wave that way; a long request among short ones is cut however many there are
  // (34 requests of 200 to 16384 tokens, 16 query rows: 229 us in one wave, 191 so, before the kernel was made
  // faster).
  const int64_t least = std::max<int64_t>(1, (total + 2 * int64_t(slots) - 1) / (2 * int64_t(slots)));
  auto pieces = [&](int64_t c, int64_t* most) {
    int64_t n = 0;
    *most = 1;
    for (int b = 0; b < num_seqs; ++b) {
      const int64_t t = tiles(b), k = ceil_div(t, c);
      n += k;
      if (k > 0) *most = std::max(*most, ceil_div(t, k));
    }
    return n;
  };
  int64_t chunk = std::max(longest, least);
  double best = 1e300;
  auto consider = [&](int64_t c) {
    int64_t most;
    const int64_t n = pieces(c, &most);
    if (n > work_rows(slots, max_num_seqs)) return;
    const double end = n <= slots ? double(most) + kPieceTiles
                                  : (double(total) + kPieceTiles * double(n)) / slots + kTail * double(most);
    if (end < best) {
      best = end;
      chunk = c;
    }
  };
  for (int64_t c = chunk; c > least; c = std::min(c - 1, c * 15 / 16)) consider(std::max(c, least));
  consider(least);
  int64_t lo = least, hi = std::max(longest, least);  // the least with which one wave holds all
  if (int64_t most; pieces(hi, &most) <= slots) {
    while (lo < hi) {
      const int64_t mid = lo + (hi - lo) / 2;
      if (pieces(mid, &most) <= slots)
        hi = mid;
      else
        lo = mid + 1;
    }
  }
  consider(lo);
  const int64_t rows = work_rows(slots, max_num_seqs);
  int32_t* work = plan_host;
  int32_t* req = plan_host + 4 * rows;
  std::memset(plan_host, 0, words * sizeof(int32_t));
  int64_t part = 0;
  for (int b = 0; b < num_seqs; ++b) {
    const int64_t t = tiles(b);
    const int64_t n = std::max<int64_t>(1, ceil_div(t, chunk)), each = std::max<int64_t>(1, ceil_div(t, n));
    int32_t* r = req + 4 * int64_t(b);
    r[0] = int32_t(part);
    r[1] = int32_t(t > 0 ? ceil_div(t, each) : 0);
    r[2] = int32_t(each);
    r[3] = int32_t(t);
    if (r[1] > 1) part += r[1];
  }
  if (part > part_cap(slots)) return MJ_ERR_CAPACITY;  // cannot be
  // the longest pieces first, so that the last to start are short ones
  struct Row {
    int32_t b, begin, end, s;
  };
  Row* out = reinterpret_cast<Row*>(work);
  int64_t at = 0;
  for (int b = 0; b < num_seqs; ++b) {
    const int32_t* r = req + 4 * int64_t(b);
    for (int s = 0; s < r[1]; ++s) {
      if (at >= rows) return MJ_ERR_CAPACITY;  // cannot be
      out[at++] = {b, s * r[2], int32_t(std::min<int64_t>((s + int64_t(1)) * r[2], r[3])), s};
    }
  }
  std::sort(out, out + at, [](const Row& x, const Row& y) {
    const int32_t lx = x.end - x.begin, ly = y.end - y.begin;
    return lx != ly ? lx > ly : (x.b != y.b ? x.b < y.b : x.s < y.s);
  });
  return MJ_OK;
}

int mj_block_workspace_size(int slots, int q_len, int h_q, int h_k, int d, size_t* bytes) {
  if (!bytes || !slots_ok(slots) || q_len < 1 || h_k < 1 || h_q < 1 || h_q % h_k) return MJ_ERR_INVALID_ARG;
  if (!mj::head_dim_ok(d)) return MJ_ERR_UNSUPPORTED;
  const int64_t n_q = int64_t(q_len) * (h_q / h_k);
  if (n_q > kMaxRows || h_k > 65535) return MJ_ERR_INVALID_ARG;
  *bytes = mj::kWsHeader + size_t(part_cap(slots) * h_k * n_q) * (size_t(d) + 2) * sizeof(float);
  return MJ_OK;
}

int mj_block_attention(const mj_block_args* a, void* stream) {
  const mj::NvtxRange range("mj_block_attention");
  if (!a) return MJ_ERR_INVALID_ARG;
  int st = check_cache(a->cache, false);
  if (st != MJ_OK) return st;
  const mj_block_cache& c = a->cache;
  if (a->num_seqs < 0 || a->num_seqs > a->max_num_seqs || a->q_len < 1 || a->h_q < 1 || a->h_q % c.h_k)
    return MJ_ERR_INVALID_ARG;
  if (int64_t(a->num_seqs) * a->q_len > kMaxTokens) return MJ_ERR_CAPACITY;
  if (!(a->softmax_scale > 0.f) || !std::isfinite(a->softmax_scale)) return MJ_ERR_INVALID_ARG;
  if (a->out_dtype != MJ_OUT_BF16 && a->out_dtype != MJ_OUT_F16) return MJ_ERR_UNSUPPORTED;
  size_t bytes = 0, words = 0;
  st = mj_block_workspace_size(a->slots, a->q_len, a->h_q, c.h_k, c.d, &bytes);
  if (st == MJ_OK) st = mj_block_plan_size(a->slots, a->max_num_seqs, &words);
  if (st == MJ_OK) st = check_rows(a->q, a->q_tok_stride, a->q_head_stride);
  if (st == MJ_OK) st = check_rows(a->out, a->out_tok_stride, a->out_head_stride);
  if (st == MJ_OK) st = check_table(a->block_table, a->block_table_stride, a->block_table_len);
  if (st != MJ_OK) return st;
  if (!a->seq_lens || !a->plan || !a->workspace) return MJ_ERR_INVALID_ARG;
  if (!aligned(a->seq_lens, 4) || !aligned(a->plan, 16) || !aligned(a->workspace, 16) || !aligned(a->lse, 4))
    return MJ_ERR_ALIGNMENT;
  if (a->workspace_bytes < bytes) return MJ_ERR_CAPACITY;
  if (!rows_apart(c.d, {{a->out_tok_stride, int64_t(a->num_seqs) * a->q_len}, {a->out_head_stride, a->h_q}}))
    return MJ_ERR_INVALID_ARG;
  if (a->num_seqs == 0) return MJ_OK;

  const int h_r = a->h_q / c.h_k, n_q = a->q_len * h_r;
  char* ws = static_cast<char*>(a->workspace);
  const int64_t parts = part_cap(a->slots) * c.h_k * n_q, rows = work_rows(a->slots, a->max_num_seqs);
  float* o_part = reinterpret_cast<float*>(ws + mj::kWsHeader);
  const int4* req = reinterpret_cast<const int4*>(a->plan + 4 * rows);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  bool unsupported = false;
  cudaError_t e = cudaSuccess;
  if (by_rows(n_q)) {
    mj::BlockPromptParams p = {};
    p.num_seqs = a->num_seqs;
    p.num_tokens = a->num_seqs * a->q_len;
    p.max_q_len = a->q_len;
    p.splits = 1;
    p.h_q = a->h_q;
    p.h_k = c.h_k;
    p.h_r = h_r;
    p.d = c.d;
    p.causal = a->causal ? 1 : 0;
    p.scale_log2 = a->softmax_scale * 1.4426950408889634f;
    p.q = static_cast<const uint16_t*>(a->q);
    p.q_ts = a->q_tok_stride;
    p.q_hs = a->q_head_stride;
    p.page_shift = mj::page_shift(c.page_size);
    p.block_shift = mj::page_shift(c.block);
    p.num_pages = c.num_pages;
    sides(c, p.side);
    p.block_table = a->block_table;
    p.bt_stride = a->block_table_stride;
    p.bt_len = a->block_table_len;
    p.seq_lens = a->seq_lens;
    p.out = static_cast<uint16_t*>(a->out);
    p.out_f16 = a->out_dtype == MJ_OUT_F16 ? 1 : 0;
    p.out_ts = a->out_tok_stride;
    p.out_hs = a->out_head_stride;
    p.lse = a->lse;
    p.status = reinterpret_cast<uint32_t*>(ws);
    p.o_part = o_part;
    p.m_part = o_part + parts * c.d;
    p.l_part = p.m_part + parts;
    p.evict_first = a->evict_first;
    p.work = reinterpret_cast<const int4*>(a->plan);
    p.req = req;
    p.num_work = int(rows);
    p.part_cap = int(part_cap(a->slots));
    e = mj::launch_block_prompt(p, s, &unsupported);
  } else {
    mj::DecodeParams p = {};
    p.num_seqs = a->num_seqs;
    p.q_len = a->q_len;
    p.h_q = a->h_q;
    p.h_k = c.h_k;
    p.h_r = h_r;
    p.n_q = n_q;
    p.d = c.d;
    p.causal = a->causal ? 1 : 0;
    p.kv_format = MJ_KV_E4M3;
    p.page_size = c.page_size;
    p.row_bytes = c.d;
    p.num_pages = c.num_pages;
    p.tw = mj_tile_width(n_q);
    p.n_row_tiles = int(ceil_div(n_q, p.tw));
    p.q_mode = mj::kQBlock;
    p.q_bf16 = static_cast<const uint16_t*>(a->q);
    p.q_ts = a->q_tok_stride;
    p.q_hs = a->q_head_stride;
    mj::BlockSide side[2];
    sides(c, side);
    p.k_cache = side[0].codes;
    p.v_cache = side[1].codes;
    p.k_sp = side[0].sp;
    p.k_st = side[0].st;
    p.k_sh = side[0].sh;
    p.v_sp = side[1].sp;
    p.v_st = side[1].st;
    p.v_sh = side[1].sh;
    p.k_exp = side[0].exps;
    p.v_exp = side[1].exps;
    p.ke_sp = side[0].esp;
    p.ke_sh = side[0].esh;
    p.ve_sp = side[1].esp;
    p.ve_sh = side[1].esh;
    p.page_shift = mj::page_shift(c.page_size);
    p.block_shift = mj::page_shift(c.block);
    p.block_table = a->block_table;
    p.bt_stride = a->block_table_stride;
    p.bt_len = a->block_table_len;
    p.seq_lens = a->seq_lens;
    p.work = a->plan;
    p.req = req;
    p.num_work = int(rows);
    p.with_reduction = 1;
    p.part_cap = int(part_cap(a->slots));
    p.qk_scale_log2 = a->softmax_scale * 1.4426950408889634f;
    p.v_fmt = 1.f;
    p.out = static_cast<uint16_t*>(a->out);
    p.out_f16 = a->out_dtype == MJ_OUT_F16 ? 1 : 0;
    p.out_ts = a->out_tok_stride;
    p.out_hs = a->out_head_stride;
    p.lse = a->lse;
    p.status = reinterpret_cast<uint32_t*>(ws);
    p.o_part = o_part;
    p.m_part = o_part + parts * c.d;
    p.l_part = p.m_part + parts;
    p.evict_first = a->evict_first;
    e = mj::launch_decode_block(p, s, &unsupported);
  }
  if (unsupported) return MJ_ERR_UNSUPPORTED;
  if (e != cudaSuccess) return MJ_ERR_CUDA;
  mj::BlockJoinParams j = {};
  j.d = c.d;
  j.units = int64_t(a->num_seqs) * c.h_k * n_q;
  j.o_part = o_part;
  j.m_part = o_part + parts * c.d;
  j.l_part = j.m_part + parts;
  j.out = static_cast<uint16_t*>(a->out);
  j.out_f16 = a->out_dtype == MJ_OUT_F16 ? 1 : 0;
  j.out_ts = a->out_tok_stride;
  j.out_hs = a->out_head_stride;
  j.lse = a->lse;
  j.status = reinterpret_cast<uint32_t*>(ws);
  j.plan = req;
  j.seq_lens = a->seq_lens;
  j.h_k = c.h_k;
  j.h_r = h_r;
  j.n_q = n_q;
  j.q_len = a->q_len;
  j.part_cap = int(part_cap(a->slots));
  return status_of(mj::launch_block_join(j, s));
}

// Pieces of a row tile's keys: as many as give every SM a CTA, none below
// kPromptMinKeys keys.
int mj_block_prompt_splits(int sm_count, int num_seqs, int max_q_len, int max_len, int h_q, int h_k, int d) {
  if (sm_count < 1 || num_seqs < 1 || max_q_len < 1 || max_len < 1 || h_k < 1 || h_q < h_k || h_q % h_k || !mj::head_dim_ok(d))
    return 1;
  const int64_t rows = int64_t(max_q_len) * (h_q / h_k);
  const int64_t ctas = ceil_div(rows, mj::block_prompt_rows(d, rows)) * h_k * num_seqs;
  const int64_t by_keys = std::max<int64_t>(1, max_len / kPromptMinKeys);
  return int(std::min<int64_t>({MJ_BLOCK_MAX_SPLITS, by_keys, std::max<int64_t>(1, sm_count / ctas)}));
}

int mj_block_prompt_workspace_size(int num_tokens, int h_q, int d, int splits, size_t* bytes) {
  if (!bytes || num_tokens < 0 || h_q < 1 || splits < 1 || splits > MJ_BLOCK_MAX_SPLITS) return MJ_ERR_INVALID_ARG;
  if (!mj::head_dim_ok(d)) return MJ_ERR_UNSUPPORTED;
  if (int64_t(num_tokens) * h_q > (int64_t(1) << 31)) return MJ_ERR_INVALID_ARG;
  *bytes = mj::kWsHeader + (splits > 1 ? size_t(splits) * num_tokens * h_q * (size_t(d) + 2) * sizeof(float) : 0);
  return MJ_OK;
}

int mj_block_prompt(const mj_block_prompt_args* a, void* stream) {
  const mj::NvtxRange range("mj_block_prompt");
  if (!a) return MJ_ERR_INVALID_ARG;
  int st = check_cache(a->cache, false);
  if (st != MJ_OK) return st;
  const mj_block_cache& c = a->cache;
  if (a->num_seqs < 0 || a->num_tokens < 0 || a->max_q_len < 0 || a->h_q < 1 || a->h_q % c.h_k) return MJ_ERR_INVALID_ARG;
  if (!(a->softmax_scale > 0.f) || !std::isfinite(a->softmax_scale)) return MJ_ERR_INVALID_ARG;
  if (a->out_dtype != MJ_OUT_BF16 && a->out_dtype != MJ_OUT_F16) return MJ_ERR_UNSUPPORTED;
  size_t bytes = 0;
  st = mj_block_prompt_workspace_size(a->num_tokens, a->h_q, c.d, a->splits, &bytes);
  if (st != MJ_OK) return st;
  const int h_r = a->h_q / c.h_k;
  if (h_r > kMaxRows) return MJ_ERR_INVALID_ARG;  // (a row's token is found by a float32 quotient, exact up to 2^21 heads)
  if (a->num_seqs > 65535 || ceil_div(int64_t(a->max_q_len) * h_r, mj::block_prompt_rows(c.d, int64_t(a->max_q_len) * h_r)) > 65535)
    return MJ_ERR_UNSUPPORTED;
  if (a->num_seqs == 0 || a->num_tokens == 0 || a->max_q_len == 0) return MJ_OK;
  st = check_rows(a->q, a->q_tok_stride, a->q_head_stride);
  if (st == MJ_OK) st = check_rows(a->out, a->out_tok_stride, a->out_head_stride);
  if (st == MJ_OK) st = check_table(a->block_table, a->block_table_stride, a->block_table_len);
  if (st != MJ_OK) return st;
  if (!a->seq_lens || !a->q_starts || !a->workspace) return MJ_ERR_INVALID_ARG;
  if (!aligned(a->seq_lens, 4) || !aligned(a->q_starts, 4) || !aligned(a->workspace, 16) || !aligned(a->lse, 4))
    return MJ_ERR_ALIGNMENT;
  if (a->workspace_bytes < bytes) return MJ_ERR_CAPACITY;
  if (!rows_apart(c.d, {{a->out_tok_stride, a->num_tokens}, {a->out_head_stride, a->h_q}})) return MJ_ERR_INVALID_ARG;

  mj::BlockPromptParams p = {};
  p.num_seqs = a->num_seqs;
  p.num_tokens = a->num_tokens;
  p.max_q_len = std::min(a->max_q_len, a->num_tokens);
  p.splits = a->splits;
  p.h_q = a->h_q;
  p.h_k = c.h_k;
  p.h_r = h_r;
  p.d = c.d;
  p.causal = a->causal ? 1 : 0;
  p.scale_log2 = a->softmax_scale * 1.4426950408889634f;
  p.q = static_cast<const uint16_t*>(a->q);
  p.q_ts = a->q_tok_stride;
  p.q_hs = a->q_head_stride;
  p.q_starts = a->q_starts;
  p.page_shift = mj::page_shift(c.page_size);
  p.block_shift = mj::page_shift(c.block);
  p.num_pages = c.num_pages;
  sides(c, p.side);
  p.block_table = a->block_table;
  p.bt_stride = a->block_table_stride;
  p.bt_len = a->block_table_len;
  p.seq_lens = a->seq_lens;
  p.out = static_cast<uint16_t*>(a->out);
  p.out_f16 = a->out_dtype == MJ_OUT_F16 ? 1 : 0;
  p.out_ts = a->out_tok_stride;
  p.out_hs = a->out_head_stride;
  p.lse = a->lse;
  char* ws = static_cast<char*>(a->workspace);
  p.status = reinterpret_cast<uint32_t*>(ws);
  const int64_t parts = int64_t(a->splits) * a->num_tokens * a->h_q;
  p.o_part = reinterpret_cast<float*>(ws + mj::kWsHeader);
  p.m_part = p.o_part + parts * c.d;
  p.l_part = p.m_part + parts;
  bool unsupported = false;
  cudaError_t e = mj::launch_block_prompt(p, static_cast<cudaStream_t>(stream), &unsupported);
  if (unsupported) return MJ_ERR_UNSUPPORTED;
  if (e != cudaSuccess || a->splits == 1) return status_of(e);
  mj::BlockJoinParams j = {};
  j.d = c.d;
  j.units = int64_t(a->num_tokens) * a->h_q;
  j.o_part = p.o_part;
  j.m_part = p.m_part;
  j.l_part = p.l_part;
  j.out = p.out;
  j.out_f16 = p.out_f16;
  j.out_ts = p.out_ts;
  j.out_hs = p.out_hs;
  j.lse = p.lse;
  j.pieces = a->splits;
  j.h_q = a->h_q;
  j.q_starts = p.q_starts;
  j.num_seqs = a->num_seqs;
  return status_of(mj::launch_block_join(j, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
