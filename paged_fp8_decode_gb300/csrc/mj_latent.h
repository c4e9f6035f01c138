// Internal definitions of the rotated cache writes and the latent-cache
// attention, shared by their host layer (mj_api_latent.cpp) and their kernels.
#pragma once

#include "mj_internal.h"

namespace mj {

// Everything a latent-attention launch needs, by value (kernel parameter).
struct LatentParams {
  int num_seqs, q_len, h, n_q;  // n_q = q_len * h rows a request
  int causal;
  int row_tile, n_row_tiles;
  float softmax_scale;
  const uint16_t* q;
  int64_t q_ts, q_hs;
  const uint8_t* cache;
  int64_t stride_page, stride_token;
  int page_size, page_shift;
  uint32_t page_span;  // bytes from a page's first row to the end of its last; 0 where its rows lie far apart
  int64_t num_pages;
  const float* descale;
  const int32_t* block_table;
  int64_t bt_stride, bt_len;
  const int32_t* seq_lens;
  int slots, max_work;     // plan: slots, rows of the work list
  const int32_t* slot_table;  // [slots][4]: first work row, end, that row's request and first tile
  const int32_t* splits;   // [max_num_seqs][2]: first partial, number of them (0: not split)
  const int32_t* work;     // [max_work][4]: request, first tile, end tile, partial (-1: none)
  const int32_t* planned;  // [max_num_seqs]: tiles the plan covers
  uint16_t* out;
  int out_f16;
  int64_t out_ts, out_hs;
  float* lse;
  uint32_t* status;
  // partials, unnormalised: [2 * slots][row tiles][4 channel blocks][row_tile / 4][128 channels][4 rows]
  float* o_part;
  float* m_part;  // [2 * slots][row tiles * row_tile]: reference max (log2 units), -inf without a key
  float* l_part;  // likewise: sum of the weights, scaled like o_part
  int evict_first;
};

inline int page_shift(int page_size) { return page_size == 16 ? 4 : (page_size == 32 ? 5 : (page_size == 64 ? 6 : 7)); }

// Words (int32) of the plan buffer's parts, each a multiple of 4.
inline int64_t latent_plan_slot_words(int slots) { return 4 * int64_t(slots); }
inline int64_t latent_plan_split_words(int max_num_seqs) { return (2 * int64_t(max_num_seqs) + 3) / 4 * 4; }
inline int64_t latent_plan_max_work(int slots, int max_num_seqs) { return int64_t(slots) + max_num_seqs; }
inline int64_t latent_plan_tile_words(int max_num_seqs) { return (int64_t(max_num_seqs) + 3) / 4 * 4; }

cudaError_t launch_rope_write(const mj_rope_write_kv_args& a, cudaStream_t stream);
cudaError_t launch_latent_write(const mj_latent_write_args& a, cudaStream_t stream);
cudaError_t launch_latent(const LatentParams& p, cudaStream_t stream);
cudaError_t launch_latent_merge(const LatentParams& p, cudaStream_t stream);
// The argument checks of mj_write_kv (MJ_OK, also for num_tokens == 0).
int check_write_kv(const mj_write_kv_args* a);

}  // namespace mj
