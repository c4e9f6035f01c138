// Internal definitions of the block-scaled cache's calls, shared by their host
// layer (mj_api_block.cpp) and their kernels.
#pragma once

#include "mj_internal.h"

namespace mj {

// One side (K or V) of the cache, as the kernels see it.
struct BlockSide {
  uint8_t* codes;
  int64_t sp, st, sh;  // bytes
  uint8_t* exps;
  int64_t esp, esh;
};

struct BlockWriteParams {
  int num_tokens, h_k;
  const uint16_t* in[2];  // key, value
  int64_t ts[2], hs[2];
  const int64_t* slots;
  int64_t num_slots;
  int page_shift, block_shift;
  BlockSide side[2];
  uint32_t* status;
  int window;  // tokens a CTA looks through
};

struct BlockReadParams {
  int num_seqs;
  int64_t num_rows;
  int h_k, page_shift, block_shift;
  int64_t num_pages;
  BlockSide side[2];
  const int32_t* block_table;
  int64_t bt_stride, bt_len;
  const int32_t* starts;
  const int32_t* first;
  uint16_t* out[2];
  int64_t ts[2], hs[2];
  int out_f16;
  int sides, side0;  // how many outputs there are, and the first of them
  uint32_t* status;
};

// Partials of rows whose keys were cut into pieces, and how they are joined:
// piece s of unit u's row lies at partial row (first + s * step).
struct BlockJoinParams {
  int d;
  int64_t units;              // rows to join
  const float* o_part;        // [partial rows][d], normalised
  const float* m_part;        // reference of each (log2 units), -inf without a key
  const float* l_part;        // sum of 2^(t - m)
  uint16_t* out;
  int out_f16;
  int64_t out_ts, out_hs;
  float* lse;
  uint32_t* status;
  // decode (plan != null): unit = (request, KV head, row)
  const int4* plan;           // per request: first partial, pieces, tiles a piece, tiles planned
  const int32_t* seq_lens;
  int h_k, h_r, n_q, q_len;
  int part_cap;               // partials that the workspace holds of each KV head
  // prompt: unit = (token, query head), `pieces` pieces each, lying `units` rows apart
  int pieces, h_q;
  const int32_t* q_starts;
  int num_seqs;
};


// 2^(e - 127) of an exponent byte, held to the range that the format has.
__host__ __device__ inline int block_exp(int e) {
  return e < MJ_BLOCK_EXP_MIN ? MJ_BLOCK_EXP_MIN : (e > MJ_BLOCK_EXP_MAX ? MJ_BLOCK_EXP_MAX : e);
}

struct BlockPromptParams {
  int num_seqs, num_tokens, max_q_len, splits;
  int h_q, h_k, h_r, d;
  int causal;
  float scale_log2;           // softmax_scale * log2(e)
  const uint16_t* q;
  int64_t q_ts, q_hs;
  const int32_t* q_starts;
  int page_shift, block_shift;
  int64_t num_pages;
  BlockSide side[2];
  const int32_t* block_table;
  int64_t bt_stride, bt_len;
  const int32_t* seq_lens;
  uint16_t* out;
  int out_f16;
  int64_t out_ts, out_hs;
  float* lse;
  uint32_t* status;
  float* o_part;              // splits > 1: [splits][num_tokens][h_q][d], then m and l alike
  float* m_part;
  float* l_part;              // -1: a row that was not computed (piece 0's)
  int tma_head_inner;
  int evict_first;
  // decode (work != null): the plan's pieces (request, first tile, end tile, piece) in place of
  // the grid's; max_q_len query tokens a request, `out` and `lse` laid out by request
  const int4* work;
  const int4* req;            // per request: first partial, pieces, tiles a piece, tiles planned
  int num_work, part_cap;
};

// Sets *unsupported (and launches nothing) where TMA cannot take the cache's strides.
cudaError_t launch_block_prompt(BlockPromptParams p, cudaStream_t stream, bool* unsupported);
int block_prompt_rows(int d, int64_t rows);  // query rows of a CTA, of so many of a request and KV head
cudaError_t launch_block_write(BlockWriteParams p, int d, cudaStream_t stream);
cudaError_t launch_block_read(const BlockReadParams& p, int d, cudaStream_t stream);
cudaError_t launch_block_join(const BlockJoinParams& p, cudaStream_t stream);

}  // namespace mj
