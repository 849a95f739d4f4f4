// Attention of packed query rows (whole prompts, drafted trees): parameter block and launchers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "plan.h"

namespace fd {

// Rows of request b: [start_b, start_b + row_lens[b]) of q. Keys: the request's own rows of k and v
// (prompt: prefix_lens == nullptr, causal), or its cache (tree: all prefix_lens[b] keys and the
// drafts behind them whose mask bit is set).
struct RowsParams {
  const void *q, *k, *v;
  int64_t q_sr, q_sh;              // element strides of row and head
  int64_t k_sr, k_sh, v_sr, v_sh;  // prompt: of k and v
  int64_t kv_sb, kv_sh;            // tree: strides of sequence (page) and head
  void* out;
  int64_t o_sr, o_sh;
  float* lse;                      // [rows][Hq]
  const int32_t *row_lens, *prefix_lens;
  const uint32_t* mask;            // [rows][mask_words]
  int32_t mask_words;
  const int32_t* block_table;      // paged cache, else nullptr
  int32_t pages_per_seq, page_size, num_pages;
  int32_t batch, rows, hq, hkv, g, d, cap;
  float scale_log2;                // log2(e) / sqrt(D)
  WsHeader* hdr;
};

cudaError_t launch_rows(const RowsParams& p, cudaStream_t stream);

}  // namespace fd
