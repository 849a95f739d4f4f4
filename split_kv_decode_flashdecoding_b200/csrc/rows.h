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
  int64_t k_sr, k_sh, v_sr, v_sh;  // prompt: of k and v (a cache's are in the tensor maps)
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
  int32_t g_recip16;               // ceil(2^16 / G): (r * g_recip16) >> 16 == r / G for 0 <= r < 128
  int32_t q_box_rows;              // tokens of one Q box (G heads each): min(128 / G, rows)
  int32_t kv_box_rows;             // keys of one K or V box: min(128; rows, S_cap or page_size)
  WsHeader* hdr;
  WsFront* front;                  // in front of hdr
  float *part_o, *part_ml;         // pieces of cut items, behind the header (launch_rows)
};

// tcgen05 kernel: bf16, D 64 or 128, G <= 16. Maps: q as (D, Hq, rows), box 64 x G x q_box_rows; k and v
// as (D, Hkv, rows) with box 64 x 1 x box rows (prompt), (D, S_cap, Hkv, B) or (D, page_size, Hkv,
// num_pages) with box 64 x box rows x 1 x 1.
size_t rows_workspace_bytes(int d, int nctas);
cudaError_t launch_rows(RowsParams p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, int nctas,
                        cudaStream_t stream);

}  // namespace fd
