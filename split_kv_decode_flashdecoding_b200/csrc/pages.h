// Parameter blocks and launchers of the page operators (pages.cu, pages_api.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "plan.h"

namespace fd {

struct AppendParams {
  const void *k_new, *v_new;          // [rows, Hkv, D]
  int64_t k_sr, k_sh, v_sr, v_sh;     // element strides of row and head
  void *k_pages, *v_pages;            // [num_pages, Hkv, page_size, D]
  int64_t pool_sp, pool_sh;           // element strides of page and head
  const int32_t *block_table, *start_lens, *new_lens;
  int64_t rows;
  int32_t batch, pages_per_seq, num_pages, page_size, hkv, d;
  float k_scale, v_scale;             // E4M3 pages
  float k_recip, v_recip;             // their reciprocals, 0: divide by the scale
  int32_t rows_per_cta;
  uint32_t* status;
};

struct ReserveParams {
  int32_t *page_refs, *block_table;
  const int32_t* want_lens;
  int32_t batch, pages_per_seq, num_pages, page_size;
  uint32_t* status;
};

struct ForkParams {
  void *k_pages, *v_pages;
  int64_t pool_sp, pool_sh;           // byte strides of page and head
  int32_t *page_refs, *block_table, *cache_lens;
  const int32_t *src_seqs, *dst_seqs;
  int4* copies;                       // [count] (from page, to page, rows, 0), workspace
  int32_t batch, count, pages_per_seq, num_pages, page_size, hkv, row_bytes;
  uint32_t* status;
};

struct FreeParams {
  int32_t *page_refs, *block_table, *cache_lens;
  const int32_t* seqs;
  int32_t batch, count, pages_per_seq, num_pages;
  uint32_t* status;
};

struct CompactParams {
  void *k_pages, *v_pages;
  int64_t pool_sp, pool_sh;           // byte strides of page and head
  int32_t *page_refs, *block_table, *cache_lens;
  const int32_t *start_lens, *keep, *keep_lens;
  int32_t* valid;                     // [batch], workspace
  int32_t batch, max_keep, pages_per_seq, num_pages, page_size, hkv, row_bytes;
  uint32_t* status;
};

cudaError_t launch_append(AppendParams p, int src_dtype, bool fp8, int nsm, cudaStream_t stream);
cudaError_t launch_reserve(const ReserveParams& p, cudaStream_t stream);
cudaError_t launch_fork(const ForkParams& p, cudaStream_t stream);
cudaError_t launch_free(const FreeParams& p, cudaStream_t stream);
cudaError_t launch_compact(const CompactParams& p, cudaStream_t stream);

#if defined(__CUDACC__)
// One reference less for `page`. A page outside the pool, or without a reference, is reported.
__device__ __forceinline__ void drop_reference(int32_t* refs, int32_t num_pages, int32_t page, uint32_t* status) {
  if (page < 0 || page >= num_pages) {
    atomicOr(status, FD_FLAG_BAD_PAGE);
  } else if (atomicSub(&refs[page], 1) <= 0) {
    atomicAdd(&refs[page], 1);
    atomicOr(status, FD_FLAG_BAD_PAGE);
  }
}
#endif

}  // namespace fd
