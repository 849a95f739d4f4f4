// C ABI of the page operators (include/fd.h): argument checks and launches.
#include <algorithm>
#include <cfloat>

#include "abi_internal.h"
#include "pages.h"

using namespace fd;
using namespace fd_abi;

namespace {

// A pair of page pools [num_pages, Hkv, page_size, D] that share shape and strides.
fd_status check_pool(const fd_tensor* k, const fd_tensor* v) {
  fd_status s;
  if ((s = check_tensor(k, "k_pages", 4)) != FD_OK) return s;
  if ((s = check_tensor(v, "v_pages", 4)) != FD_OK) return s;
  if (k->dtype != v->dtype) return fail(FD_ERR_INVALID_ARGUMENT, "k_pages and v_pages dtypes differ");
  for (int i = 0; i < 4; ++i)
    if (k->shape[i] != v->shape[i]) return fail(FD_ERR_INVALID_ARGUMENT, "k_pages and v_pages shapes differ");
  for (int i = 0; i < 4; ++i)
    if (k->stride[i] != v->stride[i]) return fail(FD_ERR_UNSUPPORTED, "k_pages and v_pages must share strides");
  if (k->shape[0] < 1) return fail(FD_ERR_INVALID_ARGUMENT, "the page pool needs at least one page");
  if (k->shape[1] < 1) return fail(FD_ERR_INVALID_ARGUMENT, "k_pages needs at least one KV head");
  if (k->shape[1] > 32767) return fail(FD_ERR_UNSUPPORTED, "more than 32767 KV heads");
  const int64_t psz = k->shape[2], d = k->shape[3];
  if (d != 64 && d != 128) return fail(FD_ERR_UNSUPPORTED, "head_dim %lld: only 64 and 128 are supported", (long long)d);
  if (!(psz == 8 || psz == 16 || psz == 32 || psz == 64 || (psz >= 128 && psz % 128 == 0)))
    return fail(FD_ERR_UNSUPPORTED, "page size %lld: must be 8, 16, 32, 64 or a multiple of 128", (long long)psz);
  if (k->stride[2] != d) return fail(FD_ERR_UNSUPPORTED, "token rows of a page must be contiguous (stride[2] == head_dim)");
  if ((k->shape[0] > 1 && k->stride[0] == 0) || (k->shape[1] > 1 && k->stride[1] == 0))
    return fail(FD_ERR_UNSUPPORTED, "pages and their heads must not share memory");
  if (!k->data || !v->data) return fail(FD_ERR_INVALID_ARGUMENT, "k_pages / v_pages data is NULL");
  if (!aligned16(k->data) || !aligned16(v->data) || !stride16(k->stride[0], k->dtype) || !stride16(k->stride[1], k->dtype))
    return fail(FD_ERR_UNSUPPORTED, "page data and strides must be 16-byte aligned");
  return FD_OK;
}

fd_status check_table(int32_t batch, int32_t pages_per_seq, int64_t page_size) {
  if (batch < 0) return fail(FD_ERR_INVALID_ARGUMENT, "batch must be >= 0");
  if (batch > kMaxPlanBatch) return fail(FD_ERR_UNSUPPORTED, "batch %d exceeds %d", batch, kMaxPlanBatch);
  if (pages_per_seq < 1) return fail(FD_ERR_INVALID_ARGUMENT, "pages_per_seq must be >= 1");
  if (static_cast<int64_t>(pages_per_seq) * page_size > INT32_MAX)
    return fail(FD_ERR_UNSUPPORTED, "pages_per_seq * page_size exceeds 2^31 keys");
  return FD_OK;
}

fd_status check_count(int32_t count) {
  if (count < 0) return fail(FD_ERR_INVALID_ARGUMENT, "count must be >= 0");
  if (count > kMaxPlanBatch) return fail(FD_ERR_UNSUPPORTED, "count %d exceeds %d", count, kMaxPlanBatch);
  return FD_OK;
}

fd_status check_new(const fd_tensor* t, const char* name, const fd_tensor* pages, bool fp8) {
  fd_status s;
  if ((s = check_tensor(t, name, 3)) != FD_OK) return s;
  if (fp8 ? (t->dtype != FD_BF16 && t->dtype != FD_F32) : t->dtype != pages->dtype)
    return fail(FD_ERR_INVALID_ARGUMENT, fp8 ? "%s must be FD_BF16 or FD_F32" : "%s dtype differs from the pages'", name);
  if (t->shape[1] != pages->shape[1] || t->shape[2] != pages->shape[3])
    return fail(FD_ERR_INVALID_ARGUMENT, "%s must be [T, %lld, %lld] like the pages", name, (long long)pages->shape[1],
                (long long)pages->shape[3]);
  if (t->shape[0] > 0 && !t->data) return fail(FD_ERR_INVALID_ARGUMENT, "%s data is NULL", name);
  if (!aligned16(t->data) || !stride16(t->stride[0], t->dtype) || !stride16(t->stride[1], t->dtype))
    return fail(FD_ERR_UNSUPPORTED, "%s data and strides must be 16-byte aligned", name);
  return FD_OK;
}

// The workspace of the stream (status word, then `bytes` of scratch) and the device's SM count.
fd_status scratch(cudaStream_t stream, size_t bytes, WorkspaceUse* use, char** ws, int* nsm) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  *nsm = sm_count(dev);
  if (*nsm < 1) return fail(FD_ERR_CUDA, "no multiprocessors reported for device %d", dev);
  void* p = nullptr;
  fd_status s = get_workspace(stream, sizeof(WsHeader) + bytes, use, &p, nullptr);
  *ws = static_cast<char*>(p);
  return s;
}

fd_status launched(cudaError_t e, const char* what) { return e == cudaSuccess ? FD_OK : cuda_fail(e, what); }

fd_status append(const fd_tensor* k_new, const fd_tensor* v_new, fd_tensor* k, fd_tensor* v, float k_scale,
                 float v_scale, bool fp8, const int32_t* block_table, int32_t pages_per_seq, int32_t batch,
                 const int32_t* start_lens, const int32_t* new_lens, cudaStream_t stream) {
  fd_status s;
  if ((s = check_pool(k, v)) != FD_OK) return s;
  if (fp8 != (k->dtype == FD_E4M3))
    return fail(FD_ERR_INVALID_ARGUMENT, fp8 ? "k_pages / v_pages must be FD_E4M3" : "FD_E4M3 pages need fd_pages_append_fp8");
  if ((s = check_new(k_new, "k_new", k, fp8)) != FD_OK) return s;
  if ((s = check_new(v_new, "v_new", k, fp8)) != FD_OK) return s;
  if (k_new->shape[0] != v_new->shape[0] || k_new->dtype != v_new->dtype)
    return fail(FD_ERR_INVALID_ARGUMENT, "k_new and v_new shapes or dtypes differ");
  if (!(k_scale > 0.f && k_scale <= FLT_MAX) || !(v_scale > 0.f && v_scale <= FLT_MAX))
    return fail(FD_ERR_INVALID_ARGUMENT, "k_scale and v_scale must be finite and > 0");
  if ((s = check_table(batch, pages_per_seq, k->shape[2])) != FD_OK) return s;
  if (batch == 0 || k_new->shape[0] == 0) return FD_OK;
  if (!block_table || !start_lens || !new_lens)
    return fail(FD_ERR_INVALID_ARGUMENT, "block_table / start_lens / new_lens is NULL");
  WorkspaceUse use;
  char* ws = nullptr;
  int nsm = 0;
  if ((s = scratch(stream, 0, &use, &ws, &nsm)) != FD_OK) return s;
  AppendParams p{};
  p.k_new = k_new->data;
  p.v_new = v_new->data;
  p.k_sr = k_new->stride[0];
  p.k_sh = k_new->stride[1];
  p.v_sr = v_new->stride[0];
  p.v_sh = v_new->stride[1];
  p.k_pages = k->data;
  p.v_pages = v->data;
  p.pool_sp = k->stride[0];
  p.pool_sh = k->stride[1];
  p.block_table = block_table;
  p.start_lens = start_lens;
  p.new_lens = new_lens;
  p.rows = k_new->shape[0];
  p.batch = batch;
  p.pages_per_seq = pages_per_seq;
  p.num_pages = static_cast<int32_t>(k->shape[0]);
  p.page_size = static_cast<int32_t>(k->shape[2]);
  p.hkv = static_cast<int32_t>(k->shape[1]);
  p.d = static_cast<int32_t>(k->shape[3]);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  // quotient()'s Newton step needs a normal reciprocal, and a rest x - q s that no rounding touches. q
  // from 2^-11 on (smaller ones are code 0 whatever their last bits) has its last bit at 2^-34 or above, s
  // from 2^e on at 2^(e - 23): their product is a multiple of 2^(e - 57), an fp32 number's last bit 2^-149
  // or more from e = -92 on.
  const auto recip = [](float s) {
    const float r = 1.f / s;
    return s >= 0x1p-90f && r >= FLT_MIN ? r : 0.f;
  };
  p.k_recip = recip(k_scale);
  p.v_recip = recip(v_scale);
  p.status = reinterpret_cast<uint32_t*>(ws);
  return launched(launch_append(p, k_new->dtype, fp8, nsm, stream), "append kernel launch");
}

}  // namespace

extern "C" {

fd_status fd_pages_append(const fd_tensor* k_new, const fd_tensor* v_new, fd_tensor* k_pages,
                          fd_tensor* v_pages, const int32_t* block_table, int32_t pages_per_seq,
                          int32_t batch, const int32_t* start_lens, const int32_t* new_lens,
                          void* stream) {
  return append(k_new, v_new, k_pages, v_pages, 1.f, 1.f, false, block_table, pages_per_seq, batch,
                start_lens, new_lens, static_cast<cudaStream_t>(stream));
}

fd_status fd_pages_append_fp8(const fd_tensor* k_new, const fd_tensor* v_new, fd_tensor* k_pages,
                              fd_tensor* v_pages, float k_scale, float v_scale,
                              const int32_t* block_table, int32_t pages_per_seq, int32_t batch,
                              const int32_t* start_lens, const int32_t* new_lens, void* stream) {
  return append(k_new, v_new, k_pages, v_pages, k_scale, v_scale, true, block_table, pages_per_seq,
                batch, start_lens, new_lens, static_cast<cudaStream_t>(stream));
}

fd_status fd_pages_reserve(int32_t* page_refs, int32_t num_pages, int32_t* block_table,
                           int32_t pages_per_seq, int32_t batch, const int32_t* want_lens,
                           int32_t page_size, void* stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  fd_status s;
  if (num_pages < 1) return fail(FD_ERR_INVALID_ARGUMENT, "num_pages must be >= 1");
  if (page_size < 1) return fail(FD_ERR_INVALID_ARGUMENT, "page_size must be >= 1");
  if ((s = check_table(batch, pages_per_seq, page_size)) != FD_OK) return s;
  if (batch == 0) return FD_OK;
  if (!page_refs || !block_table || !want_lens)
    return fail(FD_ERR_INVALID_ARGUMENT, "page_refs / block_table / want_lens is NULL");
  WorkspaceUse use;
  char* ws = nullptr;
  int nsm = 0;
  if ((s = scratch(stream, 0, &use, &ws, &nsm)) != FD_OK) return s;
  ReserveParams p{};
  p.page_refs = page_refs;
  p.block_table = block_table;
  p.want_lens = want_lens;
  p.batch = batch;
  p.pages_per_seq = pages_per_seq;
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.status = reinterpret_cast<uint32_t*>(ws);
  return launched(launch_reserve(p, stream), "reserve kernel launch");
}

fd_status fd_pages_fork(fd_tensor* k_pages, fd_tensor* v_pages, int32_t* page_refs,
                        int32_t* block_table, int32_t pages_per_seq, int32_t batch,
                        int32_t* cache_lens, const int32_t* src_seqs, const int32_t* dst_seqs,
                        int32_t count, void* stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  fd_status s;
  if ((s = check_pool(k_pages, v_pages)) != FD_OK) return s;
  if ((s = check_table(batch, pages_per_seq, k_pages->shape[2])) != FD_OK) return s;
  if ((s = check_count(count)) != FD_OK) return s;
  if (count == 0) return FD_OK;
  if (batch == 0) return fail(FD_ERR_INVALID_ARGUMENT, "%d pairs but no sequence", count);
  if (!page_refs || !block_table || !cache_lens || !src_seqs || !dst_seqs)
    return fail(FD_ERR_INVALID_ARGUMENT, "page_refs / block_table / cache_lens / src_seqs / dst_seqs is NULL");
  WorkspaceUse use;
  char* ws = nullptr;
  int nsm = 0;
  if ((s = scratch(stream, sizeof(int4) * static_cast<size_t>(count), &use, &ws, &nsm)) != FD_OK) return s;
  const int64_t es = static_cast<int64_t>(elem_size(k_pages->dtype));
  ForkParams p{};
  p.k_pages = k_pages->data;
  p.v_pages = v_pages->data;
  p.pool_sp = k_pages->stride[0] * es;
  p.pool_sh = k_pages->stride[1] * es;
  p.page_refs = page_refs;
  p.block_table = block_table;
  p.cache_lens = cache_lens;
  p.src_seqs = src_seqs;
  p.dst_seqs = dst_seqs;
  p.copies = reinterpret_cast<int4*>(ws + sizeof(WsHeader));
  p.batch = batch;
  p.count = count;
  p.pages_per_seq = pages_per_seq;
  p.num_pages = static_cast<int32_t>(k_pages->shape[0]);
  p.page_size = static_cast<int32_t>(k_pages->shape[2]);
  p.hkv = static_cast<int32_t>(k_pages->shape[1]);
  p.row_bytes = static_cast<int32_t>(k_pages->shape[3] * es);
  p.status = reinterpret_cast<uint32_t*>(ws);
  return launched(launch_fork(p, stream), "fork kernel launch");
}

fd_status fd_pages_free(int32_t* page_refs, int32_t num_pages, int32_t* block_table,
                        int32_t pages_per_seq, int32_t batch, int32_t* cache_lens,
                        const int32_t* seqs, int32_t count, void* stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  fd_status s;
  if (num_pages < 1) return fail(FD_ERR_INVALID_ARGUMENT, "num_pages must be >= 1");
  if ((s = check_table(batch, pages_per_seq, 1)) != FD_OK) return s;
  if ((s = check_count(count)) != FD_OK) return s;
  if (count == 0) return FD_OK;
  if (!page_refs || !block_table || !cache_lens || !seqs)
    return fail(FD_ERR_INVALID_ARGUMENT, "page_refs / block_table / cache_lens / seqs is NULL");
  WorkspaceUse use;
  char* ws = nullptr;
  int nsm = 0;
  if ((s = scratch(stream, 0, &use, &ws, &nsm)) != FD_OK) return s;
  FreeParams p{};
  p.page_refs = page_refs;
  p.block_table = block_table;
  p.cache_lens = cache_lens;
  p.seqs = seqs;
  p.batch = batch;
  p.count = count;
  p.pages_per_seq = pages_per_seq;
  p.num_pages = num_pages;
  p.status = reinterpret_cast<uint32_t*>(ws);
  return launched(launch_free(p, stream), "free kernel launch");
}

fd_status fd_pages_compact(fd_tensor* k_pages, fd_tensor* v_pages, int32_t* page_refs,
                           int32_t* block_table, int32_t pages_per_seq, int32_t batch,
                           int32_t* cache_lens, const int32_t* start_lens, const int32_t* keep,
                           int32_t max_keep, const int32_t* keep_lens, void* stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  fd_status s;
  if ((s = check_pool(k_pages, v_pages)) != FD_OK) return s;
  if ((s = check_table(batch, pages_per_seq, k_pages->shape[2])) != FD_OK) return s;
  if (max_keep < 0) return fail(FD_ERR_INVALID_ARGUMENT, "max_keep must be >= 0");
  if (batch == 0) return FD_OK;
  if (!page_refs || !block_table || !cache_lens || !start_lens || !keep_lens || (max_keep > 0 && !keep))
    return fail(FD_ERR_INVALID_ARGUMENT, "page_refs / block_table / cache_lens / start_lens / keep / keep_lens is NULL");
  WorkspaceUse use;
  char* ws = nullptr;
  int nsm = 0;
  if ((s = scratch(stream, 4 * static_cast<size_t>(batch), &use, &ws, &nsm)) != FD_OK) return s;
  const int64_t es = static_cast<int64_t>(elem_size(k_pages->dtype));
  CompactParams p{};
  p.k_pages = k_pages->data;
  p.v_pages = v_pages->data;
  p.pool_sp = k_pages->stride[0] * es;
  p.pool_sh = k_pages->stride[1] * es;
  p.page_refs = page_refs;
  p.block_table = block_table;
  p.cache_lens = cache_lens;
  p.start_lens = start_lens;
  p.keep = keep;
  p.keep_lens = keep_lens;
  p.valid = reinterpret_cast<int32_t*>(ws + sizeof(WsHeader));
  p.batch = batch;
  p.max_keep = max_keep;
  p.pages_per_seq = pages_per_seq;
  p.num_pages = static_cast<int32_t>(k_pages->shape[0]);
  p.page_size = static_cast<int32_t>(k_pages->shape[2]);
  p.hkv = static_cast<int32_t>(k_pages->shape[1]);
  p.row_bytes = static_cast<int32_t>(k_pages->shape[3] * es);
  p.status = reinterpret_cast<uint32_t*>(ws);
  return launched(launch_compact(p, stream), "compact kernel launch");
}

}  // extern "C"
