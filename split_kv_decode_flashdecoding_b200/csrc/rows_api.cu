// C ABI of the attention of packed query rows (include/fd.h): prompts and drafted trees.
#include <algorithm>
#include <cmath>

#include "abi_internal.h"
#include "rows.h"
#include "rows_plan.h"

using namespace fd;
using namespace fd_abi;

namespace {

constexpr int32_t kMaxMaskWords = 8;
constexpr int64_t kMaxKeys = (int64_t{1} << 31) - 1024;  // the kernel counts keys up to whole tiles in 32 bits

fd_status check_rows(const fd_tensor* t, const char* name, int64_t rows, int64_t heads, int64_t d) {
  fd_status s;
  if ((s = check_tensor(t, name, 3)) != FD_OK) return s;
  if (t->dtype != FD_BF16) return fail(FD_ERR_UNSUPPORTED, "%s must be FD_BF16", name);
  if (t->shape[0] != rows || t->shape[1] != heads || t->shape[2] != d)
    return fail(FD_ERR_INVALID_ARGUMENT, "%s must be [%lld, %lld, %lld]", name, (long long)rows, (long long)heads, (long long)d);
  if (rows > 0 && !t->data) return fail(FD_ERR_INVALID_ARGUMENT, "%s data is NULL", name);
  if (!aligned16(t->data) || !stride16(t->stride[0], t->dtype) || !stride16(t->stride[1], t->dtype))
    return fail(FD_ERR_UNSUPPORTED, "%s data and strides must be 16-byte aligned", name);
  return FD_OK;
}

// q, out, lse and the head counts of both calls; *p gets their fields.
fd_status resolve_rows(const fd_tensor* q, const fd_tensor* out, int64_t hkv, int64_t d, int32_t batch, RowsParams* p) {
  fd_status s;
  if ((s = check_tensor(q, "q", 3)) != FD_OK) return s;
  const int64_t rows = q->shape[0], hq = q->shape[1];
  if (d != 64 && d != 128) return fail(FD_ERR_UNSUPPORTED, "head_dim %lld: only 64 and 128 are supported", (long long)d);
  if ((s = check_rows(q, "q", rows, hq, d)) != FD_OK) return s;
  if ((s = check_rows(out, "out", rows, hq, d)) != FD_OK) return s;
  if (hkv < 1) return fail(FD_ERR_INVALID_ARGUMENT, "at least one KV head is needed");
  if (hq < 1 || hq % hkv != 0)
    return fail(FD_ERR_INVALID_ARGUMENT, "q heads (%lld) must be a positive multiple of KV heads (%lld)", (long long)hq, (long long)hkv);
  if (hq / hkv > 16) return fail(FD_ERR_UNSUPPORTED, "group size %lld above 16", (long long)(hq / hkv));
  if (rows > kMaxKeys) return fail(FD_ERR_UNSUPPORTED, "more than 2^31 - 1024 rows");
  if (hq > 65535) return fail(FD_ERR_UNSUPPORTED, "more than 65535 query heads");
  if ((rows > 1 && out->stride[0] == 0) || (hq > 1 && out->stride[1] == 0))
    return fail(FD_ERR_UNSUPPORTED, "out's rows and heads must not share memory");
  if (batch < 0) return fail(FD_ERR_INVALID_ARGUMENT, "batch must be >= 0");
  if (batch > kMaxPlanBatch) return fail(FD_ERR_UNSUPPORTED, "batch %d exceeds %d", batch, kMaxPlanBatch);
  p->q = q->data;
  p->q_sr = q->stride[0];
  p->q_sh = q->stride[1];
  p->out = out->data;
  p->o_sr = out->stride[0];
  p->o_sh = out->stride[1];
  p->batch = batch;
  p->rows = static_cast<int32_t>(rows);
  p->hq = static_cast<int32_t>(hq);
  p->hkv = static_cast<int32_t>(hkv);
  p->g = static_cast<int32_t>(hq / hkv);
  p->d = static_cast<int32_t>(d);
  p->g_recip16 = (65536 + p->g - 1) / p->g;
  p->scale_log2 = static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)) * 1.4426950408889634);
  return FD_OK;
}

int row_ctas(int nsm) { return std::min(nsm, kMaxRowCtas); }

// Launch on all multiprocessors. kd: dimensions of the K and V maps, ks / vs their byte strides; kv_rows: keys
// that one box may reach over.
fd_status run_rows(RowsParams* p, int kv_rank, const uint64_t* kd, const uint64_t* ks, const uint64_t* vs,
                   int kv_rows, cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  const int nctas = row_ctas(sm_count(dev));
  if (nctas < 1) return fail(FD_ERR_CUDA, "no multiprocessors reported for device %d", dev);
  void* ws = nullptr;
  WorkspaceUse use;
  fd_status s = get_workspace(stream, rows_workspace_bytes(p->d, nctas), &use, &ws, nullptr);
  if (s != FD_OK) return s;
  p->hdr = static_cast<WsHeader*>(ws);
  CUtensorMap tq, tk, tv;
  p->q_box_rows = std::min(rows_tile_tokens(p->g), p->rows);
  const uint64_t qd[3] = {static_cast<uint64_t>(p->d), static_cast<uint64_t>(p->hq), static_cast<uint64_t>(p->rows)};
  const uint64_t qs[2] = {static_cast<uint64_t>(p->q_sh) * 2, static_cast<uint64_t>(p->q_sr) * 2};
  const uint32_t qb[3] = {64, static_cast<uint32_t>(p->g), static_cast<uint32_t>(p->q_box_rows)};
  if ((s = make_tmap(&tq, p->q, 3, qd, qs, qb, "q")) != FD_OK) return s;
  p->kv_box_rows = std::min(128, kv_rows);
  uint32_t kb[4] = {64, 1, 1, 1};
  kb[kv_rank == 3 ? 2 : 1] = static_cast<uint32_t>(p->kv_box_rows);
  if ((s = make_tmap(&tk, p->k, kv_rank, kd, ks, kb, "k")) != FD_OK) return s;
  if ((s = make_tmap(&tv, p->v, kv_rank, kd, vs, kb, "v")) != FD_OK) return s;
  e = launch_rows(*p, tq, tk, tv, nctas, stream);
  return e == cudaSuccess ? FD_OK : cuda_fail(e, "attention kernel launch");
}

fd_status tree(const fd_tensor* q, const fd_tensor* k, const fd_tensor* v, const int32_t* block_table,
               int32_t pages_per_seq, int32_t batch, bool paged, const int32_t* prefix_lens,
               const int32_t* tree_lens, const int32_t* tree_mask, int32_t mask_words, fd_tensor* out,
               float* lse, cudaStream_t stream) {
  fd_status s;
  RowsParams p{};
  const char* kn = paged ? "k_pages" : "k_cache";
  const char* vn = paged ? "v_pages" : "v_cache";
  if ((s = check_tensor(k, kn, 4)) != FD_OK) return s;
  if ((s = check_tensor(v, vn, 4)) != FD_OK) return s;
  if (k->dtype != FD_BF16 || v->dtype != FD_BF16) return fail(FD_ERR_UNSUPPORTED, "%s / %s must be FD_BF16", kn, vn);
  for (int i = 0; i < 4; ++i)
    if (k->shape[i] != v->shape[i]) return fail(FD_ERR_INVALID_ARGUMENT, "%s and %s shapes differ", kn, vn);
  for (int i = 0; i < 4; ++i)
    if (k->stride[i] != v->stride[i]) return fail(FD_ERR_UNSUPPORTED, "%s and %s must share strides", kn, vn);
  if ((s = resolve_rows(q, out, k->shape[1], k->shape[3], paged ? batch : static_cast<int32_t>(k->shape[0]), &p)) != FD_OK) return s;
  if (k->shape[2] < 1) return fail(FD_ERR_INVALID_ARGUMENT, "%s capacity (dim 2) must be >= 1", kn);
  if (k->stride[2] != p.d) return fail(FD_ERR_UNSUPPORTED, "token rows must be contiguous (stride[2] == head_dim)");
  if (!aligned16(k->data) || !aligned16(v->data) || !stride16(k->stride[0], FD_BF16) || !stride16(k->stride[1], FD_BF16))
    return fail(FD_ERR_UNSUPPORTED, "%s / %s data and strides must be 16-byte aligned", kn, vn);
  if (k->shape[0] > 0 && (!k->data || !v->data)) return fail(FD_ERR_INVALID_ARGUMENT, "%s / %s data is NULL", kn, vn);
  if (mask_words < 1) return fail(FD_ERR_INVALID_ARGUMENT, "mask_words must be >= 1");
  if (mask_words > kMaxMaskWords) return fail(FD_ERR_UNSUPPORTED, "mask_words %d exceeds %d", mask_words, kMaxMaskWords);
  if (paged) {
    const int64_t psz = k->shape[2];
    if (k->shape[0] < 1) return fail(FD_ERR_INVALID_ARGUMENT, "the page pool needs at least one page");
    if (!(psz == 8 || psz == 16 || psz == 32 || psz == 64 || (psz >= 128 && psz % 128 == 0)))
      return fail(FD_ERR_UNSUPPORTED, "page size %lld: must be 8, 16, 32, 64 or a multiple of 128", (long long)psz);
    if (pages_per_seq < 1) return fail(FD_ERR_INVALID_ARGUMENT, "pages_per_seq must be >= 1");
    if (static_cast<int64_t>(pages_per_seq) * psz > INT32_MAX)
      return fail(FD_ERR_UNSUPPORTED, "pages_per_seq * page_size exceeds 2^31 keys");
    if (batch > 0 && !block_table) return fail(FD_ERR_INVALID_ARGUMENT, "block_table is NULL");
    p.block_table = block_table;
    p.pages_per_seq = pages_per_seq;
    p.page_size = static_cast<int32_t>(psz);
    p.num_pages = static_cast<int32_t>(k->shape[0]);
    p.cap = pages_per_seq * p.page_size;
  } else {
    p.cap = static_cast<int32_t>(k->shape[2]);
  }
  if (p.cap > kMaxKeys) return fail(FD_ERR_UNSUPPORTED, "a capacity of %d keys exceeds 2^31 - 1024", p.cap);
  if (p.rows == 0 || p.batch == 0) return FD_OK;
  if (!prefix_lens || !tree_lens || !tree_mask)
    return fail(FD_ERR_INVALID_ARGUMENT, "prefix_lens / tree_lens / tree_mask is NULL");
  if (!lse) return fail(FD_ERR_INVALID_ARGUMENT, "lse is NULL");
  p.k = k->data;
  p.v = v->data;
  p.lse = lse;
  p.row_lens = tree_lens;
  p.prefix_lens = prefix_lens;
  p.mask = reinterpret_cast<const uint32_t*>(tree_mask);
  p.mask_words = mask_words;
  const uint64_t kd[4] = {static_cast<uint64_t>(p.d), static_cast<uint64_t>(k->shape[2]), static_cast<uint64_t>(p.hkv),
                          static_cast<uint64_t>(k->shape[0])};
  const uint64_t ks[3] = {static_cast<uint64_t>(k->stride[2]) * 2, static_cast<uint64_t>(k->stride[1]) * 2,
                          static_cast<uint64_t>(k->stride[0]) * 2};
  return run_rows(&p, 4, kd, ks, ks, paged ? p.page_size : p.cap, stream);
}

}  // namespace

extern "C" {

fd_status fd_prompt_attention(const fd_tensor* q, const fd_tensor* k, const fd_tensor* v,
                              const int32_t* seq_lens, int32_t batch, fd_tensor* out, float* lse,
                              void* stream) {
  fd_status s;
  RowsParams p{};
  if ((s = check_tensor(q, "q", 3)) != FD_OK) return s;
  if ((s = check_tensor(k, "k", 3)) != FD_OK) return s;
  if ((s = resolve_rows(q, out, k->shape[1], k->shape[2], batch, &p)) != FD_OK) return s;
  if ((s = check_rows(k, "k", p.rows, p.hkv, p.d)) != FD_OK) return s;
  if ((s = check_rows(v, "v", p.rows, p.hkv, p.d)) != FD_OK) return s;
  if (p.rows == 0 || p.batch == 0) return FD_OK;
  if (!seq_lens) return fail(FD_ERR_INVALID_ARGUMENT, "seq_lens is NULL");
  if (!lse) return fail(FD_ERR_INVALID_ARGUMENT, "lse is NULL");
  p.k = k->data;
  p.v = v->data;
  p.k_sr = k->stride[0];
  p.k_sh = k->stride[1];
  p.v_sr = v->stride[0];
  p.v_sh = v->stride[1];
  p.lse = lse;
  p.row_lens = seq_lens;
  p.cap = p.rows;
  const uint64_t kd[3] = {static_cast<uint64_t>(p.d), static_cast<uint64_t>(p.hkv), static_cast<uint64_t>(p.rows)};
  const uint64_t ks[2] = {static_cast<uint64_t>(p.k_sh) * 2, static_cast<uint64_t>(p.k_sr) * 2};
  const uint64_t vs[2] = {static_cast<uint64_t>(p.v_sh) * 2, static_cast<uint64_t>(p.v_sr) * 2};
  return run_rows(&p, 3, kd, ks, vs, p.rows, static_cast<cudaStream_t>(stream));
}

fd_status fd_tree_attention(const fd_tensor* q, const fd_tensor* k_cache, const fd_tensor* v_cache,
                            const int32_t* prefix_lens, const int32_t* tree_lens,
                            const int32_t* tree_mask, int32_t mask_words, fd_tensor* out,
                            float* lse, void* stream) {
  return tree(q, k_cache, v_cache, nullptr, 0, 0, false, prefix_lens, tree_lens, tree_mask, mask_words,
              out, lse, static_cast<cudaStream_t>(stream));
}

fd_status fd_tree_attention_paged(const fd_tensor* q, const fd_tensor* k_pages,
                                  const fd_tensor* v_pages, const int32_t* block_table,
                                  int32_t pages_per_seq, int32_t batch,
                                  const int32_t* prefix_lens, const int32_t* tree_lens,
                                  const int32_t* tree_mask, int32_t mask_words, fd_tensor* out,
                                  float* lse, void* stream) {
  return tree(q, k_pages, v_pages, block_table, pages_per_seq, batch, true, prefix_lens, tree_lens,
              tree_mask, mask_words, out, lse, static_cast<cudaStream_t>(stream));
}

size_t fd_prompt_workspace_bytes(int32_t batch, int32_t total_rows, int32_t num_q_heads,
                                 int32_t num_kv_heads, int32_t head_dim) {
  if (batch < 0 || total_rows < 0 || num_q_heads < 1 || num_kv_heads < 1 || head_dim < 1) return 0;
  return rows_workspace_bytes(head_dim, kMaxRowCtas);
}

size_t fd_tree_workspace_bytes(int32_t batch, int32_t total_rows, int32_t num_q_heads,
                               int32_t num_kv_heads, int32_t cache_capacity, int32_t head_dim) {
  if (batch < 0 || total_rows < 0 || num_q_heads < 1 || num_kv_heads < 1 || cache_capacity < 0 || head_dim < 1) return 0;
  return rows_workspace_bytes(head_dim, kMaxRowCtas);
}

}  // extern "C"
