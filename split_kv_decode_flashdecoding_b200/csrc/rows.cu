// Attention of packed query rows on CUDA cores: one warp a (row, query head), one key at a time.
//
//   s_j = q·k_j log2(e) / sqrt(D);  m = max_j s_j;  l = sum_j 2^(s_j - m);  o = sum_j 2^(s_j - m) v_j / l
//
// with the running maximum and sum of an online softmax, over the row's visible keys in order.
#include "common.cuh"
#include "rows.h"

namespace fd {

namespace {

constexpr int kRowWarps = 8;

template <int kVec>
__global__ void __launch_bounds__(kRowWarps * 32) rows_kernel(const RowsParams p) {
  __shared__ int64_t s_start;
  __shared__ int s_b, s_bad;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x;
  if (threadIdx.x == 0) {
    int64_t at = 0;
    s_b = -1;
    s_bad = 0;
    for (int b = 0; b < p.batch; ++b) {
      const int n = p.row_lens[b];
      if (p.prefix_lens ? (n < 0 || n > 32 * p.mask_words) : false) s_bad = 1;
      if (n < 0) atomicOr(&p.hdr->status, FD_FLAG_LEN_CLAMPED);
      if (row >= at && row < at + n) {
        s_b = b;
        s_start = at;
      }
      at += max(n, 0);
    }
    if (at > p.rows) s_bad = 1;
    if (s_bad) atomicOr(&p.hdr->status, FD_FLAG_LEN_CLAMPED);
  }
  __syncthreads();
  if (s_bad || s_b < 0) return;
  const int b = s_b, i = static_cast<int>(row - s_start);
  int prefix = 0, keys = i + 1;
  if (p.prefix_lens) {
    prefix = clamp_len(p.prefix_lens[b], p.cap);
    keys = static_cast<int>(min(static_cast<int64_t>(prefix) + p.row_lens[b], static_cast<int64_t>(p.cap)));
    if (threadIdx.x == 0 && (prefix != p.prefix_lens[b] || keys < static_cast<int64_t>(prefix) + p.row_lens[b]))
      atomicOr(&p.hdr->status, FD_FLAG_LEN_CLAMPED);
  }
  for (int hq = warp; hq < p.hq; hq += kRowWarps) {
    const int h = hq / p.g;
    float q[kVec], o[kVec], m = -INFINITY, l = 0.f;
    const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(p.q) + row * p.q_sr + hq * p.q_sh + lane * kVec;
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      q[e] = to_f32(qr[e]);
      o[e] = 0.f;
    }
    for (int j = 0; j < keys; ++j) {
      int64_t ko, vo;
      if (!p.prefix_lens) {
        ko = (s_start + j) * p.k_sr + h * p.k_sh;
        vo = (s_start + j) * p.v_sr + h * p.v_sh;
      } else {
        if (j >= prefix) {
          const int t = j - prefix;
          if (!((p.mask[static_cast<int64_t>(row) * p.mask_words + (t >> 5)] >> (t & 31)) & 1u)) continue;
        }
        if (p.block_table) {
          const int page = p.block_table[static_cast<int64_t>(b) * p.pages_per_seq + j / p.page_size];
          if (page < 0 || page >= p.num_pages) {
            atomicOr(&p.hdr->status, FD_FLAG_BAD_PAGE);
            continue;
          }
          ko = page * p.kv_sb + h * p.kv_sh + static_cast<int64_t>(j % p.page_size) * p.d;
        } else {
          ko = b * p.kv_sb + h * p.kv_sh + static_cast<int64_t>(j) * p.d;
        }
        vo = ko;
      }
      const __nv_bfloat16* kr = static_cast<const __nv_bfloat16*>(p.k) + ko + lane * kVec;
      const __nv_bfloat16* vr = static_cast<const __nv_bfloat16*>(p.v) + vo + lane * kVec;
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < kVec; ++e) s = fmaf(q[e], to_f32(kr[e]), s);
      s = warp_sum_f32(s) * p.scale_log2;
      const float mn = fmaxf(m, s);
      const float a = fast_exp2(m - mn), w = fast_exp2(s - mn);
      l = fmaf(l, a, w);
#pragma unroll
      for (int e = 0; e < kVec; ++e) o[e] = fmaf(o[e], a, w * to_f32(vr[e]));
      m = mn;
    }
    __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(p.out) + row * p.o_sr + hq * p.o_sh + lane * kVec;
#pragma unroll
    for (int e = 0; e < kVec; ++e) orow[e] = __float2bfloat16_rn(l > 0.f ? o[e] / l : 0.f);
    if (lane == 0) p.lse[static_cast<int64_t>(row) * p.hq + hq] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
  }
}

}  // namespace

cudaError_t launch_rows(const RowsParams& p, cudaStream_t stream) {
  if (p.d == 64) rows_kernel<2><<<p.rows, kRowWarps * 32, 0, stream>>>(p);
  else rows_kernel<4><<<p.rows, kRowWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace fd
