// Operators of a paged cache's pages: appending new tokens, reserving, forking and freeing pages,
// compacting a sequence's tokens. Layout as in fd_decode_attention_paged: pools
// [num_pages, Hkv, page_size, D] read through a block table [batch, pages_per_seq] (FlashDecoding
// page, "部署落地的工程细节", names a paged cache without a layout).
#include <cfloat>

#include "abi_internal.h"
#include "common.cuh"
#include "pages.h"
#include "pairs.cuh"

namespace fd {

namespace {

constexpr int kTableThreads = 1024;  // the one CTA of a table kernel

// ---- block-wide helpers of the table kernels (kTableThreads threads) -----------------------------

// Inclusive sum over the block's threads; *total (all threads) the sum. s_warp: 32 entries.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* s_warp, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();  // s_warp is free again
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  if (warp == 0) {
    T w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  *total = s_warp[31];
  return warp > 0 ? v + s_warp[warp - 1] : v;
}

// Leading non-negative entries among row[0, limit), by one warp (the same value in every lane); 256
// entries are in flight.
__device__ __forceinline__ int leading_pages(const int32_t* row, int limit) {
  const int lane = threadIdx.x & 31;
  for (int c0 = 0; c0 < limit; c0 += 256) {
    int32_t e[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = c0 + 32 * k + lane;
      e[k] = c < limit ? row[c] : 0;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const unsigned neg = __ballot_sync(0xffffffffu, e[k] < 0);
      if (neg) return c0 + 32 * k + __ffs(neg) - 1;
    }
  }
  return limit;
}

// Visit free pages (page_refs == 0) lowest index first: give(rank, page) for rank = 0 .. need - 1.
// Returns how many there were (need, or all of them when there are fewer). Four 16-byte loads a
// thread are in flight, i.e. 16384 pages a round; the four counts (each sum at most 4096) are
// scanned together as 16-bit fields.
template <typename Give>
__device__ __forceinline__ int64_t visit_free_pages(const int32_t* refs, int num_pages, int64_t need,
                                                    unsigned long long* s_warp, Give give) {
  const bool vec = (reinterpret_cast<uintptr_t>(refs) & 15u) == 0;
  int64_t base = 0;
  for (int64_t p0 = 0; p0 < num_pages && base < need; p0 += 16 * kTableThreads) {
    int32_t r[4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t p = p0 + 4 * (static_cast<int64_t>(k) * kTableThreads + threadIdx.x);
      if (vec && p + 4 <= num_pages) {
        const int4 v = *reinterpret_cast<const int4*>(refs + p);
        r[k][0] = v.x; r[k][1] = v.y; r[k][2] = v.z; r[k][3] = v.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[k][i] = p + i < num_pages ? refs[p + i] : 1;
      }
    }
    unsigned long long cnt = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        cnt += static_cast<unsigned long long>(r[k][i] == 0) << (16 * k);
    unsigned long long all;
    const unsigned long long before = block_scan(cnt, s_warp, &all) - cnt;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      int64_t rank = base + static_cast<int64_t>((before >> (16 * k)) & 0xffffu);
      const int64_t p = p0 + 4 * (static_cast<int64_t>(k) * kTableThreads + threadIdx.x);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r[k][i] == 0) {
          if (rank < need) give(rank, static_cast<int32_t>(p + i));
          ++rank;
        }
      base += static_cast<int64_t>((all >> (16 * k)) & 0xffffu);
    }
  }
  return base < need ? base : need;
}

// Index of the first entry of the increasing array s[0, n) that is > x (n when there is none).
template <typename T>
__device__ __forceinline__ int upper_bound(const T* s, int n, T x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (s[mid] > x) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// Inclusive sums of the values s[0, n) in place, by the block (n <= kMaxPlanBatch).
__device__ __forceinline__ int64_t scan_array(int64_t* s, int n, int64_t* s_warp) {
  int64_t run = 0;
  for (int i0 = 0; i0 < n; i0 += kTableThreads) {
    const int i = i0 + threadIdx.x;
    int64_t total;
    const int64_t v = block_scan<int64_t>(i < n ? s[i] : 0, s_warp, &total);
    if (i < n) s[i] = run + v;
    run += total;
  }
  __syncthreads();
  return run;
}

// ---- append ---------------------------------------------------------------------------------------

constexpr int kAppendThreads = 256;
constexpr int kAppendRows = 32;  // rows whose places one CTA looks up together
// Units a lane has in flight. E4M3: two, whose 64 registers keep 4 CTAs resident (four: 97, 2 CTAs).
template <bool kFp8>
constexpr int kAppendUnits = kFp8 ? 2 : 4;

// The 16-byte loads that one 16-byte unit of the destination needs.
template <typename S, bool kFp8>
struct AppendUnit {
  static constexpr int kLoads = kFp8 ? static_cast<int>(sizeof(S)) : 1;
  uint4 v[kLoads];
};

template <typename S, bool kFp8>
__device__ __forceinline__ void append_load(AppendUnit<S, kFp8>& a, const S* src) {
#pragma unroll
  for (int i = 0; i < AppendUnit<S, kFp8>::kLoads; ++i) a.v[i] = __ldg(reinterpret_cast<const uint4*>(src) + i);
}

// x / s rounded to fp32 as the division rounds it: one Newton step on x times the rounded reciprocal r
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor", 1990), for
// scales whose reciprocal the host gives (not 0). A zero's sign may be lost. Not for quotients near overflow, whose step would
// be NaN: those above 1e6 stay as the product gives them.
__device__ __forceinline__ float quotient(float x, float s, float r) {
  const float q = x * r;
  return fabsf(q) < 1e6f ? fmaf(fmaf(-q, s, x), r, q) : q;
}

// E4M3 codes of 16 values' magnitudes x / s under the signs of the values (s > 0), which stand in the
// upper bits of their words. Two quotients an instruction; the test for large ones is made once for all.
template <typename S, bool kFp8>
__device__ __forceinline__ uint4 append_convert(const AppendUnit<S, kFp8>& a, float scale, float recip) {
  if constexpr (!kFp8) {
    return a.v[0];
  } else {
    float x[16];
    uint32_t sign[4];  // of values 4 i .. 4 i + 3, in the bytes' upper bits
#pragma unroll
    for (int i = 0; i < AppendUnit<S, kFp8>::kLoads; ++i) {
      const uint32_t w[4] = {a.v[i].x, a.v[i].y, a.v[i].z, a.v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(S) == 4) {
          x[4 * i + j] = __uint_as_float(w[j]);
        } else {  // a bf16 is the upper half of the fp32 of the same value
          x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
          x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
      }
      if constexpr (sizeof(S) == 4) {
        sign[i] = __byte_perm(__byte_perm(w[0], w[1], 0x0073), __byte_perm(w[2], w[3], 0x0073), 0x5410);
      } else {
        sign[2 * i] = __byte_perm(w[0], w[1], 0x7531);
        sign[2 * i + 1] = __byte_perm(w[2], w[3], 0x7531);
      }
    }
    uint64_t q[8];
    const uint64_t r2 = pair_f32(recip, recip), s2 = pair_f32(-scale, -scale);
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      q[i] = fma_f32x2(pair_f32(x[2 * i], x[2 * i + 1]), r2, 0ull);
      float lo, hi;
      unpair_f32(q[i], lo, hi);
      most = fmaxf(most, fmaxf(fabsf(lo), fabsf(hi)));
    }
    if (recip != 0.f && most < 1e6f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint64_t rest = fma_f32x2(q[i], s2, pair_f32(x[2 * i], x[2 * i + 1]));
        unpair_f32(fma_f32x2(rest, r2, q[i]), x[2 * i], x[2 * i + 1]);
      }
    } else {  // a large value, or a scale that is divided by (recip 0)
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = recip != 0.f ? quotient(x[i], scale, recip) : __fdiv_rn(x[i], scale);
    }
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      asm("{\n\t.reg .b16 lo, hi;\n\t"
          "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
          "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
          "mov.b32 %0, {lo, hi};\n\t}"
          : "=r"(o[i])
          : "f"(x[4 * i]), "f"(x[4 * i + 1]), "f"(x[4 * i + 2]), "f"(x[4 * i + 3]));
      o[i] = (o[i] & 0x7f7f7f7fu) | (sign[i] & 0x80808080u);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// A CTA takes p.rows_per_cta packed rows. Every thread sums new_lens (the ends of the sequences,
// shared memory); one thread a row finds the row's sequence, page and slot; then a warp takes a row, K
// and V, in 16-byte units of the destination, two or four a lane in flight. Bound by HBM: 65,536 bf16 rows
// of 8 heads of 128 in 82 us (537 MB, 6.5 TB/s); E4M3 from bf16 by the conversion's instructions as well
// (~4 a value): 65,005 rows in 74 us (399 MB, 5.4 TB/s; 95 us with ~8 a value). One token of each of 64
// sequences: 3.7 us, three dependent loads and the launch.
template <typename S, bool kFp8>
__global__ void __launch_bounds__(kAppendThreads, 4) append_kernel(const AppendParams p) {
  extern __shared__ int64_t s_end[];  // [batch] ends of the sequences' packed rows
  __shared__ int64_t s_warp[kAppendThreads / 32];
  __shared__ int64_t s_place[kAppendRows];  // element offset of the row's place in both pools, < 0: none
  __shared__ int64_t s_total;
  constexpr int kUnits = kAppendUnits<kFp8>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_launch_dependents();
  pdl_wait_prerequisites();
  int64_t run = 0;
  for (int i0 = 0; i0 < p.batch; i0 += kAppendThreads) {
    const int i = i0 + tid;
    int64_t v = i < p.batch ? max(0, p.new_lens[i]) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = v;
    __syncthreads();
    int64_t before = run;
    for (int w = 0; w < kAppendThreads / 32; ++w) {
      if (w < warp) before += s_warp[w];
      run += s_warp[w];
    }
    if (i < p.batch) s_end[i] = before + v;
  }
  if (tid == 0) s_total = run;
  __syncthreads();
  const int64_t total = s_total;
  if (total > p.rows) {
    if (tid == 0 && blockIdx.x == 0) atomicOr(p.status, FD_FLAG_LEN_CLAMPED);
    return;
  }
  const int64_t cap = static_cast<int64_t>(p.pages_per_seq) * p.page_size;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * p.rows_per_cta; r0 < total;
       r0 += static_cast<int64_t>(gridDim.x) * p.rows_per_cta) {
    const int n = static_cast<int>(min(static_cast<int64_t>(p.rows_per_cta), total - r0));
    if (tid < n) {
      const int64_t r = r0 + tid;
      const int b = upper_bound(s_end, p.batch, r);
      const int64_t start = b > 0 ? s_end[b - 1] : 0;
      const int64_t pos = static_cast<int64_t>(p.start_lens[b]) + (r - start);
      int64_t place = -1;
      if (p.start_lens[b] < 0 || pos >= cap) {
        atomicOr(p.status, FD_FLAG_LEN_CLAMPED);
      } else {
        const int page = p.block_table[static_cast<int64_t>(b) * p.pages_per_seq + pos / p.page_size];
        if (page < 0 || page >= p.num_pages) {
          atomicOr(p.status, FD_FLAG_BAD_PAGE);
        } else {
          place = page * p.pool_sp + (pos % p.page_size) * p.d;
        }
      }
      s_place[tid] = place;
    }
    __syncthreads();
    const int per_head = p.d * (kFp8 ? 1 : static_cast<int>(sizeof(S))) / 16;  // a power of two
    const int shift = __ffs(per_head) - 1;
    const int elems = p.d / per_head;  // elements of one unit
    const int half = p.hkv * per_head;
    for (int i = warp; i < n; i += kAppendThreads / 32) {
      const int64_t place = s_place[i];
      if (place < 0) continue;
      const S* k_row = static_cast<const S*>(p.k_new) + (r0 + i) * p.k_sr;
      const S* v_row = static_cast<const S*>(p.v_new) + (r0 + i) * p.v_sr;
      for (int u0 = lane; u0 < 2 * half; u0 += 32 * kUnits) {
        AppendUnit<S, kFp8> x[kUnits];
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
          const int u = u0 + 32 * j, w = u >= half ? u - half : u;
          const int h = w >> shift, e = (w & (per_head - 1)) * elems;
          if (u < 2 * half) append_load(x[j], u >= half ? v_row + h * p.v_sh + e : k_row + h * p.k_sh + e);
        }
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
          const int u = u0 + 32 * j, w = u >= half ? u - half : u;
          const int h = w >> shift, e = (w & (per_head - 1)) * elems;
          if (u < 2 * half) {
            const uint4 c = append_convert(x[j], u >= half ? p.v_scale : p.k_scale, u >= half ? p.v_recip : p.k_recip);
            char* dst = static_cast<char*>(u >= half ? p.v_pages : p.k_pages) +
                        (place + h * p.pool_sh + e) * (kFp8 ? 1 : static_cast<int>(sizeof(S)));
            *reinterpret_cast<uint4*>(dst) = c;
          }
        }
      }
    }
    __syncthreads();
  }
}

// ---- reserve --------------------------------------------------------------------------------------

constexpr int kRowsAtOnce = 4;

// One CTA. A warp counts the pages of one sequence, or of four at a time where there are more sequences than
// warps; the missing ones, summed over the sequences, are the ranks of the free pages that
// visit_free_pages gives. If they run out, the sequences whose sum exceeds what there was give back what
// they got. Bound by the latency of its dependent loads (the rows, the references): a step of 32 sequences
// of up to 415 pages took 2.1 us longer with four rows a warp.
__global__ void __launch_bounds__(kTableThreads) reserve_kernel(const ReserveParams p) {
  extern __shared__ int64_t s_sum[];  // [batch] inclusive sums of the missing pages
  int32_t* s_have = reinterpret_cast<int32_t*>(s_sum + p.batch);
  __shared__ int64_t s_warp[32];
  __shared__ unsigned long long s_warp2[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_launch_dependents();
  pdl_wait_prerequisites();
  // the pages wanted, a thread a sequence; then what stands in the rows, a warp kRowsAtOnce rows together
  for (int b = threadIdx.x; b < p.batch; b += kTableThreads) {
    int64_t want = (max(static_cast<int64_t>(p.want_lens[b]), int64_t(0)) + p.page_size - 1) / p.page_size;
    if (want > p.pages_per_seq) {
      want = p.pages_per_seq;
      atomicOr(p.status, FD_FLAG_LEN_CLAMPED);
    }
    s_have[b] = static_cast<int32_t>(want);
    s_sum[b] = want;
  }
  __syncthreads();
  if (p.batch <= kTableThreads / 32) {  // a warp for every row
    if (warp < p.batch) {
      const int have = leading_pages(p.block_table + static_cast<int64_t>(warp) * p.pages_per_seq, s_have[warp]);
      __syncwarp();
      if (lane == 0) {
        s_have[warp] = have;
        s_sum[warp] -= have;
      }
    }
  } else {
    for (int b0 = warp * kRowsAtOnce; b0 < p.batch; b0 += kTableThreads / 32 * kRowsAtOnce) {
      int most = 0, limit[kRowsAtOnce];
#pragma unroll
      for (int i = 0; i < kRowsAtOnce; ++i) {
        limit[i] = b0 + i < p.batch ? s_have[b0 + i] : 0;
        most = max(most, limit[i]);
      }
      int have[kRowsAtOnce];
#pragma unroll
      for (int i = 0; i < kRowsAtOnce; ++i) have[i] = limit[i];
      for (int c0 = 0; c0 < most; c0 += 64) {
        int32_t e[kRowsAtOnce][2];
#pragma unroll
        for (int i = 0; i < kRowsAtOnce; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int c = c0 + 32 * k + lane;
            e[i][k] = c < limit[i] ? p.block_table[static_cast<int64_t>(b0 + i) * p.pages_per_seq + c] : 0;
          }
#pragma unroll
        for (int i = 0; i < kRowsAtOnce; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const unsigned neg = __ballot_sync(0xffffffffu, e[i][k] < 0);
            if (neg) have[i] = min(have[i], c0 + 32 * k + __ffs(neg) - 1);
          }
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kRowsAtOnce; ++i)
        if (lane == 0 && b0 + i < p.batch) {
          s_have[b0 + i] = have[i];
          s_sum[b0 + i] -= have[i];
        }
    }
  }
  __syncthreads();
  const int64_t need = scan_array(s_sum, p.batch, s_warp);
  if (need == 0) return;
  auto entry = [&](int64_t rank) {
    const int b = upper_bound(s_sum, p.batch, rank);
    return p.block_table + static_cast<int64_t>(b) * p.pages_per_seq + s_have[b] + (rank - (b > 0 ? s_sum[b - 1] : 0));
  };
  const int64_t got = visit_free_pages(p.page_refs, p.num_pages, need, s_warp2, [&](int64_t rank, int32_t page) {
    *entry(rank) = page;
    p.page_refs[page] = 1;
  });
  // a sequence ends behind its new pages: what stood behind the first negative entry does not join it
  for (int b = threadIdx.x; b < p.batch; b += kTableThreads) {
    const int64_t missing = s_sum[b] - (b > 0 ? s_sum[b - 1] : 0), pages = s_have[b] + missing;
    if (missing > 0 && s_sum[b] <= got && pages < p.pages_per_seq)
      p.block_table[static_cast<int64_t>(b) * p.pages_per_seq + pages] = -1;
  }
  if (got < need) {
    if (threadIdx.x == 0) atomicOr(p.status, FD_FLAG_POOL_FULL);
    __syncthreads();
    const int b = upper_bound(s_sum, p.batch, got);  // the first sequence that is not served
    for (int64_t r = (b > 0 ? s_sum[b - 1] : 0) + threadIdx.x; r < got; r += kTableThreads) {
      int32_t* e = entry(r);
      p.page_refs[*e] = 0;
      *e = -1;
    }
  }
}

// ---- fork -----------------------------------------------------------------------------------------

// One CTA plans the pairs: checks, new pages, rows and references; the copies of the last pages'
// rows (p.copies) are fork_copy_kernel's. Bound by the latency of its dependent loads: 16 pairs 11 us, 96
// pairs of up to 118 pages 22 us from a cold cache.
__global__ void __launch_bounds__(kTableThreads) fork_plan_kernel(const ForkParams p) {
  extern __shared__ int64_t s_sum[];  // [count] inclusive sums of the new pages
  int32_t* s_len = reinterpret_cast<int32_t*>(s_sum + p.count);  // [count] tokens, -1: skipped
  int32_t* s_page = s_len + p.count;                             // [count] new page
  int32_t* s_owner = s_page + p.count;                           // [batch] first pair of a destination
  __shared__ int64_t s_warp[32];
  __shared__ unsigned long long s_warp2[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_launch_dependents();
  pdl_wait_prerequisites();
  for (int b = threadIdx.x; b < p.batch; b += kTableThreads) s_owner[b] = INT32_MAX;
  __syncthreads();
  // the indices and lengths, a thread a pair; then the sources' pages, a warp a pair
  for (int i = threadIdx.x; i < p.count; i += kTableThreads) {
    const int src = p.src_seqs[i], dst = p.dst_seqs[i];
    bool ok = dst >= 0 && dst < p.batch;
    if (ok) atomicMin(&s_owner[dst], i);
    ok = ok && src >= 0 && src < p.batch;
    s_len[i] = ok ? p.cache_lens[src] : -1;
    s_sum[i] = ok && p.block_table[static_cast<int64_t>(dst) * p.pages_per_seq] < 0 ? 1 : 0;
  }
  __syncthreads();
  for (int i = warp; i < p.count; i += kTableThreads / 32) {
    const int src = p.src_seqs[i], dst = p.dst_seqs[i];
    int len = -1;
    uint32_t flag = 0;
    if (s_sum[i] == 0 || s_owner[dst] != i) {
      flag = FD_FLAG_BAD_INDEX;
    } else {
      len = s_len[i];
      const int64_t pages = (static_cast<int64_t>(len) + p.page_size - 1) / p.page_size;
      bool ok = len >= 0 && pages <= p.pages_per_seq;
      const int32_t* row = p.block_table + static_cast<int64_t>(src) * p.pages_per_seq;
      for (int64_t c0 = 0; ok && c0 < pages; c0 += 256) {
        int32_t e[8], f[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int64_t c = c0 + 32 * k + lane;
          e[k] = c < pages ? row[c] : -1;
          f[k] = c < pages ? 0 : 1;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (e[k] >= 0 && e[k] < p.num_pages) f[k] = p.page_refs[e[k]];
#pragma unroll
        for (int k = 0; k < 8; ++k) ok = ok && f[k] > 0;
      }
      if (!__all_sync(0xffffffffu, ok)) {
        len = -1;
        flag = FD_FLAG_BAD_PAGE;
      }
    }
    __syncwarp();  // s_len and s_sum are read
    if (lane == 0) {
      if (flag) atomicOr(p.status, flag);
      s_len[i] = len;
      s_sum[i] = len > 0 && len % p.page_size != 0 ? 1 : 0;
    }
  }
  __syncthreads();
  const int64_t need = scan_array(s_sum, p.count, s_warp);
  const int64_t got = visit_free_pages(p.page_refs, p.num_pages, need, s_warp2, [&](int64_t rank, int32_t page) {
    s_page[upper_bound(s_sum, p.count, rank)] = page;
  });
  if (got < need && threadIdx.x == 0) atomicOr(p.status, FD_FLAG_POOL_FULL);
  __syncthreads();
  for (int i = warp; i < p.count; i += kTableThreads / 32) {
    const int len = s_len[i];
    const bool fresh = s_sum[i] > (i > 0 ? s_sum[i - 1] : 0);
    int4 copy = make_int4(0, 0, 0, 0);
    if (len >= 0 && (!fresh || s_sum[i] <= got)) {
      const int src = p.src_seqs[i], dst = p.dst_seqs[i];
      const int full = len / p.page_size;
      const int32_t* from = p.block_table + static_cast<int64_t>(src) * p.pages_per_seq;
      int32_t* to = p.block_table + static_cast<int64_t>(dst) * p.pages_per_seq;
      for (int c0 = 0; c0 < p.pages_per_seq; c0 += 128) {
        int32_t page[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int c = c0 + 32 * k + lane;
          page[k] = c < full ? from[c] : c == full && fresh ? s_page[i] : -1;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int c = c0 + 32 * k + lane;
          if (c < p.pages_per_seq) to[c] = page[k];
          if (page[k] >= 0) atomicAdd(&p.page_refs[page[k]], 1);
        }
      }
      if (lane == 0) {
        p.cache_lens[dst] = len;
        if (fresh) copy = make_int4(from[full], s_page[i], len % p.page_size, 0);
      }
    }
    if (lane == 0) p.copies[i] = copy;
  }
}

constexpr int kCopyThreads = 256;

// Block (i, j): the K (j even) or V rows of KV head j / 2 of copy i, contiguous in both pages. 96 copies of
// up to 127 rows of 8 heads of 128 bf16: 9 us from a cold cache (51 MB).
__global__ void __launch_bounds__(kCopyThreads) fork_copy_kernel(const ForkParams p) {
  pdl_launch_dependents();
  pdl_wait_prerequisites();
  const int4 c = p.copies[blockIdx.x];
  if (c.z == 0) return;
  const int h = blockIdx.y >> 1;
  char* pool = static_cast<char*>((blockIdx.y & 1) ? p.v_pages : p.k_pages);
  const uint4* src = reinterpret_cast<const uint4*>(pool + c.x * p.pool_sp + h * p.pool_sh);
  uint4* dst = reinterpret_cast<uint4*>(pool + c.y * p.pool_sp + h * p.pool_sh);
  const int64_t n = static_cast<int64_t>(c.z) * p.row_bytes / 16;
  for (int64_t u0 = threadIdx.x; u0 < n; u0 += 8 * kCopyThreads) {
    uint4 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (u0 + k * kCopyThreads < n) x[k] = src[u0 + k * kCopyThreads];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (u0 + k * kCopyThreads < n) dst[u0 + k * kCopyThreads] = x[k];
  }
}

// ---- free -----------------------------------------------------------------------------------------

constexpr int kFreeThreads = 128;

// One CTA a listed sequence; the first of equal entries frees it. 4 us for 16 to 96 sequences: latency.
__global__ void __launch_bounds__(kFreeThreads) free_kernel(const FreeParams p) {
  const int i = blockIdx.x, tid = threadIdx.x;
  pdl_launch_dependents();
  pdl_wait_prerequisites();
  const int b = p.seqs[i];
  if (b < 0 || b >= p.batch) {
    if (tid == 0) atomicOr(p.status, FD_FLAG_BAD_INDEX);
    return;
  }
  bool first = true;
  for (int j = tid; j < i; j += kFreeThreads) first = first && p.seqs[j] != b;
  if (!__syncthreads_and(first)) return;
  int32_t* row = p.block_table + static_cast<int64_t>(b) * p.pages_per_seq;
  for (int c0 = 0; c0 < p.pages_per_seq; c0 += kFreeThreads) {
    const int c = c0 + tid;
    const int32_t page = c < p.pages_per_seq ? row[c] : -1;
    // the sequence's pages end at the first negative entry, wherever it stands in this stretch
    __shared__ int s_end;
    __syncthreads();
    if (tid == 0) s_end = kFreeThreads;
    __syncthreads();
    if (page < 0) atomicMin(&s_end, tid);
    __syncthreads();
    if (tid < s_end) {
      row[c] = -1;
      drop_reference(p.page_refs, p.num_pages, page, p.status);
    }
    if (s_end < kFreeThreads) break;
  }
  if (tid == 0) p.cache_lens[b] = 0;
}

// ---- compact --------------------------------------------------------------------------------------

constexpr int kCompactThreads = 256;

// Whether sequence b's compaction is valid (all threads get the answer); *first: its first moved
// index. Reads the table and the references, which no CTA of compact_move_kernel writes.
__device__ __forceinline__ bool check_compact(const CompactParams& p, int b, int m, int* first, bool report) {
  const int32_t start = p.start_lens[b];
  const int32_t* keep = p.keep + static_cast<int64_t>(b) * p.max_keep;
  const int64_t cap = static_cast<int64_t>(p.pages_per_seq) * p.page_size;
  __shared__ int s_first;
  __syncthreads();
  if (threadIdx.x == 0) s_first = m;
  __syncthreads();
  bool ok = start >= 0 && m <= p.max_keep;
  if (ok) {
    for (int i = threadIdx.x; i < m; i += kCompactThreads) {
      const int k = keep[i];
      ok = ok && k > (i > 0 ? keep[i - 1] : -1);
      if (k != i) atomicMin(&s_first, i);
    }
  }
  const int64_t last = m > 0 && ok ? static_cast<int64_t>(start) + keep[m - 1] : static_cast<int64_t>(start) + m - 1;
  ok = ok && last < cap && static_cast<int64_t>(start) + m <= cap;
  if (!__syncthreads_and(ok)) {
    if (report && threadIdx.x == 0) atomicOr(p.status, FD_FLAG_BAD_INDEX);
    return false;
  }
  *first = s_first;
  if (s_first >= m) return true;
  // the pages from the first moved position to the last one read; the written ones are unshared
  const int64_t c0 = (static_cast<int64_t>(start) + s_first) / p.page_size, c1 = last / p.page_size;
  const int64_t cw = (static_cast<int64_t>(start) + m - 1) / p.page_size;
  const int32_t* row = p.block_table + static_cast<int64_t>(b) * p.pages_per_seq;
  for (int64_t c = threadIdx.x; c <= c1; c += kCompactThreads) {
    const int32_t page = row[c];
    ok = ok && page >= 0 && (c < c0 || (page < p.num_pages && (c > cw || p.page_refs[page] == 1)));
  }
  if (!__syncthreads_and(ok)) {
    if (report && threadIdx.x == 0) atomicOr(p.status, FD_FLAG_BAD_PAGE);
    return false;
  }
  return true;
}

// Block (b, j): moves the rows of K (j even) or V, KV head j / 2, of sequence b, a batch of kMove rows a
// thread after the other. The list increases strictly, so a row read lies at or behind the row written for
// it: rows read for a later batch lie behind every row written for an earlier one. A batch's rows are
// therefore loaded before the batch before it is stored, and only a batch's own loads and stores need the
// barrier between them. The places of a batch are looked up one thread a row, in a ring of four: its
// list entries four batches ahead, its pages three, both waited for a batch later, so that a batch costs one
// memory latency and not the lookup's two behind each other: half of 16 x 4096 tokens (8 heads of 128
// bf16, 268 MB) in 53 us, 5.1 TB/s, instead of 79.
constexpr int kMove = 8;
constexpr int kMoveRows = kMove * kCompactThreads / 4;  // rows of a batch at most (64-byte rows)
__global__ void __launch_bounds__(kCompactThreads) compact_move_kernel(const CompactParams p) {
  __shared__ int64_t s_from[4][kMoveRows], s_to[4][kMoveRows];
  pdl_launch_dependents();
  pdl_wait_prerequisites();
  const int b = blockIdx.x, tid = threadIdx.x;
  const int m = p.keep_lens[b];
  int first = 0;
  const bool go = m >= 0 && check_compact(p, b, m, &first, blockIdx.y == 0);
  if (blockIdx.y == 0 && tid == 0) p.valid[b] = go ? 1 : 0;
  if (!go || first >= m) return;
  const int h = blockIdx.y >> 1;
  char* pool = static_cast<char*>((blockIdx.y & 1) ? p.v_pages : p.k_pages) + h * p.pool_sh;
  const int units = p.row_bytes / 16;  // 4 .. 32, a power of two
  const int per = kCompactThreads / units, batch = kMove * per;
  const int unit = tid & (units - 1), slot = tid / units;
  const int32_t start = p.start_lens[b];
  const int32_t* keep = p.keep + static_cast<int64_t>(b) * p.max_keep;
  const int32_t* row = p.block_table + static_cast<int64_t>(b) * p.pages_per_seq;
  // lookups in flight: of the batch whose list entries are read, and of the one whose pages are
  constexpr int kLook = kMoveRows / kCompactThreads;
  int entry[kLook], pos[kLook], page_from[kLook], page_to[kLook];
  auto each = [&](int n, auto f) {
#pragma unroll
    for (int k = 0; k < kLook; ++k) {
      const int at = k * kCompactThreads + tid, i = first + n * batch + at;
      if (at < batch && i < m) f(k, at, i);
    }
  };
  auto read_list = [&](int n) { each(n, [&](int k, int, int i) { entry[k] = keep[i]; }); };
  auto read_pages = [&](int n) {
    each(n, [&](int k, int, int i) {
      pos[k] = start + entry[k];
      page_from[k] = row[pos[k] / p.page_size];
      page_to[k] = row[(start + i) / p.page_size];
    });
  };
  auto put_places = [&](int n) {
    each(n, [&](int k, int at, int i) {
      s_from[n & 3][at] = page_from[k] * p.pool_sp + static_cast<int64_t>(pos[k] % p.page_size) * p.row_bytes;
      s_to[n & 3][at] = page_to[k] * p.pool_sp + static_cast<int64_t>((start + i) % p.page_size) * p.row_bytes;
    });
  };
  auto look_up = [&](int n) {  // the places of batch n, and what the next two need
    put_places(n);
    read_pages(n + 1);
    read_list(n + 2);
  };
  auto load = [&](int n, uint4 (&x)[kMove]) {
#pragma unroll
    for (int k = 0; k < kMove; ++k)
      if (first + n * batch + k * per + slot < m)
        x[k] = reinterpret_cast<const uint4*>(pool + s_from[n & 3][k * per + slot])[unit];
  };
  auto store = [&](int n, const uint4 (&x)[kMove]) {
#pragma unroll
    for (int k = 0; k < kMove; ++k)
      if (first + n * batch + k * per + slot < m) reinterpret_cast<uint4*>(pool + s_to[n & 3][k * per + slot])[unit] = x[k];
  };
  const int batches = (m - first + batch - 1) / batch;
  uint4 x[kMove], y[kMove];
  read_list(0);
  read_pages(0);
  read_list(1);
  look_up(0);
  look_up(1);
  __syncthreads();
  load(0, x);
  // two batches a round, so that the registers keep their roles
  for (int n = 0; n < batches; n += 2) {
    if (n + 1 < batches) load(n + 1, y);
    look_up(n + 2);
    __syncthreads();  // everyone has loaded batch n (and n + 1)
    store(n, x);
    if (n + 1 >= batches) break;
    if (n + 2 < batches) load(n + 2, x);
    look_up(n + 3);
    __syncthreads();
    store(n + 1, y);
  }
}

// One CTA a sequence: the new length, the pages behind it given back.
__global__ void __launch_bounds__(kFreeThreads) compact_table_kernel(const CompactParams p) {
  const int b = blockIdx.x, tid = threadIdx.x;
  pdl_launch_dependents();
  pdl_wait_prerequisites();
  const int m = p.keep_lens[b];
  if (m < 0 || !p.valid[b]) return;
  const int64_t len = static_cast<int64_t>(p.start_lens[b]) + m;
  int32_t* row = p.block_table + static_cast<int64_t>(b) * p.pages_per_seq;
  const int from = static_cast<int>((len + p.page_size - 1) / p.page_size);
  __shared__ int s_end;
  if (tid < 32) {
    const int n = leading_pages(row, p.pages_per_seq);
    if (tid == 0) s_end = n;
  }
  __syncthreads();
  for (int c = from + tid; c < s_end; c += kFreeThreads) {
    const int32_t page = row[c];
    row[c] = -1;
    drop_reference(p.page_refs, p.num_pages, page, p.status);
  }
  if (tid == 0) p.cache_lens[b] = static_cast<int32_t>(len);
}

}  // namespace

// ---- launchers ------------------------------------------------------------------------------------

// Launched with programmatic stream serialization: a kernel becomes resident while the one before it
// runs, and waits for it before it reads or writes anything.
// `most`: the dynamic shared memory of the largest call, `smem` that of this one.
template <typename P>
static cudaError_t launch(void (*kernel)(P), dim3 grid, int threads, size_t smem, size_t most, cudaStream_t stream, const P& p) {
  const cudaError_t e = allow_dynamic_smem(kernel, smem, most);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

cudaError_t launch_append(AppendParams p, int src_dtype, bool fp8, int nsm, cudaStream_t stream) {
  const int64_t want = (p.rows + 8 * nsm - 1) / (8 * nsm);
  p.rows_per_cta = static_cast<int>(want < 1 ? 1 : want > kAppendRows ? kAppendRows : want);
  int64_t grid = (p.rows + p.rows_per_cta - 1) / p.rows_per_cta;
  if (grid > 16 * nsm) grid = 16 * nsm;
  void (*kernel)(AppendParams) = src_dtype == FD_F32 ? (fp8 ? append_kernel<float, true> : append_kernel<float, false>)
                                                     : (fp8 ? append_kernel<__nv_bfloat16, true> : append_kernel<__nv_bfloat16, false>);
  return launch(kernel, dim3(static_cast<unsigned>(grid)), kAppendThreads, sizeof(int64_t) * p.batch,
                sizeof(int64_t) * kMaxPlanBatch, stream, p);
}

cudaError_t launch_reserve(const ReserveParams& p, cudaStream_t stream) {
  const auto smem = [](int32_t batch) { return static_cast<size_t>(batch) * 12; };
  return launch(reserve_kernel, dim3(1), kTableThreads, smem(p.batch), smem(kMaxPlanBatch), stream, p);
}

cudaError_t launch_fork(const ForkParams& p, cudaStream_t stream) {
  const auto smem = [](int32_t count, int32_t batch) { return static_cast<size_t>(count) * 16 + static_cast<size_t>(batch) * 4; };
  const cudaError_t e = launch(fork_plan_kernel, dim3(1), kTableThreads, smem(p.count, p.batch), smem(kMaxPlanBatch, kMaxPlanBatch),
                               stream, p);
  if (e != cudaSuccess) return e;
  return launch(fork_copy_kernel, dim3(p.count, 2 * p.hkv), kCopyThreads, 0, 0, stream, p);
}

cudaError_t launch_free(const FreeParams& p, cudaStream_t stream) {
  return launch(free_kernel, dim3(p.count), kFreeThreads, 0, 0, stream, p);
}

cudaError_t launch_compact(const CompactParams& p, cudaStream_t stream) {
  const cudaError_t e = launch(compact_move_kernel, dim3(p.batch, 2 * p.hkv), kCompactThreads, 0, 0, stream, p);
  if (e != cudaSuccess) return e;
  return launch(compact_table_kernel, dim3(p.batch), kFreeThreads, 0, 0, stream, p);
}

}  // namespace fd
