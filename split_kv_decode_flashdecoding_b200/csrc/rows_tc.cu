// Attention of packed query rows (whole prompts, drafted trees) on the 5th-generation tensor cores.
//
// Mathematics, per query row with visible keys J, s_j = q·k_j log2(e) / sqrt(D):
//   m = max_J s_j;  l = sum_J 2^(s_j - m);  o = sum_J 2^(s_j - m) v_j / l;  lse = (m + log2 l) ln 2
// in one pass over 128-key tiles with the running m and l of an online softmax.
//
// An item (rows_plan.h) is up to 256 rows, two tiles of 128 (T = 128 / G tokens x the G query heads of
// one KV head: tile row r is token r / G of query head h G + r mod G), that walk the same key tiles:
//   S = Q_tile · K_tileᵀ     UMMA M 128, N 128, K D      (TMEM, fp32)
//   P = 2^(S scale - m)      one thread a row, bf16 over S's columns
//   O += P · V_tile          UMMA M 128, N D, K 128, P from TMEM
// The two tiles are two independent chains ("lanes") that share the K/V ring: while one lane's
// softmax runs, the tensor cores work for the other, so S, P and O need no second buffer and fill
// tensor memory exactly (2 x 128 columns of S / P, 2 x D of O). An item of at most T tokens has one
// row tile; its two lanes then take alternate key tiles and the epilogue adds their results, so a
// small tree's softmax still runs on eight warps.
//
// Rounding choice: P is rounded to bf16 (nearest) for the product with V, as V itself is bf16; l sums
// the unrounded fp32 weights. The output then carries a relative error of 2^-8 of sum p |v| / l at
// most, like its own rounding to bf16. The reference maximum moves only when the row's maximum grows
// by more than 2^8 (weights up to 2^8 are as exact), so O is rarely rescaled.
//
// What masks leave out never enters: scores of invisible keys become -inf before the maximum, V rows
// behind the last key are zeroed in shared memory, and rows of other requests share a tile only as
// rows or columns that nothing reads. Work is divided by rows_plan.h; the pieces of a cut item meet
// in the workspace and the last of its CTAs adds them in piece order, so results do not depend on
// which one that is.
//
// Warps: 0-3 and 4-7 softmax of lanes 0 and 1 (warp w reads TMEM lanes 32 (w mod 4) + [0, 32), one row a
// thread); 8-11 epilogue; 12 plan and TMA; 13, 14 tensor-core issue of lanes 0 and 1.
#include "common.cuh"
#include "rows.h"
#include "rows_plan.h"

namespace fd {

namespace {

constexpr int kRwThreads = 16 * 32;
constexpr int kRwEpi = 8, kRwProducer = 12, kRwIssue = 13;
constexpr int kRwItems = 4;                    // item descriptors in flight
constexpr uint32_t kRwTmemCols = 512;
constexpr uint32_t kRwColO = 256;              // O of lane L at kRwColO + L D; S / P of lane L at 128 L
constexpr uint32_t kRwHalf = 128 * 64 * 2;     // bytes of one 64-column half of a 128-row tile
constexpr float kRwRescale = 8.0f;             // log2 units

enum RowSource { kSrcPacked = 0, kSrcCache = 1, kSrcPaged = 2 };

struct RowItem {
  int32_t stop;
  int32_t b, h;             // request, KV head
  int32_t row0, t0, nt;     // packed row of the first token; its index in the request; tokens
  int32_t key_row0;         // prompt: packed row of the request's first key
  int32_t tile0, ntile;     // key tiles [tile0, tile0 + ntile)
  int32_t k1;               // keys of the item (all pieces): tiles hold keys < k1
  int32_t prefix;           // tree: keys every row sees
  int32_t alt;              // one row tile, the lanes take alternate key tiles
  int32_t cut0, cuts, piece;  // rows_cuts of a cut item (cuts 0: whole), this piece's index
};

template <int kD>
struct __align__(1024) RwSmem {
  static constexpr int kHalves = kD / 64;
  static constexpr int kStages = kD == 128 ? 4 : 8;  // K and V tiles alternate
  __nv_bfloat16 q[2][kHalves][128 * 64];
  __nv_bfloat16 kv[kStages][kHalves][128 * 64];
  RowItem item[kRwItems];
  float mfin[2][2][128], lfin[2][2][128];  // [item parity][lane][row]
  int64_t part_w[kRwThreads];              // plan: work, rows and items of a thread's requests
  int32_t part_r[kRwThreads], part_i[kRwThreads];
  uint64_t full[kStages], empty[kStages];
  uint64_t qfull[2], qempty[2], ifull[kRwItems], iempty[kRwItems];
  uint64_t sfull[2], pfull[2], pvdone[2], ofin[2], oempty[2];
  uint64_t lready[2][2], lfree[2][2];
  uint64_t drain[2];
  uint32_t tmem_base;
  int abort_flag;
  int bad;
};
static_assert(sizeof(RwSmem<128>) + 1024 <= 227 * 1024, "row attention shared memory");
static_assert(sizeof(RwSmem<64>) + 1024 <= 227 * 1024, "row attention shared memory");

// ---- arithmetic on pairs of fp32 ------------------------------------------------------------------

__device__ __forceinline__ uint64_t pair_f32(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair_f32(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3_f32(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <uint32_t kRegs>
__device__ __forceinline__ void set_regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <uint32_t kRegs>
__device__ __forceinline__ void set_regs_less() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// The bounded waits of common.cuh with the polling loop in line: a kernel that re-divides its
// registers between warps (setmaxnreg) cannot call a function. The status word is raised once, at
// the kernel's end.
__device__ __forceinline__ bool row_poll(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  do {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return true;
  } while (global_timer_ns() - t0 <= kWaitLimitNs);
  return false;
}
__device__ __forceinline__ bool row_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (row_poll(bar, parity)) return true;
  *abort_flag = 1;
  return false;
}

// n low bits set (n <= 0: none, n >= 32: all).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
}

// Lane L's tokens of an item, and the tiles it works on: the i-th is tile0 + first + i step.
struct LaneView {
  int nt, kend, used, first, step;
};
__device__ __forceinline__ LaneView lane_view(const RowItem& it, int lane_no, int tpt, bool causal) {
  LaneView v;
  const int at = it.alt ? 0 : lane_no * tpt;
  v.nt = it.alt ? it.nt : max(0, min(tpt, it.nt - at));
  v.kend = causal ? it.t0 + at + v.nt : it.k1;
  if (it.alt) {
    v.used = (it.ntile + 1 - lane_no) >> 1;
    v.first = lane_no;
    v.step = 2;
  } else {
    v.used = v.nt > 0 ? max(0, min(it.ntile, ((v.kend + 127) >> 7) - it.tile0)) : 0;
    v.first = 0;
    v.step = 1;
  }
  return v;
}

// The 32-key visibility words of one row in a key tile (bit i of word c: key 128 tile + 32 c + i).
template <bool kCausal>
__device__ __forceinline__ void visible_words(const RowsParams& p, const RowItem& it, int tile, int pos, bool row_ok,
                                              int64_t row, uint32_t (&w)[4]) {
  const int k0 = tile * 128;
  if constexpr (kCausal) {
    const int n = row_ok ? min(it.k1, it.t0 + pos + 1) - k0 : 128;
#pragma unroll
    for (int c = 0; c < 4; ++c) w[c] = low_bits(n - 32 * c);
  } else {
    const uint32_t* mask = p.mask + row * p.mask_words;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int base = k0 + 32 * c - it.prefix;  // draft index of the word's first key
      uint32_t x = 0xffffffffu;
      if (base > -32 && row_ok) {
        const int idx = base >> 5;  // floor: -1 when the word starts in the prefix
        const uint32_t lo = idx < 0 ? 0xffffffffu : idx < p.mask_words ? mask[idx] : 0u;
        const uint32_t hi = idx + 1 < p.mask_words ? mask[idx + 1] : 0u;
        x = __funnelshift_r(lo, hi, base & 31);
      }
      w[c] = x & low_bits(it.k1 - k0 - 32 * c);
    }
  }
}

template <int kD, int kSrc>
__global__ void __launch_bounds__(kRwThreads, 1)
    rows_tc_kernel(const RowsParams p, const __grid_constant__ CUtensorMap tmap_q,
                   const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v) {
  using Smem = RwSmem<kD>;
  constexpr bool kCausal = kSrc == kSrcPacked;
  constexpr int kHalves = Smem::kHalves, kStages = Smem::kStages;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  Smem& S = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tpt = rows_tile_tokens(p.g);

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&S.full[s], 1);
      mbar_init(&S.empty[s], 2);  // both lanes' issuers
    }
    for (int i = 0; i < kRwItems; ++i) {
      mbar_init(&S.ifull[i], 1);
      mbar_init(&S.iempty[i], 8 + 4 + 2);  // softmax and epilogue warps, issuers
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.qfull[i], 1);
      mbar_init(&S.qempty[i], 1);
      mbar_init(&S.sfull[i], 1);
      mbar_init(&S.pfull[i], 4);
      mbar_init(&S.pvdone[i], 1);
      mbar_init(&S.ofin[i], 1);
      mbar_init(&S.oempty[i], 4);
      for (int j = 0; j < 2; ++j) {
        mbar_init(&S.lready[i][j], 4);
        mbar_init(&S.lfree[i][j], 4);
      }
      mbar_init(&S.drain[i], 1);
    }
    S.abort_flag = 0;
    S.bad = 0;
    fence_mbar_init();
  }
  if (warp == kRwIssue) {
    tmem_alloc(&S.tmem_base, kRwTmemCols);
    tmem_relinquish();
  }
  if (warp == kRwProducer && lane == 0) {
    prefetch_tensor_map(&tmap_q);
    prefetch_tensor_map(&tmap_k);
    prefetch_tensor_map(&tmap_v);
  }
  pdl_launch_dependents();
  pdl_wait_prerequisites();
  __syncthreads();  // S.bad is set

  // The requests' work: thread t sums those of its stretch of the batch.
  const int per = (p.batch + kRwThreads - 1) / kRwThreads;
  auto request = [&](int b, int* n, int* keys, int* prefix) {
    const int len = p.row_lens[b];
    *n = max(len, 0);
    *keys = *n;
    *prefix = 0;
    uint32_t flag = len < 0 ? FD_FLAG_LEN_CLAMPED : 0u;
    if constexpr (!kCausal) {
      if (len < 0 || len > 32 * p.mask_words) S.bad = 1;
      const int pre = p.prefix_lens[b];
      *prefix = clamp_len(pre, p.cap);
      const int64_t end = static_cast<int64_t>(*prefix) + *n;
      *keys = static_cast<int>(min(end, static_cast<int64_t>(p.cap)));
      if (*prefix != pre || *keys != end) flag = FD_FLAG_LEN_CLAMPED;
    }
    return flag;
  };
  {
    int64_t w = 0, rows = 0;
    int items = 0;
    uint32_t flag = 0;
    for (int i = 0; i < per; ++i) {
      const int b = tid * per + i;
      if (b >= p.batch) break;
      int n, keys, prefix;
      flag |= request(b, &n, &keys, &prefix);
      const int pairs = rows_pairs(n, tpt);
      w += p.hkv * rows_weight(kCausal, tpt, keys, pairs);
      rows += n;
      items += pairs;
    }
    if (rows > p.rows) S.bad = 1;
    if (flag && blockIdx.x == 0) atomicOr(&p.hdr->status, flag);
    S.part_w[tid] = w;
    S.part_r[tid] = static_cast<int32_t>(min(rows, static_cast<int64_t>(p.rows) + 1));
    S.part_i[tid] = items;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;

  if (warp >= kRwProducer) {
    set_regs_less<72>();
    if (warp == kRwProducer) {
      // ======================= plan and TMA =======================
      // Totals of the threads' stretches, 16 a lane, then this CTA's stretch of the work.
      int64_t mine_w = 0, mine_r = 0, mine_i = 0;
      for (int i = 0; i < kRwThreads / 32; ++i) {
        mine_w += S.part_w[lane * (kRwThreads / 32) + i];
        mine_r += S.part_r[lane * (kRwThreads / 32) + i];
        mine_i += S.part_i[lane * (kRwThreads / 32) + i];
      }
      int64_t sum_w = mine_w, sum_r = mine_r, sum_i = mine_i;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t a = __shfl_up_sync(0xffffffffu, sum_w, o), b = __shfl_up_sync(0xffffffffu, sum_r, o);
        if (lane >= o) { sum_w += a; sum_r += b; }
        sum_i += __shfl_xor_sync(0xffffffffu, sum_i, o);
      }
      const int64_t weight = __shfl_sync(0xffffffffu, sum_w, 31), rows = __shfl_sync(0xffffffffu, sum_r, 31);
      bool ok = true;
      uint32_t T = 0, K = 0;  // key tiles and items so far
      const bool bad = S.bad != 0 || rows > p.rows;
      if (bad && blockIdx.x == 0 && lane == 0) atomicOr(&p.hdr->status, FD_FLAG_LEN_CLAMPED);
      const int nact = bad || weight == 0 ? 0 : rows_active(weight, sum_i * p.hkv, static_cast<int>(gridDim.x));
      if (static_cast<int>(blockIdx.x) < nact) {
        const int cta = blockIdx.x;
        const int64_t x0 = rows_bound(weight, nact, cta), x1 = rows_bound(weight, nact, cta + 1);
        // the request that x0 falls into: its lane, its thread's stretch, then one by one
        const unsigned at = __ballot_sync(0xffffffffu, sum_w > x0);
        const int src = __ffs(at) - 1;  // sum_w of the last lane is weight > x0
        int64_t base = __shfl_sync(0xffffffffu, sum_w - mine_w, src), row = __shfl_sync(0xffffffffu, sum_r - mine_r, src);
        int t = src * (kRwThreads / 32);
        while (base + S.part_w[t] <= x0) {
          base += S.part_w[t];
          row += S.part_r[t];
          ++t;
        }
        int b = t * per, n, keys, prefix;
        request(b, &n, &keys, &prefix);
        int64_t all = p.hkv * rows_weight(kCausal, tpt, keys, rows_pairs(n, tpt));
        while (base + all <= x0) {
          base += all;
          row += n;
          request(++b, &n, &keys, &prefix);
          all = p.hkv * rows_weight(kCausal, tpt, keys, rows_pairs(n, tpt));
        }
        int pairs = rows_pairs(n, tpt);
        int64_t per_head = rows_weight(kCausal, tpt, keys, pairs);
        int h = static_cast<int>((x0 - base) / per_head);
        int64_t a = base + h * per_head;
        int u = 0;
        for (int hi = pairs; hi - u > 1;) {  // the last u whose items before it end at or before x0
          const int mid = (u + hi) >> 1;
          if (a + rows_weight(kCausal, tpt, keys, mid) <= x0) u = mid; else hi = mid;
        }
        while (ok) {
          const int64_t a0 = a + rows_weight(kCausal, tpt, keys, u);
          if (a0 >= x1) break;
          const int64_t w = a + rows_weight(kCausal, tpt, keys, u + 1) - a0;
          const int k1 = rows_item_keys(kCausal, tpt, n, keys, u);
          const int tiles = (k1 + 127) >> 7;
          const int c0 = rows_cut(x0, a0, w, tiles), c1 = rows_cut(x1, a0, w, tiles);
          if (c0 < c1) {
            // ---- one piece: its descriptor, K of its first tile, Q, the rest ----
            RowItem it;
            it.stop = 0;
            it.b = b;
            it.h = h;
            it.t0 = u * 2 * tpt;
            it.nt = min(2 * tpt, n - it.t0);
            it.row0 = static_cast<int>(row) + it.t0;
            it.key_row0 = static_cast<int>(row);
            it.tile0 = c0;
            it.ntile = c1 - c0;
            it.k1 = k1;
            it.prefix = prefix;
            it.alt = it.nt <= tpt;
            it.cut0 = it.cuts = it.piece = 0;
            if (c0 > 0 || c1 < tiles) {
              rows_cuts(weight, nact, a0, w, tiles, cta, &it.cut0, &it.cuts);
              it.piece = cta + 1 - it.cut0;
            }
            const int slot = K & (kRwItems - 1);
            if (!row_wait(&S.iempty[slot], ((K / kRwItems) & 1u) ^ 1u, &S.abort_flag)) { ok = false; break; }
            if (lane == 0) {
              S.item[slot] = it;
              mbar_arrive(&S.ifull[slot]);
            }
            __syncwarp();
            // where a tile's keys lie: this lane's box (paged), else all of the tile (lane 0)
            const int psz = kSrc == kSrcPaged ? min(p.page_size, 128) : 128;
            const int boxes = kSrc == kSrcPaged ? (128 / psz) * kHalves : kHalves;
            const int box_page = lane / kHalves, box_half = lane % kHalves;
            auto page_of = [&](int tile) -> int {
              if constexpr (kSrc == kSrcPaged) {
                const int key = tile * 128 + box_page * psz;
                if (lane < boxes && key < k1) {
                  const int id = p.block_table[static_cast<int64_t>(b) * p.pages_per_seq + key / p.page_size];
                  if (id >= 0 && id < p.num_pages) return id;
                  atomicOr(&p.hdr->status, FD_FLAG_BAD_PAGE);
                }
                return p.num_pages;  // outside the map: the copy writes zeros
              }
              return 0;
            };
            auto load = [&](const CUtensorMap* map, uint32_t c, int tile, int page) -> bool {
              const int st = c % kStages;
              if (!row_wait(&S.empty[st], ((c / kStages) & 1u) ^ 1u, &S.abort_flag)) return false;
              if (lane == 0) mbar_arrive_expect_tx(&S.full[st], kHalves * 128u * static_cast<uint32_t>(p.kv_box_rows * (128 / psz)));
              __syncwarp();
              if (lane < boxes) {
                __nv_bfloat16* dst = S.kv[st][box_half] + box_page * psz * 64;
                if constexpr (kSrc == kSrcPacked) tma_load_3d(dst, map, &S.full[st], 64 * box_half, h, it.key_row0 + tile * 128);
                else if constexpr (kSrc == kSrcCache) tma_load_4d(dst, map, &S.full[st], 64 * box_half, tile * 128, h, b);
                else tma_load_4d(dst, map, &S.full[st], 64 * box_half, tile * 128 % p.page_size, h, page);
              }
              return true;
            };
            int page = page_of(c0);
            for (int j = c0; ok && j < c1; ++j, ++T) {
              if (!load(&tmap_k, 2 * T, j, page)) { ok = false; break; }
              if (j == c0) {
                for (int L = 0; ok && L < 2; ++L) {
                  if (!row_wait(&S.qempty[L], (K & 1u) ^ 1u, &S.abort_flag)) { ok = false; break; }
                  if (lane == 0) mbar_arrive_expect_tx(&S.qfull[L], kHalves * 128u * static_cast<uint32_t>(p.g * p.q_box_rows));
                  __syncwarp();
                  if (lane < kHalves)
                    tma_load_3d(S.q[L][lane], &tmap_q, &S.qfull[L], 64 * lane, h * p.g, it.row0 + (it.alt ? 0 : L * tpt));
                }
                if (!ok) break;
              }
              if (!load(&tmap_v, 2 * T + 1, j, page)) { ok = false; break; }
              if (j + 1 < c1) page = page_of(j + 1);
            }
            ++K;
          }
          if (++u == pairs) {
            u = 0;
            a += per_head;
            if (++h == p.hkv) {
              h = 0;
              base += all;
              row += n;
              do {  // the next request with rows
                if (++b >= p.batch) break;
                request(b, &n, &keys, &prefix);
              } while (n == 0);
              if (b >= p.batch) break;
              pairs = rows_pairs(n, tpt);
              per_head = rows_weight(kCausal, tpt, keys, pairs);
              all = p.hkv * per_head;
              a = base;
            }
          }
        }
      }
      if (ok) {
        const int slot = K & (kRwItems - 1);
        if (row_wait(&S.iempty[slot], ((K / kRwItems) & 1u) ^ 1u, &S.abort_flag) && lane == 0) {
          S.item[slot].stop = 1;
          mbar_arrive(&S.ifull[slot]);
        }
      }
      __syncwarp();
      if (S.abort_flag && lane == 0) {  // copies still in flight land before the CTA leaves
        for (uint32_t back = 1; back <= kStages + 1u && back <= 2 * T + 1; ++back) {
          const uint32_t c = 2 * T + 1 - back;
          (void)row_poll(&S.full[c % kStages], (c / kStages) & 1u);
        }
        for (int L = 0; L < 2; ++L) {
          if (K > 0) (void)row_poll(&S.qfull[L], (K - 1) & 1u);
          (void)row_poll(&S.qfull[L], K & 1u);
        }
      }
    } else if (warp < kRwIssue + 2 && lane == 0) {
      // ======================= tensor-core issue of one lane =======================
      const int L = warp - kRwIssue;
      const uint32_t s_col = tmem + 128 * L, o_col = tmem + kRwColO + kD * L;
      const uint32_t idesc_s = idesc_bf16_f32(128, 128, false, false);
      const uint32_t idesc_o = idesc_bf16_f32(128, kD, false, true);
      const uint64_t qd0 = smem_desc(smem_u32(S.q[L][0]), 16, 1024, kLayoutSW128);
      uint32_t T = 0, J = 0;  // key tiles of the items so far; tiles this lane has used
      bool ok = true;
      for (uint32_t K = 0; ok; ++K) {
        const int slot = K & (kRwItems - 1);
        if (!row_wait(&S.ifull[slot], (K / kRwItems) & 1u, &S.abort_flag)) break;
        const RowItem it = S.item[slot];
        mbar_arrive(&S.iempty[slot]);
        if (it.stop) break;
        const LaneView v = lane_view(it, L, tpt, kCausal);
        if (!row_wait(&S.qfull[L], K & 1u, &S.abort_flag)) break;
        if (v.used == 0) mbar_arrive(&S.qempty[L]);
        int i = 0;  // tiles used of this item
        for (int j = 0; j < it.ntile; ++j, ++T) {
          const uint32_t ck = 2 * T, cv = 2 * T + 1;
          const int sk = ck % kStages, sv = cv % kStages;
          const bool use = i < v.used && j == v.first + i * v.step;
          if (!row_wait(&S.full[sk], (ck / kStages) & 1u, &S.abort_flag)) { ok = false; break; }
          if (use) {
            // S and P share their columns: the product that read the last P is done
            if (J > 0 && !row_wait(&S.pvdone[L], (J - 1) & 1u, &S.abort_flag)) { ok = false; break; }
            tc_fence_after();
            const uint64_t kd0 = smem_desc(smem_u32(S.kv[sk][0]), 16, 1024, kLayoutSW128);
#pragma unroll
            for (int kk = 0; kk < kD / 16; ++kk) {
              const uint64_t off = static_cast<uint64_t>((kk >> 2) * (kRwHalf >> 4) + (kk & 3) * 2);
              umma_bf16_ss(s_col, qd0 + off, kd0 + off, idesc_s, kk > 0 ? 1u : 0u);
            }
            umma_commit(&S.sfull[L]);
            umma_commit(&S.empty[sk]);
            if (i == v.used - 1) umma_commit(&S.qempty[L]);
          } else {
            mbar_arrive(&S.empty[sk]);
          }
          if (!row_wait(&S.full[sv], (cv / kStages) & 1u, &S.abort_flag)) { ok = false; break; }
          if (use) {
            if (i == 0 && !row_wait(&S.oempty[L], (K & 1u) ^ 1u, &S.abort_flag)) { ok = false; break; }
            if (!row_wait(&S.pfull[L], J & 1u, &S.abort_flag)) { ok = false; break; }
            tc_fence_after();
            // key steps of 16 up to the lane's last visible key
            const int steps = (min(128, min(it.k1, v.kend) - (it.tile0 + j) * 128) + 15) >> 4;
            const uint64_t vd0 = smem_desc(smem_u32(S.kv[sv][0]), kRwHalf, 1024, kLayoutSW128);
            if (steps == 8) {
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                umma_bf16_ts(o_col, s_col + 8 * kk, vd0 + static_cast<uint64_t>(kk * 128), idesc_o, (i > 0 || kk > 0) ? 1u : 0u);
            } else {
              for (int kk = 0; kk < steps; ++kk)
                umma_bf16_ts(o_col, s_col + 8 * kk, vd0 + static_cast<uint64_t>(kk * 128), idesc_o, (i > 0 || kk > 0) ? 1u : 0u);
            }
            umma_commit(&S.pvdone[L]);
            umma_commit(&S.empty[sv]);
            if (i == v.used - 1) umma_commit(&S.ofin[L]);
            ++i;
            ++J;
          } else {
            mbar_arrive(&S.empty[sv]);
          }
        }
        if (ok && v.used == 0) {
          if (!row_wait(&S.oempty[L], (K & 1u) ^ 1u, &S.abort_flag)) break;
          mbar_arrive(&S.ofin[L]);
        }
      }
      umma_commit(&S.drain[L]);
      (void)row_poll(&S.drain[L], 0);
    }
    __syncwarp();
  } else if (warp < kRwEpi) {
    // ======================= softmax of one lane, one row a thread =======================
    set_regs_more<176>();
    const int L = warp >> 2, quad = warp & 3;
    const int r = quad * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t s_col = tmem + lane_base + 128 * L, o_col = tmem + lane_base + kRwColO + kD * L;
    const int pos_in = (r * p.g_recip16) >> 16;  // r / G
    const uint64_t scale2 = pair_f32(p.scale_log2, p.scale_log2);
    uint32_t T = 0, J = 0;
    bool ok = true;
    for (uint32_t K = 0; ok; ++K) {
      const int slot = K & (kRwItems - 1);
      if (!row_wait(&S.ifull[slot], (K / kRwItems) & 1u, &S.abort_flag)) break;
      const RowItem& it = S.item[slot];  // stays in shared memory: the scores need the registers
      if (it.stop) break;
      const LaneView v = lane_view(it, L, tpt, kCausal);
      const int pos = pos_in + (it.alt ? 0 : L * tpt);  // token of the item
      const bool row_ok = pos_in < v.nt;
      float m = -INFINITY;
      uint64_t sum2[4];
#pragma unroll
      for (int a = 0; a < 4; ++a) sum2[a] = 0;
      for (int i = 0; i < v.used; ++i, ++J) {
        const int j = v.first + i * v.step, tile = it.tile0 + j;
        uint32_t w[4];
        // tiles that every row of this warp sees whole need no mask
        bool full;
        if constexpr (kCausal) full = __all_sync(0xffffffffu, !row_ok || it.t0 + pos + 1 >= tile * 128 + 128);
        else full = tile * 128 + 128 <= it.prefix;
        if (!full) visible_words<kCausal>(p, it, tile, pos, row_ok, static_cast<int64_t>(it.row0) + pos, w);
        if (!row_wait(&S.sfull[L], J & 1u, &S.abort_flag)) { ok = false; break; }
        tc_fence_after();
        uint32_t x[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_col + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(x + 32 * c));
        tmem_wait_ld();
        if (!full) {
#pragma unroll
          for (int e = 0; e < 128; ++e) x[e] = (w[e >> 5] >> (e & 31)) & 1u ? x[e] : 0xff800000u;
        }
        float mx[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) mx[a] = fmaxf(__uint_as_float(x[2 * a]), __uint_as_float(x[2 * a + 1]));
#pragma unroll
        for (int e = 8; e < 128; e += 8)
#pragma unroll
          for (int a = 0; a < 4; ++a)
            mx[a] = max3_f32(mx[a], __uint_as_float(x[e + 2 * a]), __uint_as_float(x[e + 2 * a + 1]));
        const float mn = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2);
        const bool move = mn > m + kRwRescale || (m == -INFINITY && mn != -INFINITY);
        if (i > 0 && __any_sync(0xffffffffu, move)) {
          // the scores of this tile were issued after the last product into O had completed
          const float alpha = move ? (m == -INFINITY ? 0.f : fast_exp2(m - mn)) : 1.f;
#pragma unroll 1
          for (int c = 0; c < kD; c += 16) {
            uint32_t o[16];
            tmem_ld16(o_col + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st16(o_col + c, o);
          }
          const uint64_t alpha2 = pair_f32(alpha, alpha);
#pragma unroll
          for (int a = 0; a < 4; ++a) sum2[a] = fma_f32x2(sum2[a], alpha2, 0ull);
        }
        if (move) m = mn;
        const float negm = m == -INFINITY ? 0.f : -m;  // then every score is -inf
        const uint64_t negm2 = pair_f32(negm, negm);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t out[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float a0, a1;
            unpair_f32(fma_f32x2(pair_f32(__uint_as_float(x[32 * c + e]), __uint_as_float(x[32 * c + e + 1])), scale2, negm2), a0, a1);
            a0 = fast_exp2(a0);
            a1 = fast_exp2(a1);
            out[e >> 1] = pack_bf16(a0, a1);
            sum2[(e >> 1) & 3] = add_f32x2(sum2[(e >> 1) & 3], pair_f32(a0, a1));
          }
          tmem_st16(s_col + 16 * c, out);
        }
        const int valid = it.k1 - tile * 128;
        if (valid < 128 && (valid & 15) != 0) {
          // zero V rows [valid, next multiple of 16): they may lie behind the request's keys
          const uint32_t cv = 2 * (T + j) + 1;
          if (!row_wait(&S.full[cv % kStages], (cv / kStages) & 1u, &S.abort_flag)) { ok = false; break; }
          const int r0 = valid, nr = ((valid + 15) & ~15) - r0;
          for (int c = r; c < nr * 8 * kHalves; c += 128) {
            const int row = r0 + c / (8 * kHalves);
            *reinterpret_cast<uint4*>(reinterpret_cast<unsigned char*>(S.kv[cv % kStages][(c / 8) % kHalves]) + row * 128 +
                                      (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.pfull[L]);
      }
      if (!ok) break;
      T += it.ntile;
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.iempty[slot]);
      float s[8];
#pragma unroll
      for (int a = 0; a < 4; ++a) unpair_f32(sum2[a], s[2 * a], s[2 * a + 1]);
      const uint32_t ob = K & 1;
      if (!row_wait(&S.lfree[ob][L], ((K >> 1) & 1u) ^ 1u, &S.abort_flag)) break;
      S.mfin[ob][L][r] = m;
      S.lfin[ob][L][r] = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.lready[ob][L]);
    }
  } else {
    // ======================= epilogue: outputs, or the pieces of cut items =======================
    set_regs_less<88>();
    const int quad = warp & 3, r = quad * 32 + lane;
    const uint32_t o_base = tmem + (static_cast<uint32_t>(quad * 32) << 16) + kRwColO;
    const int pos_in = (r * p.g_recip16) >> 16, head_in = r - pos_in * p.g;
    // pieces: O as [slot][lane][D / 4][128 rows] float4, (m, l) as [slot][lane][128] float2
    float4* part_o = reinterpret_cast<float4*>(p.part_o);
    float2* part_ml = reinterpret_cast<float2*>(p.part_ml);
    bool ok = true;
    for (uint32_t K = 0; ok; ++K) {
      const int slot = K & (kRwItems - 1);
      if (!row_wait(&S.ifull[slot], (K / kRwItems) & 1u, &S.abort_flag)) break;
      const RowItem& it = S.item[slot];
      if (it.stop) break;
      const uint32_t ob = K & 1;
      const int tiles = it.alt ? 1 : 2;  // row tiles
      // one row of the output (32 columns at a time) and its log-sum-exp
      auto store = [&](int t, int c, const float (&o)[32], float inv) {
        const int pos = pos_in + t * tpt;
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + (static_cast<int64_t>(it.row0) + pos) * p.o_sr +
                             static_cast<int64_t>(it.h * p.g + head_in) * p.o_sh + c;
#pragma unroll
        for (int e = 0; e < 32; e += 8)
          *reinterpret_cast<uint4*>(dst + e) = make_uint4(pack_bf16(o[e] * inv, o[e + 1] * inv), pack_bf16(o[e + 2] * inv, o[e + 3] * inv),
                                                          pack_bf16(o[e + 4] * inv, o[e + 5] * inv), pack_bf16(o[e + 6] * inv, o[e + 7] * inv));
      };
      auto store_lse = [&](int t, float m, float l) {
        p.lse[(static_cast<int64_t>(it.row0) + pos_in + t * tpt) * p.hq + it.h * p.g + head_in] =
            l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
      };
      for (int t = 0; t < tiles; ++t) {
        const bool row_ok = pos_in < min(tpt, it.nt - t * tpt);
        float m, l, f0 = 1.f, f1 = 0.f;  // O = f0 O_first + f1 O_second
        for (int L = t; L < (it.alt ? 2 : t + 1); ++L) {
          if (!row_wait(&S.lready[ob][L], (K >> 1) & 1u, &S.abort_flag)) { ok = false; break; }
          const float ml = S.mfin[ob][L][r], ll = S.lfin[ob][L][r];
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.lfree[ob][L]);
          if (L == t) {
            m = ml;
            l = ll;
          } else {  // the other lane's key tiles of the same rows
            const float mn = fmaxf(m, ml);
            f0 = l > 0.f ? fast_exp2(m - mn) : 0.f;
            f1 = ll > 0.f ? fast_exp2(ml - mn) : 0.f;
            l = l * f0 + ll * f1;
            m = mn;
          }
          if (!row_wait(&S.ofin[L], K & 1u, &S.abort_flag)) { ok = false; break; }
        }
        if (!ok) break;
        tc_fence_after();
        const bool seen0 = !(l <= 0.f) && f0 != 0.f, seen1 = f1 != 0.f;
        const int part = 2 * static_cast<int>(blockIdx.x) + (it.piece > 0 ? 0 : 1);
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll 1
        for (int c = 0; c < kD; c += 32) {
          float o[32];
          {
            uint32_t raw[32];
            tmem_ld32(o_base + kD * t + c, raw);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = seen0 ? __uint_as_float(raw[e]) * f0 : 0.f;
            if (it.alt) {
              tmem_ld32(o_base + kD + c, raw);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = seen1 ? fmaf(__uint_as_float(raw[e]), f1, o[e]) : o[e];
            }
          }
          if (it.cuts == 0) {
            if (row_ok) store(t, c, o, inv);
          } else {
            float4* dst = part_o + ((static_cast<int64_t>(part) * 2 + t) * (kD / 4) + c / 4) * 128 + r;
#pragma unroll
            for (int e = 0; e < 8; ++e) dst[e * 128] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
        if (it.cuts == 0) {
          if (row_ok) store_lse(t, m, l);
        } else {
          part_ml[(static_cast<int64_t>(part) * 2 + t) * 128 + r] = make_float2(m, l);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&S.oempty[t]);
          if (it.alt) mbar_arrive(&S.oempty[1]);
        }
      }
      if (!ok) break;
      if (it.cuts > 0) {
        // The quad's rows of this piece are written; the warp that counts the last piece adds them all.
        __threadfence();
        __syncwarp();
        uint32_t before = 0;
        uint32_t* counter = &p.hdr->row_pieces[it.cut0];
        if (lane == 0) before = (atomicAdd(counter, 1u << (8 * quad)) >> (8 * quad)) & 0xffu;
        before = __shfl_sync(0xffffffffu, before, 0);
        if (before == static_cast<uint32_t>(it.cuts)) {
          __threadfence();
          if (lane == 0) atomicSub(counter, static_cast<uint32_t>(it.cuts + 1) << (8 * quad));
          auto piece_slot = [&](int q) { return 2 * (it.cut0 - 1 + q) + (q > 0 ? 0 : 1); };
          for (int t = 0; t < tiles; ++t) {
            const bool row_ok = pos_in < min(tpt, it.nt - t * tpt);
            float m = -INFINITY, l = 0.f;
            for (int q = 0; q <= it.cuts; ++q) {
              const float2 ml = __ldcg(part_ml + (static_cast<int64_t>(piece_slot(q)) * 2 + t) * 128 + r);
              if (!(ml.y == 0.f)) m = fmaxf(m, ml.x);
            }
            for (int q = 0; q <= it.cuts; ++q) {
              const float2 ml = __ldcg(part_ml + (static_cast<int64_t>(piece_slot(q)) * 2 + t) * 128 + r);
              if (!(ml.y == 0.f)) l = fmaf(ml.y, fast_exp2(ml.x - m), l);
            }
            const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll 1
            for (int c = 0; c < kD; c += 32) {
              float o[32];
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = 0.f;
#pragma unroll 1
              for (int q = 0; q <= it.cuts; ++q) {
                const int64_t at = static_cast<int64_t>(piece_slot(q)) * 2 + t;
                const float2 ml = __ldcg(part_ml + at * 128 + r);
                const float f = ml.y == 0.f ? 0.f : fast_exp2(ml.x - m);
                const float4* src = part_o + (at * (kD / 4) + c / 4) * 128 + r;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const float4 y = __ldcg(src + e * 128);
                  o[4 * e] = fmaf(f, y.x, o[4 * e]);
                  o[4 * e + 1] = fmaf(f, y.y, o[4 * e + 1]);
                  o[4 * e + 2] = fmaf(f, y.z, o[4 * e + 2]);
                  o[4 * e + 3] = fmaf(f, y.w, o[4 * e + 3]);
                }
              }
              if (row_ok) store(t, c, o, inv);
            }
            if (row_ok) store_lse(t, m, l);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.iempty[slot]);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && S.abort_flag) atomicOr(&p.hdr->status, FD_FLAG_WAIT_TIMEOUT);
  if (warp == kRwIssue) tmem_dealloc(tmem, kRwTmemCols);
}

template <int kD, int kSrc>
cudaError_t launch_rows_t(const RowsParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                          int nctas, cudaStream_t stream) {
  const size_t smem = sizeof(RwSmem<kD>) + 1024;
  cudaError_t e = cudaFuncSetAttribute(rows_tc_kernel<kD, kSrc>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(nctas);
  cfg.blockDim = dim3(kRwThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rows_tc_kernel<kD, kSrc>, p, tq, tk, tv);
}

}  // namespace

size_t rows_workspace_bytes(int d, int nctas) {
  return sizeof(WsHeader) + static_cast<size_t>(2 * nctas) * 2 * 128 * (d * sizeof(float) + sizeof(float2));
}

cudaError_t launch_rows(RowsParams p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, int nctas,
                        cudaStream_t stream) {
  char* base = reinterpret_cast<char*>(p.hdr);
  p.part_o = reinterpret_cast<float*>(base + sizeof(WsHeader));
  p.part_ml = p.part_o + static_cast<int64_t>(2 * nctas) * 2 * 128 * p.d;
  const int src = p.prefix_lens == nullptr ? kSrcPacked : p.block_table ? kSrcPaged : kSrcCache;
  if (p.d == 128) {
    if (src == kSrcPacked) return launch_rows_t<128, kSrcPacked>(p, tq, tk, tv, nctas, stream);
    if (src == kSrcCache) return launch_rows_t<128, kSrcCache>(p, tq, tk, tv, nctas, stream);
    return launch_rows_t<128, kSrcPaged>(p, tq, tk, tv, nctas, stream);
  }
  if (src == kSrcPacked) return launch_rows_t<64, kSrcPacked>(p, tq, tk, tv, nctas, stream);
  if (src == kSrcCache) return launch_rows_t<64, kSrcCache>(p, tq, tk, tv, nctas, stream);
  return launch_rows_t<64, kSrcPaged>(p, tq, tk, tv, nctas, stream);
}

}  // namespace fd
