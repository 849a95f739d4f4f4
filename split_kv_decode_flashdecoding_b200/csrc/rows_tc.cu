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
// small tree's softmax still runs on eight warps. Where few items or short requests are known to be all
// (rows_two_tiles), the call has one-tile items only.
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
// Warps: 0-3 and 4-7 softmax and output of lanes 0 and 1 (warp w reads TMEM lanes 32 (w mod 4) + [0, 32),
// one row a thread); 8 plan and TMA of Q and K; 9 tensor-core issue; 10 TMA of V.
#include <type_traits>

#include "common.cuh"
#include "pairs.cuh"
#include "rows.h"
#include "rows_plan.h"

namespace fd {

namespace {

constexpr int kRwThreads = 12 * 32;
constexpr int kRwProducer = 8, kRwIssue = 9, kRwVProducer = 10;
constexpr int kRwItems = 4;                    // item descriptors in flight
constexpr uint32_t kRwTmemCols = 512;
constexpr uint32_t kRwColO = 256;              // O of lane L at kRwColO + L D; S, then P, of lane L at 128 L
constexpr uint32_t kRwHalf = 128 * 64 * 2;     // bytes of one 64-column half of a 128-row tile
constexpr float kRwRescale = 8.0f;             // log2 units
constexpr uint32_t kRwWaitClocks = 0x80000000u;

enum RowSource { kSrcPacked = 0, kSrcCache = 1, kSrcPaged = 2 };

struct RowItem {
  int32_t stop;
  int32_t b, h;             // request, KV head
  int32_t row0, t0;         // packed row of the first token; its index in the request
  int32_t key_row0;         // prompt: packed row of the request's first key
  int32_t tile0, ntile;     // key tiles [tile0, tile0 + ntile)
  int32_t k1;               // keys of the item (all pieces): tiles hold keys < k1
  int32_t prefix;           // tree: keys every row sees
  int32_t alt;              // one row tile, the lanes take alternate key tiles
  // by lane: its tokens, the key tiles it uses, the end of its visible keys from tile0's first key on.
  // The i-th tile of lane L is tile0 + i, or tile0 + 2 i + L (alt).
  int32_t tokens[2], used[2], kend[2];
  int32_t whole;              // this CTA has all its key tiles; if not, when cfull has arrived:
  int32_t cut0, cuts;         // rows_cuts of the item
};

// kPairs: items of two row tiles. Of one tile, its Q serves both lanes, and V has a stage more for it: a V
// stage is held through the tile's softmax.
template <int kD, bool kPairs>
struct __align__(1024) RwSmem {
  static constexpr int kHalves = kD / 64;
  static constexpr int kKStages = kD == 128 ? 2 : 4;
  static constexpr int kVStages = kPairs ? kKStages : kD == 128 ? 3 : 6;
  static constexpr int kQ = kPairs ? 2 : 1;
  __nv_bfloat16 q[kQ][kHalves][128 * 64];
  __nv_bfloat16 k[kKStages][kHalves][128 * 64];
  __nv_bfloat16 v[kVStages][kHalves][128 * 64];
  RowItem item[kRwItems];
  int32_t req[kRwThreads][3];  // a thread's first request: rows, keys, prefix
  float2 xend[2][8][32];  // softmax warps: a row's (m, l) at the end of an alt item, for the other lane's warp
  union {
    struct {  // plan: work and rows of a thread's requests; work, rows and items of a warp's
      int64_t part_w[kRwThreads], warp_w[kRwThreads / 32];
      int32_t part_r[kRwThreads], warp_r[kRwThreads / 32], warp_i[kRwThreads / 32];
    };
    uint4 stage[8][128];  // output: a warp's rows, 32 columns
  };
  uint64_t kfull[kKStages], kempty[kKStages], vfull[kVStages], vempty[kVStages];
  uint64_t qfull[2], qempty[2], ifull[kRwItems], cfull[kRwItems], iempty[kRwItems];
  // by lane: a tile's scores are there, P of keys [0, 64) and of [64, 128) is stored, O is complete, is read
  uint64_t sfull[2], pfull[2][2], ofin[2], oempty[2];
  uint64_t xpair[4];  // exchanges of the two lanes' warps of a row quarter (alt items)
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  int bad;
};
static_assert(sizeof(RwSmem<128, true>) + 1024 <= 227 * 1024, "row attention shared memory");
static_assert(sizeof(RwSmem<128, false>) + 1024 <= 227 * 1024, "row attention shared memory");
static_assert(sizeof(RwSmem<64, true>) + 1024 <= 227 * 1024, "row attention shared memory");
static_assert(sizeof(RwSmem<64, false>) + 1024 <= 227 * 1024, "row attention shared memory");

// Maximum that a NaN wins, so that a row which sees one becomes NaN as a whole.
__device__ __forceinline__ float max3_f32(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
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

// The bounded waits of common.cuh with a short polling loop in line: a kernel that re-divides its
// registers between warps (setmaxnreg) cannot call a function. The limit counts clocks (2^31 are
// 1.1 s at 1965 MHz); the status word is raised once, at the kernel's end.
__device__ __forceinline__ bool row_poll(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint32_t t0 = static_cast<uint32_t>(clock());
#pragma unroll 1
  do {
    if (mbar_try_wait(bar, parity)) return true;
  } while (static_cast<uint32_t>(clock()) - t0 < kRwWaitClocks);
  return false;
}
__device__ __forceinline__ bool row_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (row_poll(bar, parity)) return true;
  *abort_flag = 1;
  return false;
}

// True in one lane of a converged warp. Products and commits stand under this, inside code that the
// whole warp runs, so that their descriptors stay in uniform registers: behind `lane == 0` every
// product took ~85 cycles to issue, with the tensor pipe needing 64.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// row_wait by a whole warp, with one answer.
__device__ __forceinline__ bool row_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, row_wait(bar, parity, abort_flag));
}
// Sum over a warp; running sums of its lanes.
__device__ __forceinline__ int64_t warp_sum(int64_t x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ void warp_scan(int64_t& x, int64_t& y, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, x, o), b = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) { x += a; y += b; }
  }
}
__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}

// Counts this warp's stores (after a __syncwarp) as there, and makes those counted before visible to a warp
// that passes its next __syncwarp.
__device__ __forceinline__ uint32_t atomic_add_acq_rel(uint32_t* at, uint32_t n) {
  uint32_t r;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(r) : "l"(at), "r"(n) : "memory");
  return r;
}

// n low bits set (n <= 0: none, n >= 32: all).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
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

// 1 / l; 0 for an empty row; NaN stays.
__device__ __forceinline__ float row_over(float l) { return l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l); }

// Where a thread stores: 16 bytes of rows lane / 4 + 8 i of its warp's (null: behind the last token). Found
// before O is complete.
__device__ __forceinline__ void row_places(const RowsParams& p, const RowItem& it, int quad, int lane, int t, int tpt, char* (&dst)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int rr = quad * 32 + (lane >> 2) + 8 * i, pos = (rr * p.g_recip16) >> 16;
    dst[i] = pos < it.tokens[t] ? static_cast<char*>(p.out) + 2 * ((static_cast<int64_t>(it.row0) + pos + t * tpt) * p.o_sr +
                                                                   static_cast<int64_t>(it.h * p.g + rr - pos * p.g) * p.o_sh) +
                                      16 * (lane & 3)
                                : nullptr;
  }
}

// The end of an item for one softmax warp: columns [c0, c1) of its 32 rows of row tile t, the
// accumulator at o_col (an alt item: both lanes', times f0 and f1) over l, to memory; or, for a piece of
// a cut item, unscaled to the workspace, where the warp that counts the last piece adds them all in
// piece order. Rows leave through shared memory, 32 columns at a time, so that neighbouring threads
// store neighbouring bytes: a thread storing its own row kept the load/store pipe, and with it every
// warp's barrier and tensor-memory traffic, busy for ~3000 cycles an item. The loops stay rolled: this
// code runs once an item, from a cold instruction cache.
template <int kD, bool kAlt, typename Smem>
__device__ __forceinline__ void row_output(const RowsParams& p, Smem& S, const RowItem& it, int warp, int lane, int t,
                                           int c0, int c1, uint32_t o_col, int tpt, char* const (&dst)[4], float m, float l,
                                           float scale, float f0, float f1) {
  const int quad = warp & 3;
  uint4* stage = S.stage[warp];
  auto emit = [&](int c, const uint64_t (&o)[16]) {
    uint32_t w[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float lo, hi;
      unpair_f32(o[e], lo, hi);
      w[e] = pack_bf16(lo, hi);
    }
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 4; ++e) stage[lane * 4 + (e ^ ((lane >> 1) & 3))] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = (lane >> 2) + 8 * i;
      const uint4 v = stage[row * 4 + ((lane & 3) ^ ((row >> 1) & 3))];
      if (dst[i]) *reinterpret_cast<uint4*>(dst[i] + 2 * c) = v;
    }
  };
  auto store_lse = [&](float m, float l) {
    const int r = quad * 32 + lane, pos = (r * p.g_recip16) >> 16;
    if (c0 == 0 && pos < it.tokens[t])
      p.lse[(static_cast<int64_t>(it.row0) + pos + t * tpt) * p.hq + it.h * p.g + r - pos * p.g] =
          l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  };
  const bool live = (((quad * 32 + lane) * p.g_recip16) >> 16) < it.tokens[t];  // this thread's row
  // pieces: O as [slot][row tile][D / 4][128 rows] float4, (m, l) as [slot][warp][32 rows] float2
  ulonglong2* part_o = reinterpret_cast<ulonglong2*>(p.part_o) + quad * 32 + lane;
  float2* part_ml = reinterpret_cast<float2*>(p.part_ml) + warp * 32 + lane;
  auto place = [&](int64_t slot, int c) { return ((slot * 2 + t) * (kD / 4) + c / 4) * 128; };
  const int64_t part = 2 * static_cast<int64_t>(blockIdx.x) + (it.tile0 > 0 ? 0 : 1);  // the first piece: 1
  const bool whole = it.whole != 0;
  // A lane without tiles has left its accumulator as it was: that one is not looked at.
  const bool none0 = it.used[kAlt ? 0 : t] == 0, none1 = it.used[1] == 0;
  const uint64_t s02 = pair_f32(scale * f0, scale * f0), s12 = pair_f32(scale * f1, scale * f1);
#pragma unroll 1
  for (int c = c0; c < c1; c += 32) {
    uint64_t o[16];
    uint32_t raw[32], raw1[32];
    tmem_ld32(o_col + c, raw);
    if (kAlt) tmem_ld32(o_col + kD + c, raw1);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; ++e)
      o[e] = none0 ? 0ull : fma_f32x2(pair_f32(__uint_as_float(raw[2 * e]), __uint_as_float(raw[2 * e + 1])), s02, 0ull);
    if (kAlt && !none1) {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        o[e] = fma_f32x2(pair_f32(__uint_as_float(raw1[2 * e]), __uint_as_float(raw1[2 * e + 1])), s12, o[e]);
    }
    if (c + 32 >= c1) {  // the accumulator is read: the next item's first product may start
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_n(&S.oempty[t], kAlt ? 1u : 2u);
        if (kAlt) mbar_arrive_n(&S.oempty[1], 1u);
      }
    }
    if (whole) {
      emit(c, o);
    } else if (live) {
#pragma unroll
      for (int e = 0; e < 8; ++e) part_o[place(part, c) + e * 128] = make_ulonglong2(o[2 * e], o[2 * e + 1]);
    }
  }
  if (whole) {
    store_lse(m, l);
    return;
  }
  part_ml[part * 256] = make_float2(m, l);
  __syncwarp();
  uint32_t* counter = &p.front->row_pieces[it.cut0][warp >> 2];
  uint32_t before = 0;
  if (lane == 0) before = (atomic_add_acq_rel(counter, 1u << (8 * quad)) >> (8 * quad)) & 0xffu;
  before = __shfl_sync(0xffffffffu, before, 0);
  __syncwarp();
  const int cuts = it.cuts, cut0 = it.cut0;
  if (before != static_cast<uint32_t>(cuts)) return;
  if (lane == 0) atomicSub(counter, static_cast<uint32_t>(cuts + 1) << (8 * quad));
  // Four pieces' loads at a time: a load takes ~1000 cycles, and with two in flight the merge of a wide
  // tree's pieces took 30,000.
  auto piece_slot = [&](int q) { return 2 * static_cast<int64_t>(cut0 - 1 + q) + (q > 0 ? 0 : 1); };
  float mt = -INFINITY, lt = 0.f;
#pragma unroll 1
  for (int q = 0; q <= cuts; q += 4) {
    float2 ml[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) ml[i] = q + i <= cuts ? __ldcg(part_ml + piece_slot(q + i) * 256) : make_float2(-INFINITY, 0.f);
    float mn = mt;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!(ml[i].y == 0.f)) mn = fmaxf(mn, ml[i].x);
    lt = lt == 0.f ? 0.f : lt * fast_exp2(mt - mn);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!(ml[i].y == 0.f)) lt = fmaf(ml[i].y, fast_exp2(ml[i].x - mn), lt);
    mt = mn;
  }
  const float total = row_over(lt);
#pragma unroll 1
  for (int c = c0; c < c1; c += 32) {
    uint64_t o[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = 0;
#pragma unroll 1
    for (int q = 0; q <= cuts; q += 4) {
      float2 ml[4];
      ulonglong2 y[4][8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool there = live && q + i <= cuts;
        const int64_t slot = piece_slot(q + i);
        ml[i] = there ? __ldcg(part_ml + slot * 256) : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[i][e] = there ? __ldcg(part_o + place(slot, c) + e * 128) : make_ulonglong2(0ull, 0ull);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float f = ml[i].y == 0.f ? 0.f : fast_exp2(ml[i].x - mt) * total;
        const uint64_t f2 = pair_f32(f, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          o[2 * e] = fma_f32x2(y[i][e].x, f2, o[2 * e]);
          o[2 * e + 1] = fma_f32x2(y[i][e].y, f2, o[2 * e + 1]);
        }
      }
    }
    emit(c, o);
  }
  store_lse(mt, lt);
}

// The copies of a tile of K or V into one stage, one box a lane: the box's page and 64-column half
// (paged), or its half.
template <int kD, int kSrc>
struct KeyBoxes {
  static constexpr int kHalves = kD / 64, kKeys = 128;
  int psz, boxes, box_page, box_half, lane, h, b, row0, k1;
  __device__ __forceinline__ KeyBoxes(const RowsParams& p, const RowItem& it, int lane_) {
    lane = lane_;
    psz = kSrc == kSrcPaged ? min(p.page_size, kKeys) : kKeys;
    boxes = (kKeys / psz) * kHalves;
    box_page = lane / kHalves;
    box_half = lane % kHalves;
    h = it.h;
    b = it.b;
    row0 = it.key_row0;
    k1 = it.k1;
  }
  // the page of this lane's box in piece `n` (keys [n kKeys, (n + 1) kKeys)) of the request
  __device__ __forceinline__ int page(const RowsParams& p, int n) const {
    if constexpr (kSrc == kSrcPaged) {
      const int key = n * kKeys + box_page * psz;
      if (lane < boxes && key < k1) {
        const int id = p.block_table[static_cast<int64_t>(b) * p.pages_per_seq + key / p.page_size];
        if (id >= 0 && id < p.num_pages) return id;
        atomicOr(&p.hdr->status, FD_FLAG_BAD_PAGE);
      }
      return p.num_pages;  // outside the map: the copy writes zeros
    }
    return 0;
  }
  __device__ __forceinline__ void load(const RowsParams& p, const CUtensorMap* map, uint64_t* full, __nv_bfloat16* stage,
                                       int n, int page) const {
    if (lane == 0) mbar_arrive_expect_tx(full, kHalves * 128u * static_cast<uint32_t>(p.kv_box_rows * (kKeys / psz)));
    __syncwarp();
    if (lane < boxes) {
      __nv_bfloat16* dst = stage + box_half * kKeys * 64 + box_page * psz * 64;
      if constexpr (kSrc == kSrcPacked) tma_load_3d(dst, map, full, 64 * box_half, h, row0 + n * kKeys);
      else if constexpr (kSrc == kSrcCache) tma_load_4d(dst, map, full, 64 * box_half, n * kKeys, h, b);
      else tma_load_4d(dst, map, full, 64 * box_half, n * kKeys % p.page_size, h, page);
    }
  }
};

template <int kD, int kSrc, bool kPairs>
__global__ void __launch_bounds__(kRwThreads, 1)
    rows_tc_kernel(const RowsParams p, const __grid_constant__ CUtensorMap tmap_q,
                   const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v) {
  using Smem = RwSmem<kD, kPairs>;
  constexpr bool kCausal = kSrc == kSrcPacked;
  constexpr int kHalves = Smem::kHalves, kKStages = Smem::kKStages, kVStages = Smem::kVStages;
  constexpr int kQ = Smem::kQ;  // row tiles of an item
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  Smem& S = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // the same in all lanes, and known to be
  const int tpt = rows_tile_tokens(p.g), span = kQ * tpt;

  if (tid == 0) {
    for (int s = 0; s < Smem::kKStages; ++s) {
      mbar_init(&S.kfull[s], 1);
      mbar_init(&S.kempty[s], 2);  // both lanes' products
    }
    for (int s = 0; s < Smem::kVStages; ++s) {
      mbar_init(&S.vfull[s], 1);
      mbar_init(&S.vempty[s], 2);
    }
    for (int i = 0; i < kRwItems; ++i) {
      mbar_init(&S.ifull[i], 1);
      mbar_init(&S.cfull[i], 1);
      mbar_init(&S.iempty[i], 8 + 1 + 1);  // softmax warps, the issuer, the V producer
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.qfull[i], 1);
      mbar_init(&S.qempty[i], 1);
      mbar_init(&S.sfull[i], 1);
      mbar_init(&S.pfull[i][0], 4);
      mbar_init(&S.pfull[i][1], 4);
      mbar_init(&S.ofin[i], 1);
      mbar_init(&S.oempty[i], 8);
    }
    for (int q = 0; q < 4; ++q) mbar_init(&S.xpair[q], 2);
    mbar_init(&S.drain, 1);
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
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;
  pdl_launch_dependents();
  pdl_wait_prerequisites();

  // The requests' work. Up to 32 requests are the lanes of the planning warp; of more, thread t sums those
  // of its stretch of the batch. (The second way alone, whose sums and barriers are latency: short prompts
  // 12.97 instead of 12.61 us, 8 wide trees 61.2 instead of 55.8.)
  const bool one_warp = p.batch <= 32;
  const int per = (p.batch + kRwThreads - 1) / kRwThreads;
  auto request = [&](int b, int* n, int* keys, int* prefix) {
    const int len = p.row_lens[b];
    const int pre = kCausal ? 0 : p.prefix_lens[b];
    *n = max(len, 0);
    *keys = *n;
    *prefix = 0;
    uint32_t flag = len < 0 ? FD_FLAG_LEN_CLAMPED : 0u;
    if constexpr (!kCausal) {
      if (len < 0 || len > 32 * p.mask_words) S.bad = 1;
      *prefix = clamp_len(pre, p.cap);
      const int64_t end = static_cast<int64_t>(*prefix) + *n;
      *keys = static_cast<int>(min(end, static_cast<int64_t>(p.cap)));
      if (*prefix != pre || *keys != end) flag = FD_FLAG_LEN_CLAMPED;
    }
    return flag;
  };
  if (!one_warp) {
    int64_t w = 0, rows = 0;
    int items = 0;
    uint32_t flag = 0;
    for (int i = 0; i < per; ++i) {
      const int b = tid * per + i;
      if (b >= p.batch) break;
      int n, keys, prefix;
      flag |= request(b, &n, &keys, &prefix);
      const int parts = rows_items(n, span);
      w += p.hkv * rows_weight(kCausal, span, keys, parts);
      rows += n;
      items += parts;
      if (i == 0) {
        S.req[tid][0] = n;
        S.req[tid][1] = keys;
        S.req[tid][2] = prefix;
      }
    }
    if (flag && blockIdx.x == 0) atomicOr(&p.hdr->status, flag);
    const int32_t r = static_cast<int32_t>(min(rows, static_cast<int64_t>(p.rows) + 1));
    S.part_w[tid] = w;
    S.part_r[tid] = r;
    if (warp * 32 * per < p.batch) {
      const int64_t warp_w = warp_sum(w), warp_r = warp_sum(static_cast<int64_t>(r));
      const int32_t warp_i = __reduce_add_sync(0xffffffffu, items);
      if (warp_r > p.rows) S.bad = 1;
      if (lane == 0) {
        S.warp_w[warp] = warp_w;
        S.warp_r[warp] = static_cast<int32_t>(min(warp_r, static_cast<int64_t>(p.rows)));
        S.warp_i[warp] = warp_i;
      }
    } else if (lane == 0) {
      S.warp_w[warp] = 0;
      S.warp_r[warp] = S.warp_i[warp] = 0;
    }
    __syncthreads();
  }

  if (warp >= kRwProducer) {
    set_regs_less<88>();
    if (warp == kRwProducer) {
      // ======================= plan and TMA =======================
      // Running sums of work and rows, over the requests (one_warp) or over the warps' stretches; the totals.
      int64_t own_w, own_r, items;
      if (one_warp) {
        int n = 0, keys = 0, prefix = 0;
        if (lane < p.batch) {
          const uint32_t flag = request(lane, &n, &keys, &prefix);
          if (flag && blockIdx.x == 0) atomicOr(&p.hdr->status, flag);
        }
        const int parts = rows_items(n, span);
        own_w = p.hkv * rows_weight(kCausal, span, keys, parts);
        own_r = n;
        items = __reduce_add_sync(0xffffffffu, parts);
        S.req[lane][0] = n;
        S.req[lane][1] = keys;
        S.req[lane][2] = prefix;
        __syncwarp();
      } else {
        constexpr int kWarps = kRwThreads / 32;
        own_w = lane < kWarps ? S.warp_w[lane] : 0;
        own_r = lane < kWarps ? S.warp_r[lane] : 0;
        items = warp_sum(static_cast<int64_t>(lane < kWarps ? S.warp_i[lane] : 0));
      }
      int64_t sum_w = own_w, sum_r = own_r;
      warp_scan(sum_w, sum_r, lane);
      const int64_t weight = __shfl_sync(0xffffffffu, sum_w, 31), rows = __shfl_sync(0xffffffffu, sum_r, 31);
      bool ok = true;
      uint32_t T = 0, K = 0;  // key tiles and items so far
      const bool bad = S.bad != 0 || rows > p.rows;
      if (bad && blockIdx.x == 0 && lane == 0) atomicOr(&p.hdr->status, FD_FLAG_LEN_CLAMPED);
      const int nact = bad || weight == 0 ? 0 : rows_active(weight, items * p.hkv, static_cast<int>(gridDim.x));
      if (static_cast<int>(blockIdx.x) < nact) {
        const int cta = blockIdx.x;
        const RowsLine line = rows_line(weight, nact);
        const int64_t x0 = rows_bound(line, cta), x1 = rows_bound(line, cta + 1);
        // the request that x0 falls into: its warp, its thread's stretch, then one by one
        int t = 0;
        int64_t w0 = 0, r0 = 0;
        if (!one_warp) {
          const int src = __ffs(__ballot_sync(0xffffffffu, sum_w > x0)) - 1;  // the last lane's sum is weight > x0
          t = src * 32;
          w0 = __shfl_sync(0xffffffffu, sum_w - own_w, src);
          r0 = __shfl_sync(0xffffffffu, sum_r - own_r, src);
          sum_w = own_w = S.part_w[t + lane];
          sum_r = own_r = S.part_r[t + lane];
          warp_scan(sum_w, sum_r, lane);
        }
        const int src = __ffs(__ballot_sync(0xffffffffu, w0 + sum_w > x0)) - 1;
        t += src;
        int64_t base = w0 + __shfl_sync(0xffffffffu, sum_w - own_w, src), row = r0 + __shfl_sync(0xffffffffu, sum_r - own_r, src);
        int b = t * per, n = S.req[t][0], keys = S.req[t][1], prefix = S.req[t][2];
        int64_t all = p.hkv * rows_weight(kCausal, span, keys, rows_items(n, span));
        while (base + all <= x0) {
          base += all;
          row += n;
          request(++b, &n, &keys, &prefix);
          all = p.hkv * rows_weight(kCausal, span, keys, rows_items(n, span));
        }
        int parts = rows_items(n, span);
        int64_t per_head = rows_weight(kCausal, span, keys, parts);
        int h = static_cast<int>(rows_quotient(x0 - base, per_head));
        int64_t a = base + h * per_head;
        int u = 0;
        for (int hi = parts; hi - u > 1;) {  // the last u whose items before it end at or before x0
          const int mid = (u + hi) >> 1;
          if (a + rows_weight(kCausal, span, keys, mid) <= x0) u = mid; else hi = mid;
        }
        // The next piece of this CTA's stretch into the item ring (slot K), or the stop mark. The
        // consumers get it long before its tiles: planning takes this warp ~2500 cycles.
        bool more = true;
        int64_t cut_a = 0, cut_w = 0;  // the published item, its key tiles if it is cut
        int cut_tiles = 0;
        auto publish = [&](uint32_t K_) -> bool {
          const int slot = K_ & (kRwItems - 1);
          if (!row_wait(&S.iempty[slot], ((K_ / kRwItems) & 1u) ^ 1u, &S.abort_flag)) return false;
          RowItem& it = S.item[slot];
          bool found = false;
          while (more && !found) {
            const int64_t a0 = a + rows_weight(kCausal, span, keys, u);
            if (a0 >= x1) break;
            const int64_t w = a + rows_weight(kCausal, span, keys, u + 1) - a0;
            const int k1 = rows_item_keys(kCausal, span, n, keys, u);
            const int tiles = (k1 + 127) >> 7;
            const int c0 = rows_cut(x0, a0, w, tiles), c1 = rows_cut(x1, a0, w, tiles);
            if (c0 < c1) {
              found = true;
              cut_a = a0;
              cut_w = w;
              cut_tiles = c0 > 0 || c1 < tiles ? tiles : 0;
              const int t0 = u * span, nt = min(span, n - t0);
              const bool alt = !kPairs || nt <= tpt;
              if (lane == 0) {
                it.stop = 0;
                it.b = b;
                it.h = h;
                it.t0 = t0;
                it.row0 = static_cast<int>(row) + t0;
                it.key_row0 = static_cast<int>(row);
                it.tile0 = c0;
                it.ntile = c1 - c0;
                it.k1 = k1;
                it.prefix = prefix;
                it.alt = alt;
                it.whole = cut_tiles == 0;
              }
              if (lane < 2) {
                const int first = alt ? 0 : lane * tpt, tokens = alt ? nt : min(tpt, nt - first);
                const int kend = (kCausal ? t0 + first + tokens : k1) - c0 * 128;
                it.tokens[lane] = tokens;
                it.kend[lane] = kend;
                it.used[lane] = alt ? (c1 - c0 + 1 - lane) >> 1 : max(0, min(c1 - c0, (kend + 127) >> 7));
              }
            }
            if (++u == parts) {
              u = 0;
              a += per_head;
              if (++h == p.hkv) {
                h = 0;
                base += all;
                row += n;
                do {  // the next request with rows
                  if (++b >= p.batch) break;
                  if (per == 1) {
                    n = S.req[b][0];
                    keys = S.req[b][1];
                    prefix = S.req[b][2];
                  } else {
                    request(b, &n, &keys, &prefix);
                  }
                } while (n == 0);
                more = b < p.batch;
                if (more) {
                  parts = rows_items(n, span);
                  per_head = rows_weight(kCausal, span, keys, parts);
                  all = p.hkv * per_head;
                  a = base;
                }
              }
            }
          }
          if (!found && lane == 0) it.stop = 1;
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.ifull[slot]);
          return true;
        };
        // How the piece's item is cut: only its output asks, so the first loads come before
        auto publish_cuts = [&](uint32_t K_) {
          const int slot = K_ & (kRwItems - 1);
          if (cut_tiles > 0) {
            int cut0, cuts;
            rows_cuts(line, cut_a, cut_w, cut_tiles, cta, &cut0, &cuts);
            if (lane == 0) {
              RowItem& it = S.item[slot];
              it.cut0 = cut0;
              it.cuts = cuts;
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.cfull[slot]);
        };
        ok = publish(0);
        while (ok) {
          const RowItem& it = S.item[K & (kRwItems - 1)];
          if (it.stop) break;
          const int c0 = it.tile0, c1 = it.tile0 + it.ntile, ih = it.h;
          const int q_row = it.row0, q_step = it.alt ? 0 : tpt;
          const KeyBoxes<kD, kSrc> box(p, it, lane);
          int page = box.page(p, c0);
#pragma unroll 1
          for (int j = c0; j < c1; ++j, ++T) {
            const int st = T % kKStages;
            if (!row_wait(&S.kempty[st], ((T / kKStages) & 1u) ^ 1u, &S.abort_flag)) { ok = false; break; }
            box.load(p, &tmap_k, &S.kfull[st], S.k[st][0], j, page);
            if (j == c0) {
#pragma unroll 1
              for (int L = 0; L < kQ; ++L) {
                if (!row_wait(&S.qempty[L], (K & 1u) ^ 1u, &S.abort_flag) ||
                    (!kPairs && !row_wait(&S.qempty[1], (K & 1u) ^ 1u, &S.abort_flag))) { ok = false; break; }
                if (lane == 0) mbar_arrive_expect_tx(&S.qfull[L], kHalves * 128u * static_cast<uint32_t>(p.g * p.q_box_rows));
                __syncwarp();
                if (lane < kHalves) tma_load_3d(S.q[L][lane], &tmap_q, &S.qfull[L], 64 * lane, ih * p.g, q_row + L * q_step);
              }
              if (!ok) break;
              publish_cuts(K);
            }
            if (j + 1 < c1) page = box.page(p, j + 1);
            // the ring holds two tiles: plan while they are worked on
            if (j == min(c0 + 1, c1 - 1) && !(ok = publish(K + 1))) break;
          }
          if (ok) ++K;
        }
      } else {
        if (lane == 0) {
          S.item[0].stop = 1;
          mbar_arrive(&S.ifull[0]);
        }
      }
      __syncwarp();
      if (S.abort_flag && lane == 0) {  // copies still in flight land before the CTA leaves
        for (uint32_t back = 1; back <= kKStages && back <= T; ++back) (void)row_poll(&S.kfull[(T - back) % kKStages], ((T - back) / kKStages) & 1u);
        for (int L = 0; L < kQ; ++L) {
          if (K > 0) (void)row_poll(&S.qfull[L], (K - 1) & 1u);
          (void)row_poll(&S.qfull[L], K & 1u);
        }
      }
    } else if (warp == kRwVProducer) {
      // ======================= TMA of V =======================
      // A warp of its own: V's stages are held through the softmax, and K must not queue behind them.
      uint32_t T = 0;
      bool ok = true;
      for (uint32_t K = 0; ok; ++K) {
        const int slot = K & (kRwItems - 1);
        if (!row_wait(&S.ifull[slot], (K / kRwItems) & 1u, &S.abort_flag)) break;
        const RowItem& it = S.item[slot];
        if (it.stop) break;
        const int c0 = it.tile0, c1 = it.tile0 + it.ntile;
        const KeyBoxes<kD, kSrc> box(p, it, lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.iempty[slot]);
        int page = box.page(p, c0);
#pragma unroll 1
        for (int j = c0; j < c1; ++j, ++T) {
          const int st = T % kVStages;
          if (!row_wait(&S.vempty[st], ((T / kVStages) & 1u) ^ 1u, &S.abort_flag)) { ok = false; break; }
          box.load(p, &tmap_v, &S.vfull[st], S.v[st][0], j, page);
          if (j + 1 < c1) page = box.page(p, j + 1);
        }
      }
      if (S.abort_flag && lane == 0)
        for (uint32_t back = 1; back <= kVStages && back <= T; ++back) (void)row_poll(&S.vfull[(T - back) % kVStages], ((T - back) / kVStages) & 1u);
    } else if (warp == kRwIssue) {
      // ======================= tensor-core issue =======================
      // Of a two-tile item, tile by tile and lane by lane: P·V of tile i - 1, then the scores of tile i over
      // the P just read (products of one thread run in the order of their issue). The lanes' products
      // alternate, so that one lane's softmax runs beside the other's products: with a thread a lane the
      // commits queued behind the other lane's products, both softmaxes ran at once, and a tile took 4830
      // cycles. Scores ahead of P·V did not pay: D 128 has the columns for half a tile only, and a 128 x 64
      // product costs the tensor pipe as much as a 128 x 128 one (849 instead of 1098 TFLOP/s at 16384);
      // with D 64, which has them for a whole tile, 602 instead of 644 TFLOP/s at 8192. An item of one row
      // tile has its lanes on alternate key tiles.
      const uint32_t idesc_s = idesc_bf16_f32(128, 128, false, false);
      const uint32_t idesc_o = idesc_bf16_f32(128, kD, false, true);
      const uint64_t q_desc = smem_desc(smem_u32(S.q[0][0]), 16, 1024, kLayoutSW128);
      const uint64_t k_desc = smem_desc(smem_u32(S.k[0][0]), 16, 1024, kLayoutSW128);
      const uint64_t v_desc = smem_desc(smem_u32(S.v[0][0]), kRwHalf, 1024, kLayoutSW128);
      constexpr uint32_t kTileDesc = kHalves * (kRwHalf >> 4);  // 128 rows in the start-address field
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      // A lane's state (both lanes' stay in registers: every use names its lane at compile time).
      struct Turn {
        uint32_t pend = 0;        // 1 + the tile count T of the tile whose product is still to issue
        uint32_t steps = 0;       // its key steps of 16
        uint32_t J = 0;           // tiles of the lane started
        int first = 0, last = 0;  // the pending tile is its item's first (2 + a parity) / last
        bool alone = false;       // the other lane does not use it
        int i = 0, used = 0, kend = 0;  // this item: tiles done, all, the end of the lane's keys
      } st0, st1;
      uint32_t T = 0;  // tiles of the items before
      bool ok = true;
      // the scores of tile count t into the lane's columns
      auto scores = [&](auto lane_no, uint32_t t) -> bool {
        constexpr int L = decltype(lane_no)::value;
        const uint32_t st = t % kKStages;
        if (!row_wait_warp(&S.kfull[st], (t / kKStages) & 1u, &S.abort_flag)) return false;
        tc_fence_after();
        const uint64_t qd = q_desc + static_cast<uint64_t>(kPairs ? L * kTileDesc : 0), kd = k_desc + static_cast<uint64_t>(st * kTileDesc);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kD / 16; ++kk) {
            const uint64_t off = static_cast<uint64_t>((kk >> 2) * (kRwHalf >> 4) + (kk & 3) * 2);
            umma_bf16_ss(tm + 128 * L, qd + off, kd + off, idesc_s, kk > 0 ? 1u : 0u);
          }
          umma_commit(&S.sfull[L]);  // the softmax gives K's stage back
        }
        __syncwarp();
        return true;
      };
      auto product = [&](auto lane_no, Turn& st) -> bool {  // P·V of the lane's pending tile
        constexpr int L = decltype(lane_no)::value;
        const uint32_t t = st.pend - 1, sv = t % kVStages;
        st.pend = 0;
        if (!row_wait_warp(&S.vfull[sv], (t / kVStages) & 1u, &S.abort_flag)) return false;
        if (st.first != 0 && !row_wait_warp(&S.oempty[L], st.first & 1u, &S.abort_flag)) return false;
        const uint32_t s_col = tm + 128 * L, o_col = tm + kRwColO + kD * L;
        const uint64_t vd = v_desc + static_cast<uint64_t>(sv * kTileDesc);
        const uint32_t acc = st.first != 0 ? 0u : 1u;
#pragma unroll
        for (uint32_t half = 0; half < 2; ++half) {
          if (!row_wait_warp(&S.pfull[L][half], (st.J - 1) & 1u, &S.abort_flag)) return false;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (uint32_t kk = 4 * half; kk < 4 * half + 4; ++kk)
              if (kk < st.steps) umma_bf16_ts(o_col, s_col + 8 * kk, vd + static_cast<uint64_t>(kk * 128), idesc_o, kk > 0 ? 1u : acc);
          }
        }
        if (elect_one()) {
          umma_commit(&S.vempty[sv]);
          if (st.alone) umma_commit(&S.vempty[sv]);
          if (st.last != 0) umma_commit(&S.ofin[L]);
        }
        __syncwarp();
        return true;
      };
      // the lane's next tile of this item, count t, whose scores are issued
      auto started = [&](auto lane_no, Turn& st, uint32_t K, uint32_t t, int tile, bool alone) {
        constexpr int L = decltype(lane_no)::value;
        st.pend = t + 1;
        // key steps of 16 up to the lane's last visible key
        st.steps = static_cast<uint32_t>(min(128, st.kend - tile * 128) + 15) >> 4;
        st.first = st.i == 0 ? 2 + static_cast<int>((K & 1u) ^ 1u) : 0;
        st.last = ++st.i == st.used;
        st.alone = alone;
        if (st.last != 0 && elect_one()) umma_commit(&S.qempty[L]);
        __syncwarp();
        ++st.J;
      };
      // a tile of the lane, after the product that is still to issue
      auto begin = [&](auto lane_no, Turn& st, uint32_t K, uint32_t t, int tile, bool alone) -> bool {
        constexpr int L = decltype(lane_no)::value;
        if (st.pend != 0 && !product(lane_no, st)) return false;  // first: its output waits for it
        if (st.i == 0 && !row_wait_warp(&S.qfull[kPairs ? L : 0], K & 1u, &S.abort_flag)) return false;
        if (!scores(lane_no, t)) return false;
        started(lane_no, st, K, t, tile, alone);
        return true;
      };
      // an item that gives the lane nothing to do: its Q goes back unread, its (empty) O is there
      auto skip = [&](auto lane_no, Turn& st, uint32_t K) -> bool {
        constexpr int L = decltype(lane_no)::value;
        if (st.pend != 0 && !product(lane_no, st)) return false;
        if (!row_wait_warp(&S.qfull[kPairs ? L : 0], K & 1u, &S.abort_flag)) return false;
        if (lane == 0) mbar_arrive(&S.qempty[L]);
        if (!row_wait_warp(&S.oempty[L], (K & 1u) ^ 1u, &S.abort_flag)) return false;
        if (lane == 0) mbar_arrive(&S.ofin[L]);
        return true;
      };
      constexpr std::integral_constant<int, 0> lane0{};
      constexpr std::integral_constant<int, 1> lane1{};
      for (uint32_t K = 0; ok; ++K) {
        const int slot = K & (kRwItems - 1);
        if (!row_wait_warp(&S.ifull[slot], (K / kRwItems) & 1u, &S.abort_flag)) { ok = false; break; }
        const RowItem& it = S.item[slot];
        const auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
        if (uniform(it.stop)) break;
        const int ntile = uniform(it.ntile);
        const bool alt = !kPairs || uniform(it.alt);
        st0.i = st1.i = 0;
        st0.used = uniform(it.used[0]);
        st1.used = uniform(it.used[1]);
        st0.kend = uniform(it.kend[0]);
        st1.kend = uniform(it.kend[1]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.iempty[slot]);
        if (!kPairs || alt) {
#pragma unroll 1
          for (int j = 0; ok && j < ntile; ++j)
            ok = (j & 1) == 0 ? begin(lane0, st0, K, T + j, j, true) : begin(lane1, st1, K, T + j, j, true);
          if (ok && st1.used == 0) ok = skip(lane1, st1, K);
        } else if constexpr (kPairs) {
          // lane 1 uses every tile, lane 0 all but the last or all
          const int n0 = st0.used;
          if (n0 > 0) ok = begin(lane0, st0, K, T, 0, false);
          ok = ok && begin(lane1, st1, K, T, 0, n0 == 0);
          if (ok && n0 == 0) ok = skip(lane0, st0, K);
          // Tiles that both lanes use: whole products of the tile before. Kept lean: with the bookkeeping
          // of begin() in this loop the issuing warp, not the tensor pipe, set the pace (976 instead of
          // 1073 TFLOP/s at 4096).
          const uint32_t first = (K & 1u) ^ 1u;
#pragma unroll 1
          for (int j = 1; ok && j < n0; ++j) {
            const uint32_t tv = T + j - 1, ts = T + j;
            const uint32_t sv = tv % kVStages, sk = ts % kKStages;
            ok = row_wait_warp(&S.vfull[sv], (tv / kVStages) & 1u, &S.abort_flag) &&
                 row_wait_warp(&S.kfull[sk], (ts / kKStages) & 1u, &S.abort_flag);
            if (j == 1)
              ok = ok && row_wait_warp(&S.oempty[0], first, &S.abort_flag) && row_wait_warp(&S.oempty[1], first, &S.abort_flag);
            if (!ok) break;
            const uint64_t vd = v_desc + static_cast<uint64_t>(sv * kTileDesc), kd = k_desc + static_cast<uint64_t>(sk * kTileDesc);
            const uint32_t acc = j > 1 ? 1u : 0u;
            auto lean = [&](auto lane_no, Turn& st, bool last) -> bool {
              constexpr int L = decltype(lane_no)::value;
              const uint32_t s_col = tm + 128 * L, o_col = tm + kRwColO + kD * L, parity = (st.J - 1) & 1u;
              if (!row_wait_warp(&S.pfull[L][0], parity, &S.abort_flag)) return false;
              tc_fence_after();
              if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  umma_bf16_ts(o_col, s_col + 8 * kk, vd + static_cast<uint64_t>(kk * 128), idesc_o, kk > 0 ? 1u : acc);
              }
              if (!row_wait_warp(&S.pfull[L][1], parity, &S.abort_flag)) return false;
              tc_fence_after();
              if (elect_one()) {
#pragma unroll
                for (int kk = 4; kk < 8; ++kk)
                  umma_bf16_ts(o_col, s_col + 8 * kk, vd + static_cast<uint64_t>(kk * 128), idesc_o, 1u);
                umma_commit(&S.vempty[sv]);
#pragma unroll
                for (int kk = 0; kk < kD / 16; ++kk) {
                  const uint64_t off = static_cast<uint64_t>((kk >> 2) * (kRwHalf >> 4) + (kk & 3) * 2);
                  umma_bf16_ss(s_col, q_desc + L * kTileDesc + off, kd + off, idesc_s, kk > 0 ? 1u : 0u);
                }
                umma_commit(&S.sfull[L]);
                if (last) umma_commit(&S.qempty[L]);
              }
              ++st.J;
              __syncwarp();
              return true;
            };
            ok = lean(lane0, st0, j == n0 - 1) && lean(lane1, st1, j == ntile - 1);
          }
          if (n0 > 1) {
            auto forward = [&](Turn& st) {
              st.pend = T + n0;
              st.steps = static_cast<uint32_t>(min(128, st.kend - (n0 - 1) * 128) + 15) >> 4;
              st.first = 0;
              st.alone = false;
              st.i = n0;
              st.last = n0 == st.used;
            };
            forward(st0);
            forward(st1);
          }
          if (ok && ntile > n0 && ntile > 1) ok = begin(lane1, st1, K, T + ntile - 1, ntile - 1, true);  // lane 1's last
        }
        T += ntile;
      }
      if (ok && st0.pend != 0) ok = product(lane0, st0);
      if (ok && st1.pend != 0) ok = product(lane1, st1);
      if (elect_one()) umma_commit(&S.drain);
      __syncwarp();
      (void)row_poll(&S.drain, 0);
    }
    __syncwarp();
  } else {
    // ======================= softmax and output of one lane, one row a thread =======================
    set_regs_more<208>();
    const int L = warp >> 2, quad = warp & 3;
    const int r = quad * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t o_base = tmem + lane_base + kRwColO, s_col = tmem + lane_base + 128 * L, o_col = o_base + kD * L;
    const int pos_in = (r * p.g_recip16) >> 16;  // r / G
    const uint64_t scale2 = pair_f32(p.scale_log2, p.scale_log2);
    uint32_t T = 0, J = 0, X = 0;  // key tiles, the lane's tiles, exchanges
    bool ok = true;
    for (uint32_t K = 0; ok; ++K) {
      const int slot = K & (kRwItems - 1);
      if (!row_wait(&S.ifull[slot], (K / kRwItems) & 1u, &S.abort_flag)) break;
      const RowItem& it = S.item[slot];  // stays in shared memory: the scores need the registers
      if (it.stop) break;
      const int used = it.used[L];
      const bool alt = !kPairs || it.alt;
      const int both = alt ? 0 : it.used[0];        // tiles that both lanes use
      const int pos = pos_in + (alt ? 0 : L * tpt);  // token of the item
      const bool row_ok = pos_in < it.tokens[L];
      float m = -INFINITY;
      uint64_t sum2[4];
#pragma unroll
      for (int a = 0; a < 4; ++a) sum2[a] = 0;
      for (int i = 0; i < used; ++i, ++J) {
        const int j = alt ? 2 * i + L : i, tile = it.tile0 + j;
        const uint32_t t = T + j;
        uint32_t w[4];
        // tiles that every row of this warp sees whole need no mask
        bool full;
        if constexpr (kCausal) full = __all_sync(0xffffffffu, !row_ok || it.t0 + pos + 1 >= tile * 128 + 128);
        else full = tile * 128 + 128 <= it.prefix;
        if (!full) visible_words<kCausal>(p, it, tile, pos, row_ok, static_cast<int64_t>(it.row0) + pos, w);
        if (!row_wait(&S.sfull[L], J & 1u, &S.abort_flag)) { ok = false; break; }
        tc_fence_after();
        // K is no longer read (its stage expects two arrivals; a tile of one lane gives both)
        if (warp == 4 * L && lane == 0) mbar_arrive_n(&S.kempty[t % kKStages], i < both ? 1u : 2u);
        if (!full) {
          // in tensor memory, so that the scores below come straight from there in every tile
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t y[32];
            tmem_ld32(s_col + 32 * c, y);
            tmem_wait_ld();
            const uint32_t bits = c < 2 ? (c == 0 ? w[0] : w[1]) : (c == 2 ? w[2] : w[3]);
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = (bits >> e) & 1u ? y[e] : 0xff800000u;
            tmem_st32(s_col + 32 * c, y);
          }
          tmem_wait_st();
        }
        const int valid = it.k1 - tile * 128;
        if (valid < 128 && (valid & 15) != 0) {
          // zero V rows [valid, next multiple of 16): they may lie behind the request's keys
          if (!row_wait(&S.vfull[t % kVStages], (t / kVStages) & 1u, &S.abort_flag)) { ok = false; break; }
          const int r0 = valid, nr = ((valid + 15) & ~15) - r0;
          for (int c = r; c < nr * 8 * kHalves; c += 128) {
            const int row = r0 + c / (8 * kHalves);
            *reinterpret_cast<uint4*>(reinterpret_cast<unsigned char*>(S.v[t % kVStages][(c / 8) % kHalves]) + row * 128 +
                                      (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        uint32_t x[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_col + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(x + 32 * c));
        tmem_wait_ld();
        // weights 2^(score - m) of 64 scores as bf16 pairs, their sums into add2. -m: 0 where every score is
        // -inf so far, NaN for a row that saw +inf (as for one that saw NaN)
        uint64_t add2[4];
        auto weights = [&](int half, uint32_t (&out)[32]) {
          const float n = m == -INFINITY ? 0.f : fmaf(m, 0.f, -m);
          const uint64_t negm2 = pair_f32(n, n);
#pragma unroll
          for (int e = 0; e < 64; e += 2) {
            float a0, a1;
            unpair_f32(fma_f32x2(pair_f32(__uint_as_float(x[64 * half + e]), __uint_as_float(x[64 * half + e + 1])), scale2, negm2), a0, a1);
            a0 = fast_exp2(a0);
            a1 = fast_exp2(a1);
            out[e >> 1] = pack_bf16(a0, a1);
            add2[(e >> 1) & 3] = add_f32x2(add2[(e >> 1) & 3], pair_f32(a0, a1));
          }
        };
        // The first half of the tile is weighted with the maximum so far while the whole tile's maximum
        // is found beside it; only where that has grown by more than 2^8 is it weighted again.
        uint32_t out[32];
        bool checked = false;
        for (;;) {
#pragma unroll
          for (int a = 0; a < 4; ++a) add2[a] = 0;
          if (i > 0 || checked) weights(0, out);
          if (checked) break;
          checked = true;
          float mx[4];
#pragma unroll
          for (int a = 0; a < 4; ++a) mx[a] = max3_f32(__uint_as_float(x[2 * a]), __uint_as_float(x[2 * a + 1]), -INFINITY);
#pragma unroll
          for (int e = 8; e < 128; e += 8)
#pragma unroll
            for (int a = 0; a < 4; ++a)
              mx[a] = max3_f32(mx[a], __uint_as_float(x[e + 2 * a]), __uint_as_float(x[e + 2 * a + 1]));
          const float mn = max3_f32(m, max3_f32(max3_f32(mx[0], mx[1], mx[2]), mx[3], -INFINITY) * p.scale_log2, -INFINITY);
          const bool move = !(mn <= m + kRwRescale);  // from -inf, and for NaN too
          if (i > 0 && !__any_sync(0xffffffffu, move)) break;
          const float alpha = move ? (m == -INFINITY ? 0.f : fast_exp2(m - mn)) : 1.f;
          if (move) m = mn;
          if (i > 0) {
            // the scores of this tile were issued after the last product into O, and are there
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
        }
        tmem_st32(s_col, out);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.pfull[L][0]);
        weights(1, out);
        tmem_st32(s_col + 32, out);
#pragma unroll
        for (int a = 0; a < 4; ++a) sum2[a] = add_f32x2(sum2[a], add2[a]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.pfull[L][1]);
      }
      if (!ok) break;
      T += it.ntile;
      float l, f0 = 1.f, f1 = 0.f;  // O = f0 O_lane0 + f1 O_lane1 (alt)
      {
        float s[8];
#pragma unroll
        for (int a = 0; a < 4; ++a) unpair_f32(sum2[a], s[2 * a], s[2 * a + 1]);
        l = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
      }
      // While the last product runs: the row's own part of the output, and where it goes.
      if (alt) {
        // the other lane's part of the row: post, meet, read. The next post but one finds it read: it comes
        // after the next meeting.
        S.xend[X & 1u][warp][lane] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.xpair[quad]);
      }
      char* dst[4];
      row_places(p, it, quad, lane, alt ? 0 : L, tpt, dst);
      if (alt) {
        if (!row_wait(&S.xpair[quad], X & 1u, &S.abort_flag)) break;
        const float2 y = S.xend[X & 1u][warp ^ 4][lane];
        ++X;
        const float ma = L == 0 ? m : y.x, mb = L == 0 ? y.x : m, la = L == 0 ? l : y.y, lb = L == 0 ? y.y : l;
        m = fmaxf(ma, mb);
        f0 = la == 0.f ? 0.f : fast_exp2(ma - m);
        f1 = lb == 0.f ? 0.f : fast_exp2(mb - m);
        l = la * f0 + lb * f1;
      }
      const float scale = it.whole ? row_over(l) : 1.f;
      if (!row_wait(&S.ofin[L], K & 1u, &S.abort_flag) || (alt && !row_wait(&S.ofin[L ^ 1], K & 1u, &S.abort_flag)) ||
          !row_wait(&S.cfull[slot], (K / kRwItems) & 1u, &S.abort_flag))
        break;
      tc_fence_after();
      if (alt) row_output<kD, true>(p, S, it, warp, lane, 0, L * (kD / 2), (L + 1) * (kD / 2), o_base, tpt, dst, m, l, scale, f0, f1);
      else if constexpr (kPairs) row_output<kD, false>(p, S, it, warp, lane, L, 0, kD, o_col, tpt, dst, m, l, scale, 1.f, 0.f);
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

template <int kD, int kSrc, bool kPairs>
cudaError_t launch_rows_t(const RowsParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                          int nctas, cudaStream_t stream) {
  const size_t smem = sizeof(RwSmem<kD, kPairs>) + 1024;
  cudaError_t e = cudaFuncSetAttribute(rows_tc_kernel<kD, kSrc, kPairs>, cudaFuncAttributeMaxDynamicSharedMemorySize,
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
  return cudaLaunchKernelEx(&cfg, rows_tc_kernel<kD, kSrc, kPairs>, p, tq, tk, tv);
}

}  // namespace

size_t rows_workspace_bytes(int d, int nctas) {
  return sizeof(WsHeader) + static_cast<size_t>(2 * nctas) * (2 * 128 * d * sizeof(float) + 8 * 32 * sizeof(float2));
}

cudaError_t launch_rows(RowsParams p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, int nctas,
                        cudaStream_t stream) {
  char* base = reinterpret_cast<char*>(p.hdr);
  p.front = reinterpret_cast<WsFront*>(base) - 1;
  p.part_o = reinterpret_cast<float*>(base + sizeof(WsHeader));
  p.part_ml = p.part_o + static_cast<int64_t>(2 * nctas) * 2 * 128 * p.d;
  const int src = p.prefix_lens == nullptr ? kSrcPacked : p.block_table ? kSrcPaged : kSrcCache;
  const auto launch = [&](auto d, auto pairs) {
    constexpr int kD = decltype(d)::value;
    constexpr bool kPairs = decltype(pairs)::value;
    if (src == kSrcPacked) return launch_rows_t<kD, kSrcPacked, kPairs>(p, tq, tk, tv, nctas, stream);
    if (src == kSrcCache) return launch_rows_t<kD, kSrcCache, kPairs>(p, tq, tk, tv, nctas, stream);
    return launch_rows_t<kD, kSrcPaged, kPairs>(p, tq, tk, tv, nctas, stream);
  };
  const std::integral_constant<int, 128> d128{};
  const std::integral_constant<int, 64> d64{};
  if (rows_two_tiles(p.rows, p.batch, p.hkv, p.g, nctas)) return p.d == 128 ? launch(d128, std::true_type{}) : launch(d64, std::true_type{});
  return p.d == 128 ? launch(d128, std::false_type{}) : launch(d64, std::false_type{});
}

}  // namespace fd
