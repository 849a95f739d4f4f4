// How the attention of packed query rows (rows_tc.cu) is divided over the CTAs.
//
// Request b with n rows is cut into items of `span` tokens, T or 2 T with T = 128 / G: one or two 128-row
// tiles (T tokens of all G query heads of one KV head) that walk the same key tiles. The items of
// all (request, KV head, span of tokens) stand in one line, each as long as its work, counted in 1/128
// of a key tile plus a fixed part; CTA i of n takes the stretch [W i / n, W (i + 1) / n). An item
// that a stretch ends in is cut at the key tile in proportion, so that every CTA has the same work
// whatever the lengths are; its pieces are merged by the last of their CTAs to finish. A cut that
// would leave a piece below kMinPiece key tiles is moved to the item's nearer end: such a piece
// costs less than a merge does. Every CTA derives its own stretch from the lengths; there is no plan
// in memory.
#pragma once

#include <stdint.h>

#include "plan.h"

namespace fd {

constexpr int32_t kItemFixed = 256;  // an item's fixed cost (Q, first scores, output): two key tiles
constexpr int32_t kMinPiece = 4;     // key tiles of the smallest piece of a cut item
constexpr int32_t kMaxRowCtas = 192; // CTAs of one call (merge counters in front of the workspace)

FD_HD int32_t rows_tile_tokens(int32_t g) { return kQTile / g; }
FD_HD int32_t rows_items(int32_t n, int32_t span) { return cdiv32(n, span); }

// Two row tiles an item (K and V come once for both), or one? One where two would leave CTAs without an
// item, and where the requests' mean length fits one tile. Seen from the host, which has the sums of the
// lengths at most. Drafted trees of 1 to 64 over 8 requests of up to 8000 keys, 8 KV heads, G 4 (64 two-tile
// items): 61.7 us with one tile, 64.5 with two, whose pieces are twice the bytes to merge; 32 trees of 16
// drafts, G 8, 5 to 32 K keys: 466 and 473 us.
FD_HD bool rows_two_tiles(int32_t rows, int32_t batch, int32_t hkv, int32_t g, int32_t nctas) {
  const int64_t t = rows_tile_tokens(g);
  return rows > t * batch && (rows / (2 * t) + batch) * hkv >= nctas;
}

// Work of the first u items of one (request, KV head). A prompt's item u sees (u + 1) span keys, taken
// as half a tile more on average when rounded up to tiles; every item of a tree sees all its keys.
FD_HD int64_t rows_weight(bool causal, int32_t span, int32_t keys, int64_t u) {
  return causal ? u * (kItemFixed + 64) + ((span * u * (u + 1)) >> 1)
                : u * (kItemFixed + static_cast<int64_t>(cdiv32(keys, 128)) * 128);
}

// Keys that item u of a request sees.
FD_HD int32_t rows_item_keys(bool causal, int32_t span, int32_t n, int32_t keys, int32_t u) {
  if (!causal) return keys;
  const int64_t end = static_cast<int64_t>(u + 1) * span;
  return end < n ? static_cast<int32_t>(end) : n;
}

// CTAs that take part: as many as there are items, or as there are stretches of kMinPiece tiles.
FD_HD int32_t rows_active(int64_t weight, int64_t items, int32_t nctas) {
  const int64_t n = weight / (kMinPiece * 128);  // a shift
  const int64_t m = items > n ? items : n;
  return m < nctas ? (m < 1 ? 1 : static_cast<int32_t>(m)) : nctas;
}

// The line cut into stretches, of `share` units each and one more in the first `rest`. Dividing 64-bit
// integers is a subroutine of ~100 dependent instructions, and a CTA looks at some twenty bounds before
// its first load: one division here, of 32-bit integers or in doubles, none below.
struct RowsLine {
  int64_t share;
  int32_t rest, nact;
};
FD_HD int64_t rows_quotient(int64_t x, int64_t d) {  // floor(x / d), x >= 0, d > 0
  if (((x | d) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(d);
  int64_t q = static_cast<int64_t>(static_cast<double>(x) / static_cast<double>(d));
  while (q * d > x) --q;
  while ((q + 1) * d <= x) ++q;
  return q;
}
FD_HD RowsLine rows_line(int64_t weight, int32_t nact) {
  RowsLine n;
  n.share = rows_quotient(weight, nact);
  n.rest = static_cast<int32_t>(weight - n.share * nact);
  n.nact = nact;
  return n;
}
// Where CTA i's stretch begins (i = nact: the line's end).
FD_HD int64_t rows_bound(const RowsLine& n, int32_t i) { return n.share * i + (i < n.rest ? i : n.rest); }

// The key tile at which the point x of the line cuts an item of `tiles` key tiles at [a, a + w). In fp32:
// every CTA finds the same tile, and each rounding keeps the order of two points.
FD_HD int32_t rows_cut(int64_t x, int64_t a, int64_t w, int32_t tiles) {
  if (x <= a) return 0;
  if (x >= a + w) return tiles;
  const float part = static_cast<float>(static_cast<uint32_t>(x - a)) / static_cast<float>(static_cast<uint32_t>(w));
  const int32_t t = static_cast<int32_t>(part * static_cast<float>(tiles));
  if (t < kMinPiece) return 0;
  return tiles - t < kMinPiece ? tiles : t;
}

// The cuts of an item: bounds first .. first + count - 1 cut it (count 0: one CTA has all of it).
// Bounds that lie inside the item without cutting it stand at its ends, a few at most.
FD_HD void rows_cuts(const RowsLine& n, int64_t a, int64_t w, int32_t tiles, int32_t cta, int32_t* first, int32_t* count) {
  int32_t lo = cta, hi = cta;  // a bound in or at the item: the caller's own stretch meets the item
  while (lo > 0 && rows_cut(rows_bound(n, lo), a, w, tiles) > 0) {
    // step down in strides as long as the bound stays inside
    int32_t step = 1;
    while (lo - 2 * step > 0 && rows_cut(rows_bound(n, lo - 2 * step), a, w, tiles) > 0) step *= 2;
    lo -= step;
  }
  ++lo;
  while (rows_cut(rows_bound(n, lo), a, w, tiles) == 0) ++lo;  // bounds snapped to the start
  if (hi < lo) hi = lo;
  while (hi < n.nact && rows_cut(rows_bound(n, hi), a, w, tiles) < tiles) {
    int32_t step = 1;
    while (hi + 2 * step < n.nact && rows_cut(rows_bound(n, hi + 2 * step), a, w, tiles) < tiles) step *= 2;
    hi += step;
  }
  *first = lo;
  *count = hi - lo;
}

}  // namespace fd
