// The work of a batch of prompts: items of 512 query rows of one head (or of two heads' rows, where
// a request has 256 at most), each with the tiles of 128 keys that its rows see, and how all items
// lie on one line of places: a place for each tile, then kExtra for what an item costs besides. A
// pair of CTAs takes an item, as two halves of 256 rows. Host and device code include this.
#pragma once

#include "internal.h"

namespace mlafold {
namespace prompt {

constexpr int kRows = 512;       // query rows of an item
constexpr int kHalf = 256;       // of its half
constexpr int kKeys = 128;       // keys of a tile
constexpr int kStep = kRows / kKeys;
// Requests of no more rows than a half have two heads to an item, a half each (up to 148 rows, 27
// requests of 64 heads: 196 -> 135 us; 95 rows on 1,700 keys, four heads to a K and V: 656 -> 381 us;
// 9 rows on 800 keys each: 494 -> 379 us).
constexpr int kAlone = 256;
// Items of no more tiles are never cut, so that batches of up to 512 keys need no launch that joins
// pieces. (2, 4 and 8 measured the same.)
constexpr int kUncut = 4;
// Places of a part, at least (64 heads of 8k: 924 us with 1, 917 with 3 and 6).
constexpr int kMinPart = 3;
// What an item costs besides its tiles: its first softmax, its output (24 prompts up to 2k: 141 us with 0,
// 128 with 1, 125 with 2; 512 rows on 16k keys 49.5, 47.7, 46.5; with 3 and 4 some gain, some lose).
constexpr int kExtra = 2;
// Items stay whole where a pair has so many of the longest's tiles (3: 24 prompts up to 2k 136 us, 128
// with 6; 20, and 64 heads of 8k are cut: 934 us, 917 with 6).
constexpr int kWhole = 6;

// A request of n query tokens and m keys; causal: query i sees keys j <= i + m - n.
struct Request {
  int n, m;
  bool causal;
};

// ceil(x / 128) for any x.
__host__ __device__ inline int tiles_of(int x) { return x >= 0 ? (x + 127) >> 7 : -((-x) >> 7); }

__host__ __device__ inline int items(const Request& q) { return (q.n + kRows - 1) / kRows; }
// Keys that query row i sees.
__host__ __device__ inline int limit(const Request& q, int i) {
  if (!q.causal) return q.m;
  const int e = i + 1 + (q.m - q.n);
  return e < 0 ? 0 : e < q.m ? e : q.m;
}
// Whether a request has two heads to an item.
__host__ __device__ inline bool twins(const Request& q, bool allowed) { return allowed && q.n <= kAlone; }
// Heads, or pairs of heads, that have items of their own.
__host__ __device__ inline int units(const Request& q, int H, bool allowed) {
  return twins(q, allowed) ? (H + 1) / 2 : H;
}
// Tiles of item u: those that its last row sees, one where there are none.
__host__ __device__ inline int item_tiles(const Request& q, int u) {
  const int last = (u + 1) * kRows < q.n ? (u + 1) * kRows : q.n;
  const int t = tiles_of(limit(q, last - 1));
  return t < 1 ? 1 : t;
}
// Tiles of the items before item u, 0 <= u <= items. All items but the last have 512 rows,
// so item v of them sees 512 (v + 1) + m - n keys: max(1, 4 (v + 1) + ceil((m - n) / 128))
// tiles, of which the first z are ones.
__host__ __device__ inline long long tiles_before(const Request& q, int u) {
  const int I = items(q);
  if (I == 0) return 0;
  const long long v = u < I ? u : I - 1, last = u < I ? 0 : item_tiles(q, I - 1);
  if (!q.causal) {
    const int t = tiles_of(q.m);
    return v * (t < 1 ? 1 : t) + last;
  }
  const long long c = tiles_of(q.m - q.n);
  long long z = c < 0 ? -c / kStep : 0;
  if (z > v) z = v;
  return z + kStep / 2 * (v * (v + 1) - z * (z + 1)) + (v - z) * c + last;
}
// Places of the items before item u.
__host__ __device__ inline long long before(const Request& q, int u) {
  return tiles_before(q, u) + (long long)kExtra * u;
}
__host__ __device__ inline long long places(const Request& q) { return before(q, items(q)); }
// x = unit * per + rest, 0 <= rest < per, without a division of 64 bits.
__host__ __device__ inline int head_at(long long x, long long per, int H) {
  int lo = 0, hi = H;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (mid * per <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}
// The item that holds place x of its head, 0 <= x < places.
__host__ __device__ inline int item_at(const Request& q, long long x) {
  int lo = 0, hi = items(q);
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (before(q, mid) <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Items in the order in which they are claimed: heads in groups, within a group the longest
// first, so that the last ones are short and few heads' keys are in use at a time. Groups of equal
// size, of about `wide` items. x = item of the request -> its head and place in it.
__host__ __device__ inline void claimed_item(const Request& q, int H, int wide, int x, int& head, int& u) {
  const int I = items(q), most = (wide + I - 1) / I, groups = most < H ? H / most : 1;
  const int heads = (H + groups - 1) / groups;
  const int g = x / (heads * I), y = x - g * heads * I;
  const int here = H - g * heads < heads ? H - g * heads : heads;
  u = I - 1 - y / here;
  head = g * heads + y % here;
}

// The plan in the workspace: this, then the requests' first places and items (R + 1 each), then a
// Join for each pair.
struct Plan {
  long long total, all_items;    // places and items of the batch
  long long len;                 // places of a part
  int parts;                     // > 0: the line is cut into so many; 0: whole items, claimed
  int claimed;                   // items claimed beyond the first of each pair
};
// An item that a cut runs through, by the pair whose part it begins in (rows 0: none): its pieces
// are that part's last and the first ones of the parts up to `last`.
struct Join {
  int row0, rows, head, last;    // last: with a bit below it, whether the item has two heads
};
// Where part p begins.
__host__ __device__ inline long long part_at(long long total, long long len, int p) {
  return len * p < total ? len * p : total;
}
// How a batch is shared out among the pairs of CTAs, by its places and its longest item: whole
// items where a pair's share is worth several of them, claimed one by one, else equal parts of
// the line.
__host__ __device__ inline bool whole_items(long long total, int longest, int pairs) {
  return longest <= kUncut || total >= (long long)kWhole * longest * pairs;
}
// Parts aimed at; their length is total over them, rounded up, which may leave fewer.
__host__ __device__ inline int parts_of(long long total, int pairs) {
  const long long p = cdiv(total, kMinPart);
  return (int)(p < pairs ? p : pairs);
}

constexpr size_t kSlotBytes = (size_t)kRows * 128 * 4;     // a piece's FP32 rows
inline int pairs_of(int ctas) { return ctas < 2 ? 1 : ctas / 2; }
inline size_t plan_bytes(int R, int pairs) {
  return align256(sizeof(Plan) + 2 * (size_t)(R + 1) * 8 + (size_t)pairs * sizeof(Join));
}
inline size_t lse_bytes(int pairs) { return align256((size_t)2 * pairs * kRows * 4); }

}  // namespace prompt
}  // namespace mlafold
