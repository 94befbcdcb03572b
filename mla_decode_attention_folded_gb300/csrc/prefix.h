// The shared-prefix decode's work: which (rows, keys) tiles there are and how they
// are cut into parts (prefix_wide.cu computes them, prefix.cu plans and joins).
//
// A segment is a block of up to 128 rows with the keys it attends to: block b of
// all N rows with the prefix's keys (segments 0 .. blocks - 1), then block j of
// request r's M rows with the request's own keys (segment blocks + r * own_blocks
// + j). A segment of t > 0 tiles takes t places and a few more of one line of places,
// one per tile, the others for what a piece costs besides (Q, new maxima, 256 KB of
// partial rows out); segments without keys take none.
// The line is cut into equal parts, part u from floor(u * places / used), one per
// pair of CTAs. The piece of segment s that part u holds has partial slot u + s:
// along the line one of the two grows with every piece, so no two share a slot and
// a segment's slots are consecutive.
#pragma once

#include "internal.h"

namespace mlafold {

constexpr int kWideRows = 128;     // query rows per block
constexpr int kWideKeys = 256;     // keys per tile
// A piece costs about three tiles' time. Measured with 2, 3, 4: 32 x 4 x 8 behind 4k 27.8,
// 29.2, 29.1 us; 64 x 7 x 8 behind 16k 102, 99, 99 us; 24 x 1 x 64 behind 64k 132, 115, 114
// us; 128 x 7 x 64 behind 16k 1200, 1149, 1148 us; geometric mean over 21 shapes 40.2, 39.3,
// 39.8 us (the five listed by perf/operators.py and 16 drawn, random.Random(77)); over 35 others
// (random.Random(101)) 2.2 % and 0.1 % above that for 3.
// A cost of its own for pieces of own keys gains 2-5 % there at 2 and 5, and loses 4 %
// over 21 shapes.
constexpr int kWideCost = 3;
// A tile of own keys takes about an eighth longer beside a long prefix, since they come from
// HBM where the prefix's come from L2: one place more for every 8, behind a segment's tiles.
// Without, and for every 16, 8, 4: 64 x 7 x 8 behind 16k 101, 100, 98, 97 us; 128 x 7 x 64
// behind 16k 1134, 1123, 1102, 1113 us; 4 x 2 x 8 behind 20k, up to 9k own keys 35.5, 35.2,
// 34.5, 34.1 us. It costs where nearly all keys are own ones, as the part at a segment's end
// then has fewer tiles than the others: 44 x 2 x 16 behind 12, up to 10k own keys 58.5, 58.7,
// 64.5, 65.8 us; 13 x 7 x 64 behind 8, up to 13k 63.6, 63.3, 68.4, 69.3 us. Over 35 shapes
// drawn by perf/operators.py (random.Random(101)), most of them within 1 %, the geometric mean
// is 1.1, 0.8, 0, 0.5 % below that for 8.
constexpr int kOwnSlow = 8;

struct WideArgs {
  const int32_t* prefix_table;     // [prefix_pages]
  const int32_t* prefix_len;       // [1]
  const int32_t* block_table;      // [R][max_pages]
  const int32_t* seq_lens;         // [R]
  int32_t* plan;                   // [R + 1]: first place of each request's segments
  float* part_o;                   // [slots][128][512]
  float* part_lse;                 // [slots][128]
  int32_t* status;                 // may be null
  float bmm1_log2;
  long long N;                     // query rows
  int R, M, prefix_pages, max_pages, num_pages, units, blocks, own_blocks;
  int own_tiles, own_most;         // tiles of a full table row, places when all rows are full
  // Failure-detection test, where not 0: the bound of every pipeline wait; CTA 0 never loads its
  // first queries, so that one must run out.
  unsigned long long wait_limit_ns;
};

// Keys of a table row of `pages` entries.
__host__ __device__ __forceinline__ int wide_len(int len, int pages) {
  const long long most = (long long)pages * kPage;
  return len < 0 ? 0 : (int)(len < most ? len : most);
}

// Tiles of `len` keys.
__host__ __device__ __forceinline__ int wide_tiles(int len) {
  return (int)(((unsigned)len + kWideKeys - 1) / kWideKeys);
}
// Places of a block with t > 0 tiles of own keys, and back.
__host__ __device__ __forceinline__ long long wide_own_span(long long t) {
  return t + t / kOwnSlow + kWideCost;
}
__host__ __device__ __forceinline__ int wide_own_tiles(int span) {
  return span - kWideCost - (span - kWideCost) / (kOwnSlow + 1);
}
// Places of a request with `len` keys.
__host__ __device__ __forceinline__ int wide_places(int len, int own_blocks) {
  const int t = wide_tiles(len);
  return t > 0 ? own_blocks * (int)wide_own_span(t) : 0;
}
// Places of the requests' own keys when every table row is full: no plan has more.
__host__ __device__ __forceinline__ long long wide_own_most(int R, int own_blocks, int max_pages) {
  return (long long)R * own_blocks * wide_own_span(cdiv((long long)max_pages * kPage, kWideKeys));
}

// A plan serves when its words are places of the shape and hold every tile of the lengths at
// hand: it may be one of other lengths. Each thread of wide_kernel looks at words of its
// own; where any finds a flaw, the lengths are laid out anew (wide_places), so that no plan
// loses keys or leads out of the tables, rows and slots. Word 0, the place where the line
// begins, is 0 where the plan serves and kPlanAnew (or no place at all) where it does not: the
// merge goes by it.
enum : int { kPlanNone = 1, kPlanShort = 2 };       // no plan of the shape; too few tiles
constexpr int kPlanAnew = -1;
__device__ __forceinline__ int wide_ends_flaw(int begin, int end, int own_most) {
  return (begin == 0 || begin == kPlanAnew) && end >= 0 && end <= own_most ? 0 : kPlanNone;
}
// Of a request with `len` keys and places [first, end).
__device__ __forceinline__ int wide_flaw(int first, int end, int len, int own_blocks,
                                         int own_tiles) {
  if ((unsigned)end - (unsigned)first == (unsigned)wide_places(len, own_blocks)) return 0;
  if (first < 0 || end < first) return kPlanNone;
  const int span = (int)((unsigned)(end - first) / (unsigned)own_blocks);
  if (span * own_blocks != end - first) return kPlanNone;
  if (span == 0) return kPlanShort;
  if (span <= kWideCost) return kPlanNone;
  const int tiles = wide_own_tiles(span);
  if (wide_own_span(tiles) != span || tiles > own_tiles) return kPlanNone;
  return tiles < wide_tiles(len) ? kPlanShort : 0;
}

// The whole line, and how it is cut. Places fit 31 bits (the host checks).
struct WideLine {
  int prefix_len, prefix_tiles, prefix_places, places;
  int used;                        // parts: no more than there are places
  __device__ __forceinline__ WideLine(int prefix_len_, int own_places, int prefix_pages, int blocks,
                                      int units) {
    prefix_len = wide_len(prefix_len_, prefix_pages);
    prefix_tiles = (int)cdiv(prefix_len, kWideKeys);
    prefix_places = prefix_tiles > 0 ? blocks * (prefix_tiles + kWideCost) : 0;
    places = prefix_places + own_places;
    used = places < units ? places : units;
  }
  __device__ __forceinline__ int part(int unit) const {
    return unit < used ? (int)((long long)unit * places / used) : places;
  }
  __device__ __forceinline__ int unit_of(int place) const {
    return (int)(((place + 1LL) * used - 1) / places);
  }
};

// What one part does with one segment.
struct WidePiece {
  const int32_t* table;
  int row0, row_end;               // first row; rows from row_end on are others'
  int slot;
  int len, tile, count;            // keys, first tile, tiles
};

// The pieces of part `unit`, in order, from a plan that serves (word 0 is 0) and the lengths
// ([R] each, the plan with its end) and the prefix's length as the caller holds them.
struct WideWalk {
  const WideArgs& a;
  const int32_t* plan;
  const int32_t* lens;
  int prefix_len, prefix_tiles, prefix_places;
  int pos, end, unit, r = 0;
  __device__ WideWalk(const WideArgs& a_, const int32_t* plan_, const int32_t* lens_,
                      int prefix_len_, int unit_)
      : a(a_), plan(plan_), lens(lens_), unit(unit_) {
    const WideLine line(prefix_len_, plan_[a_.R], a_.prefix_pages, a_.blocks, a_.units);
    prefix_len = line.prefix_len;
    prefix_tiles = line.prefix_tiles;
    prefix_places = line.prefix_places;
    pos = line.part(unit);
    end = line.part(unit + 1);
    const int at = pos - prefix_places;
    for (int step = 1 << 30; step; step >>= 1)       // the last request that begins at or before
      if (r + step < a.R && plan[r + step] <= at) r += step;
  }
  __device__ bool next(WidePiece& p) {
    while (pos < end) {
      int first, tiles, after, segment;              // first place, tiles, places after them
      if (pos < prefix_places) {
        tiles = prefix_tiles;
        after = kWideCost;
        segment = (int)((unsigned)pos / (unsigned)(tiles + kWideCost));
        first = segment * (tiles + kWideCost);
        p.table = a.prefix_table;
        p.len = prefix_len;
        p.row0 = segment * kWideRows;
        p.row_end = (int)a.N;
      } else {
        const int at = pos - prefix_places;
        while (r + 1 < a.R && plan[r + 1] <= at) ++r;
        const int span = (int)((unsigned)(plan[r + 1] - plan[r]) / (unsigned)a.own_blocks);
        const int j = (int)((unsigned)(at - plan[r]) / (unsigned)span);
        tiles = wide_own_tiles(span);
        after = span - tiles;
        segment = a.blocks + r * a.own_blocks + j;
        first = prefix_places + plan[r] + j * span;
        p.table = a.block_table + (long long)r * a.max_pages;
        p.len = lens[r];
        p.row0 = r * a.M + j * kWideRows;
        p.row_end = (r + 1) * a.M;
      }
      const int last = first + tiles, stop = end < last ? end : last, from = pos;
      pos = stop < last ? stop : last + after;
      if (from >= last) continue;                    // the places after the tiles
      p.tile = from - first;
      p.count = stop - from;
      p.slot = (unit + segment) * kWideRows;
      return true;
    }
    return false;
  }
};

cudaError_t launch_wide(const WideArgs& a, const uint8_t* q, const uint8_t* kv, cudaStream_t st);

}  // namespace mlafold
