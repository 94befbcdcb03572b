// The shared-prefix decode's work: which (rows, keys) tiles there are and how they
// are cut into parts (prefix_wide.cu computes them, prefix.cu plans and joins).
//
// A segment is a block of up to 128 rows with the keys it attends to: block b of
// all N rows with the prefix's keys (segments 0 .. blocks - 1), then block j of
// request r's M rows with the request's own keys (segment blocks + r * own_blocks
// + j). A segment of t > 0 tiles takes t + 1 places of one line of places, one per
// tile and one for what a segment costs besides; segments without keys take none.
// The line is cut into equal parts, part u from floor(u * places / used), one per
// pair of CTAs. The piece of segment s that part u holds has partial slot u + s:
// along the line one of the two grows with every piece, so no two share a slot and
// a segment's slots are consecutive.
#pragma once

#include "internal.h"

namespace mlafold {

constexpr int kWideRows = 128;     // query rows per block
constexpr int kWideKeys = 256;     // keys per tile

struct WideArgs {
  const int32_t* prefix_table;     // [prefix_pages]
  const int32_t* prefix_len;       // [1]
  const int32_t* block_table;      // [R][max_pages]
  const int32_t* seq_lens;         // [R]
  const long long* plan;           // [R + 1]: first place of each request's segments
  float* part_o;                   // [slots][128][512]
  float* part_lse;                 // [slots][128]
  int32_t* status;                 // may be null
  float bmm1_log2;
  long long N;                     // query rows
  int R, M, prefix_pages, max_pages, num_pages, units, blocks, own_blocks;
};

// Keys of a table row of `pages` entries.
__host__ __device__ __forceinline__ int wide_len(int len, int pages) {
  const long long most = (long long)pages * kPage;
  return len < 0 ? 0 : (int)(len < most ? len : most);
}

// The whole line, and how it is cut.
struct WideLine {
  int prefix_len, prefix_tiles;
  long long prefix_places, places;
  long long used;                  // parts: no more than there are places
  __device__ __forceinline__ WideLine(int prefix_len_, long long own_places, int prefix_pages,
                                      int blocks, int units) {
    prefix_len = wide_len(prefix_len_, prefix_pages);
    prefix_tiles = (int)cdiv(prefix_len, kWideKeys);
    prefix_places = prefix_tiles > 0 ? (long long)blocks * (prefix_tiles + 1) : 0;
    places = prefix_places + own_places;
    used = places < units ? places : units;
  }
  __device__ __forceinline__ long long part(long long unit) const {
    return unit < used ? unit * places / used : places;
  }
  __device__ __forceinline__ int unit_of(long long place) const {
    return (int)(((place + 1) * used - 1) / places);
  }
};

// What one part does with one segment.
struct WidePiece {
  const int32_t* table;
  long long row0;                  // first row; rows from row_end on are others'
  long long row_end;
  size_t slot;
  int len, tile, count;            // keys, first tile, tiles
};

// The pieces of part `unit`, in order. `plan` may lie in shared memory.
struct WideWalk {
  const WideArgs& a;
  const long long* plan;
  const WideLine line;
  long long pos, end;
  int unit;
  __device__ WideWalk(const WideArgs& a_, const long long* plan_, int unit_)
      : a(a_), plan(plan_),
        line(*a_.prefix_len, plan_[a_.R], a_.prefix_pages, a_.blocks, a_.units), unit(unit_) {
    pos = line.part(unit);
    end = line.part(unit + 1);
  }
  __device__ bool next(WidePiece& p) {
    while (pos < end) {
      long long first;             // the segment's first place
      int tiles, segment;
      if (pos < line.prefix_places) {
        segment = (int)(pos / (line.prefix_tiles + 1));
        tiles = line.prefix_tiles;
        first = (long long)segment * (tiles + 1);
        p.table = a.prefix_table;
        p.len = line.prefix_len;
        p.row0 = (long long)segment * kWideRows;
        p.row_end = a.N;
      } else {
        const long long at = pos - line.prefix_places;
        int lo = 0, hi = a.R - 1;  // the last request that begins at or before it
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (plan[mid] <= at) lo = mid; else hi = mid - 1;
        }
        const long long span = (plan[lo + 1] - plan[lo]) / a.own_blocks;
        if (span < 2) return false;                  // not a plan of this shape
        const int j = (int)((at - plan[lo]) / span);
        segment = a.blocks + lo * a.own_blocks + j;
        tiles = (int)(span - 1);
        first = line.prefix_places + plan[lo] + j * span;
        p.table = a.block_table + (long long)lo * a.max_pages;
        p.len = wide_len(a.seq_lens[lo], a.max_pages);
        p.row0 = (long long)lo * a.M + (long long)j * kWideRows;
        p.row_end = (long long)(lo + 1) * a.M;
      }
      const long long last = first + tiles, stop = end < last ? end : last;
      const long long from = pos;
      pos = stop < last ? stop : last + 1;
      if (from >= last) continue;                    // the place after the tiles
      p.tile = (int)(from - first);
      p.count = (int)(stop - from);
      p.slot = (size_t)(unit + segment) * kWideRows;
      return true;
    }
    return false;
  }
};

cudaError_t launch_wide(const WideArgs& a, const uint8_t* q, const uint8_t* kv, cudaStream_t st);

}  // namespace mlafold
