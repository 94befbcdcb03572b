// The shared-prefix decode's pieces: how the prefix's tiles are cut into parts
// (prefix_wide.cu computes them, prefix.cu joins them).
#pragma once

#include "internal.h"

namespace mlafold {

constexpr int kWideRows = 128;     // query rows per block
constexpr int kWideKeys = 256;     // keys per tile

struct WideArgs {
  const int32_t* prefix_table;     // [prefix_pages]
  const int32_t* prefix_len;       // [1]
  float* part_o;                   // [units + blocks - 1][128][512]
  float* part_lse;                 // [units + blocks - 1][128]
  int32_t* status;                 // may be null
  float bmm1_log2;
  long long N;                     // query rows
  int prefix_pages, num_pages, units, blocks;
};

// The keys of the prefix, within its table.
__device__ __forceinline__ int wide_len(const int32_t* prefix_len, int prefix_pages,
                                        int32_t* status, bool report) {
  const long long most = (long long)prefix_pages * kPage;
  long long len = max(*prefix_len, 0);
  if (len > most) {
    if (report && status) atomicOr(status, MLA_FAULT_PAGE_RANGE);
    len = most;
  }
  return (int)len;
}

// The tiles of all blocks, block after block, are cut into `used` equal parts
// (no more than there are tiles): part u begins at floor(u * total / used).
struct WidePart {
  int len, tiles;                  // keys, tiles per block
  int unit;
  long long begin, end;            // this part's tiles
};
__device__ __forceinline__ WidePart wide_part(const WideArgs& a, int unit, bool report) {
  WidePart w;
  w.len = wide_len(a.prefix_len, a.prefix_pages, a.status, report);
  w.tiles = (int)cdiv(w.len, kWideKeys);
  w.unit = unit;
  const long long total = (long long)w.tiles * a.blocks;
  const long long used = total < a.units ? total : a.units;
  w.begin = unit < used ? unit * total / used : 0;
  w.end = unit < used ? (unit + 1) * total / used : 0;
  return w;
}
// The part that holds tile f.
__device__ __forceinline__ int wide_unit_of(long long f, long long total, long long used) {
  return (int)(((f + 1) * used - 1) / total);
}

cudaError_t launch_wide(const WideArgs& a, const uint8_t* q, const uint8_t* kv, cudaStream_t st);

}  // namespace mlafold
