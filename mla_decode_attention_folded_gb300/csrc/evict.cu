// Eviction from the paged latent cache by accumulated attention weight.
//
// Of a request's n keys the `keep` first in this order stay: keys held by their
// position (below `sinks`, or among the `recent` newest), then by weight from
// the largest, ties to the lower slot; NaN counts as less than any weight. Attention
// does not depend on the order of its keys, so the keys that stay behind slot
// `keep` move into the slots of dropped ones, the i-th of them into the i-th such
// slot, and nothing else moves: the fewest rows that can be read and written, every
// source behind `keep` and every target before it, so no two copies touch the same row.
//
// Bound by HBM for large evictions (16 B per key, 1,152 B per moved key) and by latency for
// a step's few keys. A cluster per request orders its keys: 32-bit codes that sort as the
// rule does, held in shared memory; the keep-th largest by three digits of histograms, summed
// in the first CTA (12.5 -> 10.2 us against every CTA reading all); places by ordered counts. It
// lists the moves and makes them, 9 threads a row; where the clusters of a batch leave enough SMs
// idle, a second launch makes them on all.
//
// Measured (graph replays; in brackets with L2 flushed before each call): 128 requests drop 7 of 2,055
// keys in 10.3 us (13.4), nearly all of it the select's chain of dependent steps; 8 x 20k to 32k keys to 4k
// in 23.8 us (28.8), 1.5 TB/s of what has to move; 128k keys to 64k in 29.8 us (35.0), 1.35 TB/s: the walks
// over the keys and the scattered rows.
#include <climits>

#include "checks.h"
#include "internal.h"
#include "pair.cuh"
#include "ptx.cuh"

namespace mlafold {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kBins = 2048;                      // 11 + 11 + 10 bits
constexpr int kMaxCluster = 16;
constexpr int kCached = 40960;                   // keys a CTA holds in shared memory (160 KB)
constexpr uint32_t kHeld = 0xFFFFFFFFu;          // above the code of any weight

constexpr int kRowThreads = kDqk / 64;           // threads that copy a row, 64 bytes each

struct EvictArgs {
  uint8_t* kv;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const float* weights;
  const int32_t* positions;      // may be null: a key's position is its slot
  const int32_t* keep;
  float* weights_out;
  int32_t* positions_out;        // null where positions is
  int32_t* lens_out;
  int32_t* moves;                // [R][cap][2]: from, to
  int32_t* count;                // [R]
  int32_t* status;
  long long cap;
  int R, max_pages, num_pages, recent, sinks, cluster, chunk;
  int apart;                     // a second launch makes the moves
};

// One of the 9 threads that move a key: its row, and with part 0 its weight and position.
struct Move {
  int from, to, page_from, page_to;
};
__device__ __forceinline__ Move read_move(const EvictArgs& a, int r, long long m) {
  const int2 mv = reinterpret_cast<const int2*>(a.moves + (size_t)r * a.cap * 2)[m];
  const int32_t* table = a.block_table + (size_t)r * a.max_pages;
  return {mv.x, mv.y, table[mv.x / kPage], table[mv.y / kPage]};
}
__device__ __forceinline__ void make_move(const EvictArgs& a, int r, const Move& mv, int part) {
  const bool ok = mv.page_from >= 0 && mv.page_from < a.num_pages && mv.page_to >= 0 &&
                  mv.page_to < a.num_pages;
  if (ok) {
    const uint4* src =
        reinterpret_cast<const uint4*>(a.kv + ((size_t)mv.page_from * kPage + mv.from % kPage) * kDqk) + part;
    uint4* dst = reinterpret_cast<uint4*>(a.kv + ((size_t)mv.page_to * kPage + mv.to % kPage) * kDqk) + part;
    uint4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = src[u * kRowThreads];
#pragma unroll
    for (int u = 0; u < 4; ++u) dst[u * kRowThreads] = v[u];
  }
  if (part == 0) {
    if (!ok && a.status) atomicOr(a.status, MLA_FAULT_PAGE_RANGE);
    const size_t row = (size_t)r * a.max_pages * kPage;
    const float w = a.weights[row + mv.from];
    a.weights_out[row + mv.to] = w;
    a.weights_out[row + mv.from] = 0.f;
    if (a.positions) {
      const int32_t p = a.positions[row + mv.from];
      a.positions_out[row + mv.to] = p;
      a.positions_out[row + mv.from] = -1;
    }
  }
}

// A code that sorts as the weights do (-0 as 0, NaN lowest), below kHeld.
__device__ __forceinline__ uint32_t weight_code(float w) {
  const uint32_t b = __float_as_uint(w + 0.f);
  if ((b << 1) > 0xFF000000u) return 0u;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ void st_rank(void* p, int rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(tc::map_rank(p, rank)), "r"(v) : "memory");
}

struct Shared {
  uint32_t hist[3][kBins];       // the first CTA's: of the cluster
  unsigned long long sums[kWarps];
  uint32_t digit[3];             // what holds the wanted place, the places left in it, its codes
  int top;                       // newest position of this CTA's keys
  // What the cluster's CTAs tell all: newest positions or equals, holes, movers.
  uint32_t told[3][kMaxCluster];
};

__device__ __forceinline__ void join(int cluster) {
  if (cluster > 1) tc::cluster_sync();
  else __syncthreads();
}

// A value of each of the cluster's CTAs, told to all: thread c tells CTA c. The join is the caller's.
__device__ __forceinline__ void tell(Shared& sh, int what, int rank, int cluster, uint32_t v) {
  if ((int)threadIdx.x < cluster) st_rank(&sh.told[what][rank], threadIdx.x, v);
}
// Exclusive sum over the block's threads; `total` gets the whole.
__device__ __forceinline__ unsigned long long scan(unsigned long long v, unsigned long long* sums,
                                                   unsigned long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) sums[warp] = s;
  __syncthreads();
  if (warp == 0) {
    unsigned long long w = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    sums[lane] = w;
  }
  __syncthreads();
  total = sums[kWarps - 1];
  const unsigned long long before = warp ? sums[warp - 1] : 0;
  __syncthreads();
  return before + s - v;
}

__global__ void __launch_bounds__(kThreads, 1) evict_select_kernel(const EvictArgs a) {
  extern __shared__ uint32_t codes[];            // this CTA's codes, where they fit
  __shared__ Shared sh;
  const int rank = a.cluster > 1 ? (int)tc::cluster_rank() : 0;
  const int r = blockIdx.x / a.cluster, tid = threadIdx.x, lane = tid & 31;
  for (int i = tid; i < 3 * kBins; i += kThreads) sh.hist[i / kBins][i % kBins] = 0;
  if (tid == 0) sh.top = INT_MIN;
  grid_dep_wait();
  grid_dep_launch();
  const int most = a.max_pages * kPage, given = a.seq_lens[r], keep = max(a.keep[r], 0);
  const int n = min(max(given, 0), most);
  if (given > most && a.status && tid == 0 && rank == 0) atomicOr(a.status, MLA_FAULT_PAGE_RANGE);
  const size_t row = (size_t)r * most;
  const float* w = a.weights + row;
  const int32_t* p = a.positions ? a.positions + row : nullptr;
  float* wo = a.weights_out + row;
  int32_t* po = a.positions ? a.positions_out + row : nullptr;
  const bool copies_w = wo != w, copies_p = p && po != p;
  // This CTA's slots, and this thread's among them: runs in order, of odd length, so that the
  // threads' places in shared memory lie in different banks.
  const int each = (int)cdiv(n, a.cluster);
  const int first = min(rank * each, n), len = min(each, n - first);
  const int run = (int)cdiv(len, kThreads) | 1;
  const int b0 = min(tid * run, len), b1 = min(b0 + run, len);

  if (n <= keep) {                               // nothing to drop
#pragma unroll 4
    for (int i = first + tid; i < first + len; i += kThreads) {
      if (copies_w) wo[i] = w[i];
      if (copies_p) po[i] = p[i];
    }
    // seq_lens may be lens_out: what others of the cluster then read instead comes to the same.
    if (rank == 0 && tid == 0) {
      a.count[r] = 0;
      a.lens_out[r] = n;
    }
    return;
  }

  const bool cached = len <= a.chunk;
  long long newest = LLONG_MAX;                  // positions from here on are held
  join(a.cluster);                               // the histograms are cleared, in the first CTA too
  if (a.recent > 0) {
    int top = n - 1;
    if (p) {
      int mine = INT_MIN;
#pragma unroll 8
      for (int i = tid; i < len; i += kThreads) {
        const int pos = p[first + i];
        if (cached) codes[i] = (uint32_t)pos;
        mine = max(mine, pos);
      }
      mine = __reduce_max_sync(0xffffffffu, mine);
      if (lane == 0) atomicMax(&sh.top, mine);
      __syncthreads();
      top = sh.top;
      if (a.cluster > 1) {
        tell(sh, 0, rank, a.cluster, (uint32_t)top);
        tc::cluster_sync();
        for (int c = 0; c < a.cluster; ++c) top = max(top, (int)sh.told[0][c]);
      }
    }
    newest = (long long)top + 1 - a.recent;
  }
  auto make = [&](int i, int pos) {              // the code of this CTA's i-th slot
    return pos < a.sinks || pos >= newest ? kHeld : weight_code(w[first + i]);
  };
  auto code = [&](int i) { return cached ? codes[i] : make(i, p ? p[first + i] : first + i); };

  // The keep-th largest code, digit by digit, and how many of its equals stay.
  uint32_t want = keep, found = 0, same = 0;
  if (keep > 0) {
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      if (pass == 0) {
        // Four slots' loads at a time.
        const bool have = cached && p && a.recent > 0;
        for (int i0 = tid; i0 < len; i0 += 4 * kThreads) {
          float x[4];
          int pos[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * kThreads;
            if (i < len) {
              x[u] = w[first + i];
              pos[u] = !p ? first + i : have ? (int)codes[i] : p[first + i];
            }
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * kThreads;
            if (i < len) {
              const uint32_t c = pos[u] < a.sinks || pos[u] >= newest ? kHeld : weight_code(x[u]);
              if (cached) codes[i] = c;
              atomicAdd(&sh.hist[0][c >> 21], 1u);
            }
          }
        }
      } else {
#pragma unroll 4
        for (int i = tid; i < len; i += kThreads) {
          const uint32_t c = code(i);
          if (c >> (shift + bits) == found >> (shift + bits))
            atomicAdd(&sh.hist[pass][(c >> shift) & ((1 << bits) - 1)], 1u);
        }
      }
      const int hi = kBins - 2 - 2 * tid;        // this thread's two digits: this and the next
      if (a.cluster > 1) {
        __syncthreads();
        // Added in 32 bits, as the first CTA adds its own codes meanwhile: additions of two widths to the
        // same words are not atomic to one another. (In 64, to a second histogram, the times are the same.)
        if (rank > 0) {
#pragma unroll
          for (int u = 0; u < 2; ++u)
            if (const uint32_t v = sh.hist[pass][hi + u])
              asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(
                               tc::map_rank(&sh.hist[pass][hi + u], 0)),
                           "r"(v)
                           : "memory");
        }
      }
      join(a.cluster);
      // Digits from the largest down; the first CTA finds the one and tells the others.
      if (rank == 0) {
        const uint32_t h0 = sh.hist[pass][hi + 1], h1 = sh.hist[pass][hi];
        unsigned long long total;
        const uint32_t above = (uint32_t)scan(h0 + h1, sh.sums, total);
        const bool here = above < want && want <= above + h0 + h1, second = above + h0 < want;
        const uint32_t at[3] = {(uint32_t)(hi + (second ? 0 : 1)), want - above - (second ? h0 : 0),
                                second ? h1 : h0};
        if (a.cluster == 1) {
          if (here) {
#pragma unroll
            for (int u = 0; u < 3; ++u) sh.digit[u] = at[u];
          }
        } else if (const unsigned m = __ballot_sync(0xffffffffu, here)) {
          // Its warp tells the cluster, a CTA each lane (128k keys: 31.0 us by its thread alone, 29.5).
#pragma unroll
          for (int u = 0; u < 3; ++u) {
            const uint32_t v = __shfl_sync(0xffffffffu, at[u], __ffs(m) - 1);
            if (lane == 0) sh.digit[u] = v;
            else if (lane < a.cluster) st_rank(&sh.digit[u], lane, v);
          }
        }
      }
      join(a.cluster);
      found |= sh.digit[0] << shift;
      want = sh.digit[1];
      same = sh.digit[2];
      // (The next digit is told after the next join.)
    }
  } else {
    found = kHeld;                               // no code is larger, and no equal stays
  }

  // Equals stay in the order of their slots; mostly all do.
  unsigned long long total;
  uint32_t eq = 0;
  if (same != want) {
    uint32_t equal = 0;
    for (int i = b0; i < b1; ++i) equal += code(i) == found;
    eq = (uint32_t)scan(equal, sh.sums, total);
    if (a.cluster > 1) {
      tell(sh, 0, rank, a.cluster, (uint32_t)total);
      tc::cluster_sync();
      for (int c = 0; c < rank; ++c) eq += sh.told[0][c];
    }
  }
  // A dropped key's slot before `keep` is a hole; a kept key behind it moves.
  auto walk = [&](auto&& each_slot) {
    uint32_t e = eq;
    for (int i = b0; i < b1; ++i) {
      const uint32_t c = keep > 0 ? code(i) : 0u;
      each_slot(i, c > found || (c == found && e++ < want));
    }
  };
  uint32_t holes = 0, movers = 0;
  walk([&](int i, bool stays) {
    if (first + i < keep) holes += !stays;
    else movers += stays;
  });
  const unsigned long long at = scan((unsigned long long)holes << 32 | movers, sh.sums, total);
  uint32_t hole = (uint32_t)(at >> 32), mover = (uint32_t)at, all = (uint32_t)total;
  if (a.cluster > 1) {
    tell(sh, 1, rank, a.cluster, (uint32_t)(total >> 32));
    tell(sh, 2, rank, a.cluster, (uint32_t)total);
    tc::cluster_sync();
    all = 0;
    for (int c = 0; c < a.cluster; ++c) {
      if (c < rank) {
        hole += sh.told[1][c];
        mover += sh.told[2][c];
      }
      all += sh.told[2][c];
    }
  }
  auto settle = [&](int slot, bool stays) {      // the books of a key that does not move
    if (stays) {
      if (slot >= keep) return;
      if (copies_w) wo[slot] = w[slot];
      if (copies_p) po[slot] = p[slot];
    } else if (slot >= keep) {
      wo[slot] = 0.f;
      if (p) po[slot] = -1;
    }
  };
  int32_t* list = a.moves + (size_t)r * a.cap * 2;
  walk([&](int i, bool stays) {
    const int slot = first + i;
    if (slot < keep && !stays) list[2 * (size_t)hole++ + 1] = slot;
    if (slot >= keep && stays) list[2 * (size_t)mover++] = slot;
    if (cached) codes[i] = stays;
    else settle(slot, stays);
  });
  __syncthreads();
  if (cached)
    for (int i0 = tid; i0 < len; i0 += 4 * kThreads) {   // as settle(), four slots' loads at a time
      float x[4];
      int pos[4];
      bool copies[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * kThreads;
        copies[u] = i < len && codes[i] && first + i < keep;
        if (copies[u] && copies_w) x[u] = w[first + i];
        if (copies[u] && copies_p) pos[u] = p[first + i];
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * kThreads, slot = first + i;
        if (copies[u]) {
          if (copies_w) wo[slot] = x[u];
          if (copies_p) po[slot] = pos[u];
        } else if (i < len && !codes[i] && slot >= keep) {
          wo[slot] = 0.f;
          if (p) po[slot] = -1;
        }
      }
    }
  if (rank == 0 && tid == 0) {
    a.count[r] = (int)all;
    a.lens_out[r] = keep;
  }
  if (a.cluster > 1) tc::cluster_sync();         // the lists are whole; no CTA reads others' any more
  if (a.apart) return;
  const int group = tid / kRowThreads, part = tid % kRowThreads;
  const uint32_t groups = kThreads / kRowThreads * a.cluster;
  uint32_t m = rank * (kThreads / kRowThreads) + group;
  if (group >= kThreads / kRowThreads || m >= all) return;
  // Three moves at a time: one's row, the next one's pages, the list entry of the one after.
  const int2* entry = reinterpret_cast<const int2*>(list);
  const int32_t* table = a.block_table + (size_t)r * a.max_pages;
  auto pages = [&](int2 mv) { return Move{mv.x, mv.y, table[mv.x / kPage], table[mv.y / kPage]}; };
  Move mv = pages(entry[m]);
  int2 after = m + groups < all ? entry[m + groups] : make_int2(0, 0);
  for (; m < all; m += groups) {
    const uint32_t m1 = m + groups, m2 = m1 + groups;
    const Move next = m1 < all ? pages(after) : mv;
    if (m2 < all) after = entry[m2];
    make_move(a, r, mv, part);
    mv = next;
  }
}

// The listed moves of all requests on all SMs.
constexpr int kRows = 28, kMoveThreads = 256;

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a) {
  __shared__ long long before[kMaxR + 1];
  __shared__ long long sums[kMoveThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_wait();
  grid_dep_launch();
  long long base = 0;                            // the moves of the requests before each
  for (int r0 = 0; r0 < a.R; r0 += kMoveThreads) {
    const long long v = r0 + tid < a.R ? a.count[r0 + tid] : 0;
    long long s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    if (lane == 31) sums[warp] = s;
    __syncthreads();
    long long add = base;
    for (int i = 0; i < warp; ++i) add += sums[i];
    if (r0 + tid < a.R) before[r0 + tid] = add + s - v;
    for (int i = 0; i < kMoveThreads / 32; ++i) base += sums[i];
    __syncthreads();
  }
  if (tid == 0) before[a.R] = base;
  __syncthreads();
  const int group = tid / kRowThreads, part = tid % kRowThreads;
  if (group >= kRows) return;
  for (long long m = (long long)blockIdx.x * kRows + group; m < base; m += (long long)gridDim.x * kRows) {
    int lo = 0, hi = a.R;                        // before[lo] <= m < before[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (before[mid] <= m) lo = mid;
      else hi = mid;
    }
    make_move(a, lo, read_move(a, lo, m - before[lo]), part);
  }
}

int check_evict(const mla_cache_shape* s) {
  if (!s) return MLA_ERR_NULL;
  if (s->page_size != kPage) return MLA_ERR_UNSUPPORTED;
  if (s->R < 1 || s->R > kMaxR || s->max_pages < 1 || s->max_pages > (1 << 20) ||
      s->num_pages < 1 || s->num_pages >= (1 << 25))
    return MLA_ERR_SHAPE;
  return MLA_OK;
}
size_t list_bytes(const mla_cache_shape* s) {
  return align256((size_t)s->R * s->max_pages * (kPage / 2) * 8);
}

}  // namespace
}  // namespace mlafold

using namespace mlafold;

extern "C" int32_t mla_kv_evict_workspace_bytes(const mla_cache_shape* s, size_t* bytes) {
  const int st = check_evict(s);
  if (st != MLA_OK) return st;
  if (!bytes) return MLA_ERR_NULL;
  *bytes = list_bytes(s) + align256((size_t)s->R * 4);
  return MLA_OK;
}

extern "C" int32_t mla_kv_evict(const mla_cache_shape* s, void* kv, const int32_t* block_table,
                                const int32_t* seq_lens, const float* weights,
                                const int32_t* positions, const int32_t* keep, int32_t recent,
                                int32_t sinks, float* weights_out, int32_t* positions_out,
                                int32_t* lens_out, void* workspace, size_t workspace_bytes_given,
                                int32_t* status, mla_stream_t stream) {
  int st = check_evict(s);
  if (st != MLA_OK) return st;
  if (recent < 0 || sinks < 0) return MLA_ERR_SHAPE;
  if (!kv || !block_table || !seq_lens || !weights || !keep || !weights_out || !lens_out ||
      !workspace || (positions != nullptr) != (positions_out != nullptr))
    return MLA_ERR_NULL;
  if (!aligned(kv, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(weights, 4) ||
      !aligned(positions, 4) || !aligned(keep, 4) || !aligned(weights_out, 4) ||
      !aligned(positions_out, 4) || !aligned(lens_out, 4) || !aligned(workspace, 256) ||
      !aligned(status, 4))
    return MLA_ERR_ALIGN;
  const size_t lists = list_bytes(s);
  if (workspace_bytes_given < lists + align256((size_t)s->R * 4)) return MLA_ERR_WORKSPACE;
  if ((st = check_device()) != MLA_OK) return st;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MLA_ERR_CUDA;

  EvictArgs a;
  a.kv = static_cast<uint8_t*>(kv);
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.weights = weights;
  a.positions = positions;
  a.keep = keep;
  a.weights_out = weights_out;
  a.positions_out = positions_out;
  a.lens_out = lens_out;
  a.moves = static_cast<int32_t*>(workspace);
  a.count = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + lists);
  a.status = status;
  a.cap = (long long)s->max_pages * (kPage / 2);
  a.R = s->R;
  a.max_pages = s->max_pages;
  a.num_pages = s->num_pages;
  a.recent = recent;
  a.sinks = sinks;
  // CTAs per request: doubled while each has more than 4,096 slots (1 x 8k: 17.8 us on 2, 17.0 on 1;
  // 4 x 32k: 22.6 on 8, 30.7 on 2) and the batch's fit on the SMs, clusters of 8 or 16 on two thirds of
  // them: more of those do not run at a time (16 x 32k: 31.5 us on clusters of 4, 47 on 8; 10 x
  // 20k: 27.8 and 25.6). More where the codes of a table's width would not fit into shared memory.
  const long long slots = (long long)s->max_pages * kPage;
  a.cluster = 1;
  while (a.cluster < kMaxCluster &&
         ((slots > 4096ll * a.cluster && s->R * a.cluster * 2 <= (a.cluster < 4 ? sms : sms * 2 / 3)) ||
          slots > (long long)kCached * a.cluster))
    a.cluster *= 2;
  const long long each = cdiv(slots, a.cluster);
  a.chunk = (int)(each < kCached ? each : kCached);
  static bool attr_set[64] = {};
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    if (cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kCached * 4) != cudaSuccess ||
        cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed,
                             1) != cudaSuccess)
      return MLA_ERR_CUDA;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(s->R * a.cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)a.chunk * 4;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)a.cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.cluster > 1 ? 2 : 1;
  // A second launch makes the moves on all SMs where the clusters leave a third of them idle (128k to
  // 64k: 31 us with it, 60 without; 10 x 20k to 10k: 25.6 and 29.0; on more SMs it only costs: 32 x 16k
  // to 2k 28.1 and 26.3) and the requests may have many (64 x 2,112 slots: 12.9 and 10.4 us).
  a.apart = (long long)s->R * a.cluster * 3 <= sms * 2ll && slots > 2304ll * a.cluster;
  if (cudaLaunchKernelEx(&cfg, evict_select_kernel, a) != cudaSuccess) return MLA_ERR_CUDA;
  if (!a.apart) return MLA_OK;
  // At most half of a request's keys move.
  const long long most = (long long)s->R * a.cap;
  const long long grid = cdiv(most, kRows);
  cfg.gridDim = dim3((unsigned)(grid < 8ll * sms ? grid : 8ll * sms));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_move_kernel, a) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
