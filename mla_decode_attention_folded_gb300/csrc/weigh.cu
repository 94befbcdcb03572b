// Attention weight per cached key, summed over a decode step's query rows.
//
//   w[r][j] = decay w[r][j] + sum over the request's M rows of 2^(x[m][j] - lse[r][m]),
//   x[m][j] = bmm1 log2(e) q[r][m] . kv[page(r, j)][j % 64]
//
// The LSEs come from the decode, so one pass over the keys is enough: 128 keys are the MMA's
// M and a block of query rows its N, the 576 dims its K (18 FP8 MMAs), and a thread that owns
// a key reads the key's scores from its TMEM lane, takes their exponentials and adds them up
// in FP32 without a shuffle. Rows beyond a block follow as further blocks over the same tiles
// (from L2, a few tiles at a time), in order: no atomics, the same sums every time.
//
// Up to 128 rows (HBM-bound: 576 B a key) a CTA works alone, its block all rows. With more the
// FP8 tensor pipe is the bound, and a CTA alone would need its tiles twice as often as L2 can
// bring them: a pair of CTAs (cta_group::2) takes 256 keys, 128 in each, and blocks of up to 256 rows,
// half of them in each CTA's shared memory. All tiles of the batch are one line, cut into equal
// runs, one per CTA or pair: keys need no joining, so a cut costs nothing.
//
// Measured (graph replays; in brackets with L2 flushed before each call): 64 requests of up to 8k keys, 56
// rows, 30.8 us (39.7), 5.2 TB/s; 16 of 16k to 64k, 256 rows, 73 us (82), 5.2 TB/s and 2,610 TFLOP/s; 128 of
// up to 4k, 448 rows, 67 us (75), 2,270 TFLOP/s of FP8; two short ones 5.3 us (6.6). What is left at many rows is the pipe's wait for keys and
// queries at the change of a block: shared memory has room for two tiles beside the queries.
// Dropped: tiles in bands of 128 dims, refilled as they are multiplied (69.6 -> 76.7 us), the queries
// in bands (68.7 -> 67.7, but two short requests 5.7 -> 5.9).
#include <cmath>

#include "checks.h"
#include "decode_common.cuh"
#include "formats.cuh"
#include "internal.h"
#include "pair.cuh"
#include "ptx.cuh"
#include "tc.cuh"

namespace mlafold {
namespace {

constexpr int kTile = 128;                       // keys of a CTA's tile: its M
constexpr int kMine = 128;                       // rows in a CTA's shared memory, at most
constexpr int kStages = 2;                       // tiles in flight
constexpr int kChunk = kTile * 128, kStageBytes = kTile * kDqk;
constexpr int kOffQ = kStages * kStageBytes;
constexpr int kMostRun = 16;                     // ... at most: their page ids are a lane's each
constexpr int kSum = 256;                        // summing threads: two per key
constexpr int kThreads = 64 + kSum;
constexpr uint32_t kTmemCols = 512;
constexpr unsigned long long kWaitLimitNs = 2000000000ull;   // 2 s

template <bool PAIR>
struct Cfg {
  static constexpr int kCtas = PAIR ? 2 : 1;
  static constexpr int kMaxRows = kCtas * kMine;     // rows of a block: the MMA's N
  static constexpr int kBufs = kTmemCols / kMaxRows; // score buffers in TMEM
  // Tiles that a row block goes over, single CTAs': at least (256 rows: groups of 2 78 us, of 6 74).
  static constexpr int kRun = PAIR ? 6 : 8;
};
// MMAs wait on the first CTA's barriers of a pair, and arrive on both CTAs'.
struct WeighCtl {
  uint64_t kv_full[kStages], kv_empty[kStages];
  uint64_t q_full, q_empty;
  uint64_t s_full[4], s_empty[4];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  int first_r, first_tile;                       // where this unit's run begins
  long long total;                               // tiles of the batch
};
// Behind the tiles: the queries, then the sums of a group's tiles (what the queries leave of
// their place is the sums'), -lse of a block's rows in two buffers, the barriers.
template <bool PAIR>
constexpr int off_neg() { return kOffQ + kMine * kDqk + Cfg<PAIR>::kRun * 2 * kTile * 4; }
template <bool PAIR>
constexpr int off_ctl() { return off_neg<PAIR>() + 2 * Cfg<PAIR>::kMaxRows * 4; }
template <bool PAIR>
constexpr int smem_bytes() { return off_ctl<PAIR>() + (int)sizeof(WeighCtl) + 1024; }
static_assert(smem_bytes<false>() <= 227 * 1024 && smem_bytes<true>() <= 227 * 1024, "shared memory");

struct WeighArgs {
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* starts;
  const int32_t* rope_starts;    // may be null: starts
  const float* lse;              // [R][M]
  float* weights;                // [R][max_pages 64]
  int32_t* positions;            // may be null
  int32_t* status;
  float scale_log2, decay;
  int R, M, max_pages, num_pages;
  int rows, blocks;              // rows per block, blocks per request
  int run;                       // tiles of a group, at most
  unsigned long long wait_limit_ns;
  int withhold;                  // failure-detection test: CTA 0 never loads its first tile
};

__device__ __forceinline__ bool wg_wait(uint64_t* bar, uint32_t parity, WeighCtl* ctl,
                                        const WeighArgs& a) {
  // Reading the timer takes longer than most waits: not before the barrier was tried for a while.
#pragma unroll 1
  for (int i = 0; i < 32; ++i)
    if (tc::mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = tc::globaltimer_ns();
  while (true) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    if (*reinterpret_cast<volatile int*>(&ctl->abort_flag)) return false;
    if (tc::globaltimer_ns() - t0 > a.wait_limit_ns) {
      *reinterpret_cast<volatile int*>(&ctl->abort_flag) = 1;
      if (a.status) atomicOr(a.status, MLA_FAULT_WAIT_TIMEOUT);
      return false;
    }
  }
}
// One lane of a whole warp, always the same.
__device__ __forceinline__ bool elect() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}
// The keys of request r that are weighed.
__device__ __forceinline__ int weigh_len(const WeighArgs& a, int r) {
  const long long n = a.starts[r] < 0 ? 0 : a.seq_lens[r], most = (long long)a.max_pages * kPage;
  return (int)(n < 0 ? 0 : n < most ? n : most);
}
// A unit's tiles (of KEYS keys) as groups: up to a.run tiles of one request. The row blocks go
// over a group's tiles in turn, forwards and backwards, so that the last block of a group is
// the first of the next and its queries stay.
template <int KEYS>
struct Walk {
  int r, tile, tiles, len;       // request, its next tile, tiles of the group, its keys
  long long left;                // tiles of the unit's run from here on
  bool before, after, back;      // the request has a group before, after; blocks go backwards
  __device__ __forceinline__ bool next(const WeighArgs& a) {
    tile += tiles;
    left -= tiles;
    if (left <= 0) return false;
    before = tiles > 0;
    back = before && !back;
    while (tile >= (int)cdiv(len, KEYS)) {
      tile = 0;
      before = back = false;
      if (++r >= a.R) return false;
      len = weigh_len(a, r);
    }
    const long long rest = cdiv(len, KEYS) - tile;
    tiles = (int)min(min(rest, left), (long long)a.run);
    after = tiles < rest && tiles < left;
    return true;
  }
  __device__ __forceinline__ int block(const WeighArgs& a, int i) const { return back ? a.blocks - 1 - i : i; }
  // Whether the i-th block's queries are there already, and whether they stay.
  __device__ __forceinline__ bool has_q(int i) const { return i == 0 && before; }
  __device__ __forceinline__ bool keeps_q(const WeighArgs& a, int i) const { return i == a.blocks - 1 && after; }
};

template <bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
weigh_kernel(const WeighArgs a, const __grid_constant__ CUtensorMap tm_kv,
             const __grid_constant__ CUtensorMap tm_kvr, const __grid_constant__ CUtensorMap tm_q,
             const __grid_constant__ CUtensorMap tm_qr) {
  using C = Cfg<PAIR>;
  constexpr int kKeys = C::kCtas * kTile;        // keys of a unit's tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  WeighCtl* ctl = reinterpret_cast<WeighCtl*>(smem + off_ctl<PAIR>());
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = PAIR ? (int)tc::cluster_rank() : 0;
  const int unit = PAIR ? blockIdx.x >> 1 : blockIdx.x, units = PAIR ? gridDim.x >> 1 : gridDim.x;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(&ctl->kv_full[i], C::kCtas);
      tc::mbar_init(&ctl->kv_empty[i], 1);
    }
    tc::mbar_init(&ctl->q_full, C::kCtas);
    tc::mbar_init(&ctl->q_empty, 1);
    for (int i = 0; i < C::kBufs; ++i) {
      tc::mbar_init(&ctl->s_full[i], 1);
      tc::mbar_init(&ctl->s_empty[i], C::kCtas * kSum / 32);
    }
    tc::mbar_init(&ctl->drain, 1);
    ctl->abort_flag = 0;
    tc::fence_barrier_init();
    tc::prefetch_tmap(&tm_kv);
    tc::prefetch_tmap(&tm_kvr);
    tc::prefetch_tmap(&tm_q);
    tc::prefetch_tmap(&tm_qr);
  }
  if (warp == 1) {
    if (PAIR) {
      tc::tmem_alloc_pair(&ctl->tmem_base, kTmemCols);
      tc::tmem_relinquish_pair();
    } else {
      tc::tmem_alloc(&ctl->tmem_base, kTmemCols);
      tc::tmem_relinquish();
    }
  }
  grid_dep_wait();
  grid_dep_launch();
  // The line of tiles: warp 0 sums the requests' tiles, 32 at a time, and finds where the
  // run of this unit begins.
  if (warp == 0) {
    const long long v0 = lane < a.R ? cdiv(weigh_len(a, lane), kKeys) : 0;
    long long total = v0;
    for (int r0 = 32; r0 < a.R; r0 += 32)
      total += r0 + lane < a.R ? cdiv(weigh_len(a, r0 + lane), kKeys) : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    const long long begin = cdiv(total * unit, units);
    long long before = 0;
    int fr = a.R, ft = 0;
    for (int r0 = 0; r0 < a.R && fr == a.R; r0 += 32) {
      const long long v = r0 == 0 ? v0 : r0 + lane < a.R ? cdiv(weigh_len(a, r0 + lane), kKeys) : 0;
      long long s = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
      }
      const unsigned m = __ballot_sync(0xffffffffu, before + s > begin);
      if (m) {
        const int l = __ffs(m) - 1;
        fr = r0 + l;
        ft = (int)(begin - before - __shfl_sync(0xffffffffu, s - v, l));
      }
      before += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) {
      ctl->total = total;
      ctl->first_r = fr;
      ctl->first_tile = ft;
    }
  }
  tc::fence_before_sync();
  if (PAIR) tc::cluster_sync();                  // both CTAs' barriers and TMEM are there
  else __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = ctl->tmem_base;
  Walk<kKeys> w;
  w.r = ctl->first_r;
  w.tile = ctl->first_tile;
  w.tiles = 0;
  w.back = false;
  w.left = cdiv(ctl->total * (unit + 1), units) - cdiv(ctl->total * unit, units);
  w.len = w.r < a.R ? weigh_len(a, w.r) : 0;
  const int held = a.rows / C::kCtas, qchunk = held * 128;   // rows in this CTA's shared memory

  if (warp == 0) {
    // Copies: a block's queries, then the group's tiles, block after block.
    uint32_t g = 0, x = 0;
    bool ok = true;
    auto wait0 = [&](uint64_t* bar, uint32_t parity) {
      int v = 1;
      if (lane == 0) v = wg_wait(bar, parity, ctl, a) ? 1 : 0;
      return __shfl_sync(0xffffffffu, v, 0) != 0;
    };
    auto load = [&](void* dst, const CUtensorMap* m, uint64_t* bar, int col, int row) {
      if (PAIR) tc::tma_load_2d_pair(dst, m, tc::map_rank(bar, 0), col, row);
      else tc::tma_load_2d(dst, m, bar, col, row);
    };
    auto expect = [&](uint64_t* bar, uint32_t bytes) {
      if (PAIR) tc::remote_arrive_expect_tx(tc::map_rank(bar, 0), bytes);
      else tc::mbar_arrive_expect_tx(bar, bytes);
    };
    const bool withheld = a.withhold && blockIdx.x == 0;
    while (ok && w.next(a)) {
      // Page ids of the group: lane i has the i-th of this CTA's; one outside the cache is read
      // behind the cache's end, where the copy fills in zeros.
      const int page = (w.tile + (lane >> 1)) * (kKeys / kPage) + rank * 2 + (lane & 1);
      int id = a.num_pages;
      if (lane < 2 * w.tiles && page < (int)cdiv(w.len, kPage)) {
        id = a.block_table[(size_t)w.r * a.max_pages + page];
        if (id < 0 || id >= a.num_pages) {
          if (a.status) atomicOr(a.status, MLA_FAULT_PAGE_RANGE);
          id = a.num_pages;
        }
      }
      for (int i = 0; ok && i < a.blocks; ++i) {
        for (int t = 0; t < w.tiles; ++t, ++g) {
          const int st = g % kStages;
          if (g >= kStages && !(ok = wait0(&ctl->kv_empty[st], (g / kStages - 1) & 1))) break;
          const int p0 = __shfl_sync(0xffffffffu, id, 2 * t), p1 = __shfl_sync(0xffffffffu, id, 2 * t + 1);
          const int key = (w.tile + t) * kKeys + rank * kTile;
          const int pages = key >= w.len ? 0 : key + kPage < w.len ? 2 : 1;
          if (lane == 0 && !(withheld && g == 0)) {
            uint8_t* s = smem + st * kStageBytes;
            expect(&ctl->kv_full[st], pages * kPage * kDqk);
            for (int h = 0; h < pages; ++h) {
              const int row = (h ? p1 : p0) * kPage;
              for (int c = 0; c < 4; ++c)
                load(s + c * kChunk + h * (kChunk / 2), &tm_kv, &ctl->kv_full[st], c * 128, row);
              load(s + 4 * kChunk + h * kPage * 64, &tm_kvr, &ctl->kv_full[st], kDv, row);
            }
          }
          // The queries after the first tile's keys, whose place is free before theirs.
          if (t == 0 && !w.has_q(i)) {
            if (x > 0 && !(ok = wait0(&ctl->q_empty, (x - 1) & 1))) {
              ++g;                               // loaded
              break;
            }
            if (lane == 0) {
              uint8_t* q = smem + kOffQ;
              const int row = w.r * a.M + w.block(a, i) * a.rows + rank * held;
              expect(&ctl->q_full, held * kDqk);
              for (int c = 0; c < 4; ++c) load(q + c * qchunk, &tm_q, &ctl->q_full, c * 128, row);
              load(q + 4 * qchunk, &tm_qr, &ctl->q_full, kDv, row);
            }
            ++x;
          }
        }
      }
    }
    // Never leave with copies in flight: another role may have given up a wait. (The pair's count on
    // the first CTA, and the CTAs leave together.)
    if (lane == 0 && rank == 0) {
      const unsigned long long t0 = tc::globaltimer_ns();
      for (uint32_t i = g < kStages ? 0 : g - kStages; i < g; ++i)
        while (!(withheld && i == 0) && !tc::mbar_try_wait(&ctl->kv_full[i % kStages], (i / kStages) & 1) &&
               tc::globaltimer_ns() - t0 < a.wait_limit_ns) {
        }
      while (x > 0 && !tc::mbar_try_wait(&ctl->q_full, (x - 1) & 1) &&
             tc::globaltimer_ns() - t0 < a.wait_limit_ns) {
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      // The whole warp waits, so that what the MMAs are given stays in uniform registers; one lane
      // issues.
      const bool one = elect();
      bool ok = true;
      uint32_t g = 0, x = 0;
      const uint32_t idesc = tc::idesc_e4m3_f32(kKeys, a.rows, false, false);
      const uint64_t q = tc::smem_desc(tc::smem_u32(smem + kOffQ), 16, 1024, tc::kSw128);
      const uint64_t qr = tc::smem_desc(tc::smem_u32(smem + kOffQ) + 4 * qchunk, 16, 512, tc::kSw64);
      const uint32_t s0 = tc::smem_u32(smem);
      auto wait = [&](uint64_t* bar, uint32_t parity) { return ok = wg_wait(bar, parity, ctl, a); };
      auto mma = [&](uint32_t d, uint64_t k, uint64_t n, bool accumulate) {
        if (PAIR) tc::mma_f8_pair(d, k, n, idesc, accumulate);
        else tc::mma_e4m3(d, k, n, idesc, accumulate);
      };
      auto commit = [&](uint64_t* bar) {
        if (PAIR) tc::mma_commit_pair(bar);
        else tc::mma_commit(bar);
      };
      while (ok && w.next(a)) {
        for (int i = 0; ok && i < a.blocks; ++i) {
          if (!w.has_q(i) && !wait(&ctl->q_full, x++ & 1)) break;
          for (int t = 0; t < w.tiles; ++t, ++g) {
            const int st = g % kStages, bf = g % C::kBufs;
            if (!wait(&ctl->kv_full[st], (g / kStages) & 1)) break;
            if (g >= C::kBufs && !wait(&ctl->s_empty[bf], (g / C::kBufs - 1) & 1)) break;
            tc::fence_after_sync();
            const uint64_t k = tc::smem_desc(s0 + st * kStageBytes, 16, 1024, tc::kSw128);
            const uint64_t kr = tc::smem_desc(s0 + st * kStageBytes + 4 * kChunk, 16, 512, tc::kSw64);
            const uint32_t d = tmem + bf * C::kMaxRows;
            if (one) {
#pragma unroll
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  mma(d, k + ((c * kChunk + kk * 32) >> 4), q + ((c * qchunk + kk * 32) >> 4), c + kk != 0);
#pragma unroll
              for (int kk = 0; kk < 2; ++kk) mma(d, kr + (kk * 32 >> 4), qr + (kk * 32 >> 4), true);
              commit(&ctl->s_full[bf]);
              commit(&ctl->kv_empty[st]);
              if (t == w.tiles - 1 && !w.keeps_q(a, i)) commit(&ctl->q_empty);
            }
          }
        }
        ok = __all_sync(0xffffffffu, ok);
      }
      if (one) {
        commit(&ctl->drain);                       // every MMA done before TMEM is released
        const unsigned long long t0 = tc::globaltimer_ns();
        while (!tc::mbar_try_wait(&ctl->drain, 0) && tc::globaltimer_ns() - t0 < a.wait_limit_ns) {
        }
      }
    }
  } else {
    // Sums: thread (quarter, lane) owns a key, the two groups the two halves of a block's rows.
    // After a wait that ran out the threads go on without waiting, so that all meet at
    // the group's barriers; they write nothing more.
    const int quarter = warp & 3, half = (warp - 2) >> 2, st = tid - 64;
    const int key = quarter * 32 + lane, cols = a.rows / 2;
    float* neg = reinterpret_cast<float*>(smem + off_neg<PAIR>());     // [x & 1][row]
    float* sums = neg - a.run * 2 * kTile;                             // [tile][half][key]
    const uint64_t c2 = pack_f32x2(a.scale_log2, a.scale_log2);
    uint32_t g = 0, x = 0;
    bool ok = true;
    // -lse of a block's row; rows that have none (behind the request's, or with an LSE that is
    // no number) get -inf, so that their weights are 0.
    auto row_neg = [&](int r, int b) {
      const int m = b * a.rows + st;
      if (st >= a.rows || m >= a.M || r >= a.R) return -INFINITY;
      const float l = a.lse[(size_t)r * a.M + m];
      return fabsf(l) < INFINITY ? -l : -INFINITY;
    };
    auto slot_of = [&](int i) { return (w.tile + i / kTile) * kKeys + rank * kTile + i % kTile; };
    constexpr int kOwn = kMostRun * kTile / kSum;  // slots of a group that a thread writes
    while (w.next(a)) {
      float ahead = row_neg(w.r, w.block(a, 0));
      const int new_at = a.starts[w.r];
      float* weights = a.weights + (size_t)w.r * a.max_pages * kPage;
      float old[kOwn];                             // earlier weights, asked for while S is made
#pragma unroll
      for (int u = 0; u < kOwn; ++u) {
        const int i = st + u * kSum, slot = slot_of(i);
        old[u] = i < w.tiles * kTile && slot < w.len && slot < new_at ? weights[slot] : 0.f;
      }
      for (int b = 0; b < a.blocks; ++b, ++x) {    // the b-th of the group
        if (st < C::kMaxRows) neg[(x & 1) * C::kMaxRows + st] = ahead;
        if (b + 1 < a.blocks) ahead = row_neg(w.r, w.block(a, b + 1));
        // (Not bar.sync, which a warp's threads have to reach together.)
        asm volatile("barrier.sync 1, %0;" ::"r"(kSum) : "memory");
        const float* ng = neg + (x & 1) * C::kMaxRows + half * cols;
        for (int t = 0; t < w.tiles; ++t, ++g) {
          const int bf = g % C::kBufs;
          ok = __all_sync(0xffffffffu, wg_wait(&ctl->s_full[bf], (g / C::kBufs) & 1, ctl, a)) && ok;
          tc::fence_after_sync();
          const uint32_t src = tmem + ((uint32_t)(quarter * 32) << 16) + bf * C::kMaxRows + half * cols;
          uint64_t acc[2] = {0, 0};
          // The half's columns 64 at a time (the last time 16, 32, 48 or 64), then read no more.
#pragma unroll 1
          for (int c0 = 0; c0 < cols; c0 += 64) {
            uint32_t raw[4][16];
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (c0 + 16 * c < cols) tc::tmem_ld16(src + c0 + 16 * c, raw[c]);
            tc::tmem_wait_ld();
            if (c0 + 64 >= cols) {
              tc::fence_before_sync();
              __syncwarp();
              if (lane == 0) {
                if (PAIR) tc::remote_arrive(tc::map_rank(&ctl->s_empty[bf], 0));
                else tc::mbar_arrive(&ctl->s_empty[bf]);
              }
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (c0 + 16 * c >= cols) break;
#pragma unroll
              for (int i = 0; i < 16; i += 4) {
                const float4 n4 = *reinterpret_cast<const float4*>(ng + c0 + 16 * c + i);
                float e[4];
                unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(raw[c][i]), __uint_as_float(raw[c][i + 1])),
                                       c2, pack_f32x2(n4.x, n4.y)), e[0], e[1]);
                unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(raw[c][i + 2]), __uint_as_float(raw[c][i + 3])),
                                       c2, pack_f32x2(n4.z, n4.w)), e[2], e[3]);
                // fmaxf: a score that is NaN adds 0.
#pragma unroll
                for (int u = 0; u < 4; ++u) e[u] = fmaxf(ex2(e[u]), 0.f);
                acc[0] = add_f32x2(acc[0], pack_f32x2(e[0], e[1]));
                acc[1] = add_f32x2(acc[1], pack_f32x2(e[2], e[3]));
              }
            }
          }
          float s0, s1;
          unpack_f32x2(add_f32x2(acc[0], acc[1]), s0, s1);
          float* at = sums + (t * 2 + half) * kTile + key;
          *at = (b ? *at : 0.f) + s0 + s1;
        }
      }
      asm volatile("bar.sync 1, %0;" ::"r"(kSum) : "memory");
#pragma unroll
      for (int u = 0; u < kOwn; ++u) {
        const int i = st + u * kSum, slot = slot_of(i);
        if (i >= w.tiles * kTile || slot >= w.len || !ok) continue;
        const float* at = sums + (i / kTile) * 2 * kTile + i % kTile;
        const float s = at[0] + at[kTile];
        weights[slot] = slot < new_at ? old[u] * a.decay + s : s;
        if (a.positions && slot >= new_at)
          a.positions[(size_t)w.r * a.max_pages * kPage + slot] =
              (a.rope_starts ? a.rope_starts[w.r] : new_at) + (slot - new_at);
      }
      asm volatile("barrier.sync 1, %0;" ::"r"(kSum) : "memory");
    }
  }
  tc::fence_before_sync();
  if (PAIR) tc::cluster_sync();    // no CTA leaves while the other's MMAs or arrivals may reach it
  else __syncthreads();
  tc::fence_after_sync();
  if (warp == 1) {
    if (PAIR) tc::tmem_dealloc_pair(tmem, kTmemCols);
    else tc::tmem_dealloc(tmem, kTmemCols);
  }
}

int32_t weigh_impl(const mla_cache_shape* s, const void* q, const void* kv,
                   const int32_t* block_table, const int32_t* seq_lens, const float* lse,
                   float bmm1_scale, float decay, const int32_t* starts, const int32_t* rope_starts,
                   float* weights, int32_t* positions, int32_t* status, mla_stream_t stream,
                   unsigned long long wait_limit_ns, int withhold) {
  if (!s) return MLA_ERR_NULL;
  if (s->page_size != kPage) return MLA_ERR_UNSUPPORTED;
  if (s->R < 1 || s->R > kMaxR || s->k < 1 || s->H < 1 || (long long)s->k * s->H > kMaxM ||
      s->max_pages < 1 || s->max_pages > (1 << 20) || s->num_pages < 1 ||
      s->num_pages >= (1 << 25))
    return MLA_ERR_SHAPE;
  if (!scales_ok(bmm1_scale, 0.f) || !std::isfinite(decay) || decay < 0.f) return MLA_ERR_SHAPE;
  if (!q || !kv || !block_table || !seq_lens || !lse || !starts || !weights) return MLA_ERR_NULL;
  if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(lse, 4) || !aligned(starts, 4) || !aligned(rope_starts, 4) || !aligned(weights, 4) ||
      !aligned(positions, 4) || !aligned(status, 4))
    return MLA_ERR_ALIGN;
  int st = check_device();
  if (st != MLA_OK) return st;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MLA_ERR_CUDA;
  WeighArgs a;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.starts = starts;
  a.rope_starts = rope_starts;
  a.lse = lse;
  a.weights = weights;
  a.positions = positions;
  a.status = status;
  a.scale_log2 = (float)((double)bmm1_scale * 1.4426950408889634);
  a.decay = decay;
  a.R = s->R;
  a.M = s->k * s->H;
  a.max_pages = s->max_pages;
  a.num_pages = s->num_pages;
  // Pairs of CTAs beyond 128 rows (448: 94 us by single CTAs, 67 by pairs; 256: 103 and 74; but 56 rows
  // 30.7 us by single ones, 31.5 by pairs). Blocks of equal size, as few as hold the rows.
  const bool pair = a.M > kMine && sms >= 2;
  const int most_rows = pair ? 2 * kMine : kMine;
  a.blocks = (int)cdiv(a.M, most_rows);
  a.rows = (int)cdiv(cdiv(a.M, a.blocks), 32) * 32;
  // Groups of tiles: without a second block as long as there is room for their sums. With one no longer
  // than L2 keeps for it (76 pairs' groups of 6 are 67 MB; 32 x 7 x 64 on 16k keys: 78.9 us, of 10 83.3,
  // of 3 81.6).
  const int spare = (kMine - a.rows) * kDqk / (2 * kTile * 4), room = Cfg<false>::kRun + spare;
  a.run = pair ? Cfg<true>::kRun : room < kMostRun ? room : kMostRun;
  a.wait_limit_ns = wait_limit_ns;
  a.withhold = withhold;
  CUtensorMap tkv, tkvr, tq, tqr;
  const cuuint32_t held = (cuuint32_t)(pair ? a.rows / 2 : a.rows);
  const cuuint64_t kv_dims[2] = {kDqk, (cuuint64_t)s->num_pages * kPage}, str[1] = {kDqk};
  const cuuint64_t q_dims[2] = {kDqk, (cuuint64_t)s->R * a.M};
  const cuuint32_t box[2] = {128, kPage}, box_r[2] = {64, kPage};
  const cuuint32_t qbox[2] = {128, held}, qbox_r[2] = {64, held};
  if (!dec::encode(&tkv, kv, 2, kv_dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !dec::encode(&tkvr, kv, 2, kv_dims, str, box_r, CU_TENSOR_MAP_SWIZZLE_64B) ||
      !dec::encode(&tq, q, 2, q_dims, str, qbox, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !dec::encode(&tqr, q, 2, q_dims, str, qbox_r, CU_TENSOR_MAP_SWIZZLE_64B))
    return MLA_ERR_CUDA;
  static bool attr_set[2][64] = {};
  auto* kernel = pair ? weigh_kernel<true> : weigh_kernel<false>;
  const int smem = pair ? smem_bytes<true>() : smem_bytes<false>();
  if (dec::set_smem(kernel, smem, attr_set[pair]) != cudaSuccess) return MLA_ERR_CUDA;
  const long long most = (long long)s->R * cdiv((long long)s->max_pages * kPage, pair ? 2 * kTile : kTile);
  const int units = pair ? sms / 2 : sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(most < units ? most : units) * (pair ? 2 : 1));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pair ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a, tkv, tkvr, tq, tqr);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace
}  // namespace mlafold

using namespace mlafold;

extern "C" int32_t mla_kv_weigh(const mla_cache_shape* s, const void* q, const void* kv,
                                const int32_t* block_table, const int32_t* seq_lens,
                                const float* lse, float bmm1_scale, float decay,
                                const int32_t* starts, const int32_t* rope_starts, float* weights,
                                int32_t* positions, int32_t* status, mla_stream_t stream) {
  return weigh_impl(s, q, kv, block_table, seq_lens, lse, bmm1_scale, decay, starts, rope_starts,
                    weights, positions, status, stream, kWaitLimitNs, 0);
}

extern "C" int32_t mla_kv_weigh_wait_test(const mla_cache_shape* s, const void* q, const void* kv,
                                          const int32_t* block_table, const int32_t* seq_lens,
                                          const float* lse, float bmm1_scale, float decay,
                                          const int32_t* starts, const int32_t* rope_starts,
                                          float* weights, int32_t* positions, int32_t* status,
                                          uint64_t wait_limit_ns, mla_stream_t stream) {
  if (!status) return MLA_ERR_NULL;
  if (wait_limit_ns < 1000000ull || wait_limit_ns > kWaitLimitNs) return MLA_ERR_SHAPE;
  return weigh_impl(s, q, kv, block_table, seq_lens, lse, bmm1_scale, decay, starts, rope_starts,
                    weights, positions, status, stream, wait_limit_ns, 1);
}
