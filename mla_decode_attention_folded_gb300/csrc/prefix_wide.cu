// The shared prefix's keys against every row of the batch (prefix.cu joins the
// result with the requests' own keys): N = R*k*H query rows, one set of keys.
//
// Bound by the FP8 tensor pipe: 2 * 1088 FLOP per (row, key) beside 576 bytes
// per key. What sets the shape is TMEM: a 512-dim FP32 accumulator of 128 rows
// fills an SM's 512 columns, and MMAs of fewer than 128 columns run at half
// the rate. A pair of CTAs (tcgen05 cta_group::2) therefore shares a block of
// 128 rows and splits the 512 value dims:
//
//   S^T[256 keys, 128 rows]  = K[256, 576] . Q[128, 576]^T    18 MMAs, M = 256, N = 128
//   O^T[512 dims, 128 rows] += V^T[512, 256] . P^T[256, 128]  2 x 16 MMAs, M = 256, N = 128
//
// CTA c computes S for keys 128 c .. 128 c + 127 of a 256-key tile (its TMEM
// lanes) and O for value dims 256 c .. 256 c + 255: 256 columns of O beside two
// S buffers of 128. Both operands of the second product are in place: a KV
// stage holds the CTA's own 128 keys for S (four 128-dim bands and the rope);
// once S is done its two bands of the other CTA's dims are overwritten with
// the other CTA's keys of its own dims, so the slots (i, key half) of V lie at
// the same offsets in both CTAs, as the pair's MMA wants. P^T is split by
// rows: CTA c holds rows 64 c .. 64 c + 63 for all 256 keys, each CTA writing
// its keys' half of the rows into the other's shared memory.
//
// P enters the product as an E4M3 and an E5M2 term: p16 = fp16(p), hi =
// e4m3(p16), lo = e5m2(p16 - hi). E5M2's range keeps the second term where hi
// is subnormal (p < 2^-6, absolute step 2^-9), so hi + lo is p to 2^-7 relative
// down to 2^-13 of absolute error. The running max is lazy as in decode_tc.cu
// (moved when a score exceeds it by more than 8, to 2 below the new one) and
// agreed between the CTAs of a pair, whose scores share accumulators: P is
// computed and written as if no row moved, and each warp's vote goes to the PV
// issuer; where a row did move that says so instead of issuing, and the softmax
// takes the tile back and writes its P again with new maxima.
//
// Work: the tiles of all row blocks, block after block, are one sequence cut
// into equal parts, one per pair; a part's piece of a block goes to partial
// slot unit + block. No plan: the cuts follow from the prefix's length.
#include "decode_common.cuh"
#include "internal.h"
#include "prefix.h"
#include "ptx.cuh"
#include "tc.cuh"

namespace mlafold {
namespace {

using dec::kChunkBytes;      // 128 keys x 128 dims
using dec::kRopeBytes;       // 128 keys x 64 dims
using dec::kStageBytes;

constexpr int kRows = kWideRows;              // query rows per block: the MMA's N
constexpr int kKeys = kWideKeys;              // keys per tile, half of them per CTA
// Five warpgroups: two TMA warps and two for S and PV (rank 0) or the relays (rank
// 1); four of softmax warps. Registers move to the softmax (32 row sums and 16
// words of codes a thread) from the first: the launch's 5 x 96 a thread go 64 +
// 4 x 104.
constexpr int kSoft = 512;                    // softmax threads: a key and 32 rows each
constexpr int kSoftWarps = kSoft / 32;
constexpr int kThreads = 128 + kSoft;
constexpr int kRegsIssue = 64, kRegsSoft = 104;
static_assert(kRegsIssue + 4 * kRegsSoft <= 5 * (65536 / kThreads / 8 * 8), "register pool");
constexpr int kQChunk = 64 * 128;             // this CTA's 64 rows x 128 dims
constexpr int kQBytes = 64 * kDqk;
constexpr int kPRow = 128;                    // a key's 64 hi codes, then its 64 lo codes
constexpr int kPBytes = kKeys * kPRow;
constexpr int kOffQ = 2 * kStageBytes;
constexpr int kOffP = kOffQ + kQBytes;
constexpr int kOffStage = kOffP + kPBytes;    // P of keys 64 .. 127 on its way to the other CTA
constexpr int kOffCtl = kOffStage + 64 * kPRow;
static_assert(64 * kPRow <= kRopeBytes, "the first 64 keys' P waits in the rope's place");
constexpr uint32_t kTmemCols = 512;
constexpr int kSCol = 256;                    // S buffers after O's two blocks of 128 columns
constexpr unsigned long long kTimeoutNs = 2000000000ull;
constexpr uint32_t kIdescS = tc::idesc_e4m3_f32(256, kRows, false, false);
constexpr uint32_t kIdescHi = tc::idesc_e4m3_f32(256, kRows, true, true);
constexpr uint32_t kIdescLo = kIdescHi | (1u << 10);      // B in E5M2
static_assert(kOffQ % 1024 == 0 && kOffP % 1024 == 0, "swizzle atoms need 1 KB alignment");

struct WideCtl {
  uint64_t k_full[2];      // rank 0: TMA of both CTAs -> S: both CTAs' keys landed
  uint64_t v_full[2];      // TMA -> PV, relay: the other CTA's keys of the own dims landed
  uint64_t s_full[2];      // MMA -> softmax, TMA: S of a tile done
  uint64_t p_own;          // rank 0: softmax -> PV: P of CTA 0's keys written or under way
  uint64_t p_in;           // bulk copies of the other CTA -> PV, relay: P of its keys landed
  uint64_t v_peer[2];      // rank 0: V complete in rank 1
  uint64_t p_peer[2];      // rank 0: P of CTA 0's keys complete in rank 1; its
                           // softmax: P of CTA 1's keys written or under way
  uint64_t pv_half[2];     // MMA -> softmax of rank 0, TMA: O holds CTA 0's keys of the tile
  uint64_t pv_done[2];     // MMA -> softmax, TMA: O holds the tile; P and the stage are free
  uint64_t q_full;         // rank 0: TMA of both CTAs -> S
  uint64_t q_empty;        // MMA -> TMA
  uint64_t votes[2];       // rank 0: softmax of rank 1 -> PV: its votes are in vote[1]
  uint64_t sync;           // softmax among themselves (a bounded barrier)
  uint64_t pair[4];        // the two warps that send a quarter's P to the other CTA
  uint64_t swap_bar[2];    // the other CTA's row values are in swap
  uint64_t drain[2];
  uint32_t vote[2][2];     // rank 0: whether CTA i saw a row move, for two votes
  uint32_t moved;          // how many tiles PV sent back
  uint32_t tmem_base;
  int abort_flag;
  alignas(16) float neg_max[kRows]; // minus the running row max (base-2 scores), read four at a time
  alignas(16) float vec[kRows];     // rescale factors, then 1 / l
  float red[4][kRows];
  float swap[2][kRows];
};
static_assert(offsetof(WideCtl, neg_max) % 16 == 0, "16-byte reads");
constexpr int kSmemBytes = kOffCtl + (int)sizeof(WideCtl) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

__device__ __forceinline__ bool w_wait(uint64_t* bar, uint32_t parity, WideCtl* ctl,
                                       int32_t* status) {
  if (tc::mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = tc::globaltimer_ns();
  while (true) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    if (*reinterpret_cast<volatile int*>(&ctl->abort_flag)) return false;
    if (tc::globaltimer_ns() - t0 > kTimeoutNs) {
      *reinterpret_cast<volatile int*>(&ctl->abort_flag) = 1;
      if (status) atomicOr(status, MLA_FAULT_WAIT_TIMEOUT);
      return false;
    }
  }
}
__device__ __forceinline__ uint32_t peek(const uint32_t* p) {
  return *reinterpret_cast<const volatile uint32_t*>(p);
}

// ---------------------------------------------------------------- loads
// The page ids of a tile, in lanes 0-3 of a warp: asked for a tile ahead, checked
// when used.
struct Pages {
  const WideArgs& a;
  int tile, tiles, all, lane;                      // tile: within its block, the next one to ask for
  int next;
  bool report;
  __device__ Pages(const WideArgs& a_, const WidePart& w, bool report_)
      : a(a_), tile((int)(w.begin % w.tiles)), tiles(w.tiles), all((int)cdiv(w.len, kPage)),
        lane(threadIdx.x & 31), report(report_) {
    next = ask();
  }
  __device__ int ask() {
    const int p = tile * (kKeys / kPage) + lane;
    if (++tile == tiles) tile = 0;
    return lane < kKeys / kPage && p < all ? a.prefix_table[p] : -2;      // -2: no such page
  }
  __device__ int take(bool more) {
    int cur = next;
    next = more ? ask() : -2;
    if (cur != -2 && (cur < 0 || cur >= a.num_pages)) {
      if (report && a.status) atomicOr(a.status, MLA_FAULT_PAGE_RANGE);
      cur = -1;
    }
    return cur;
  }
};

// Own keys (and Q at each block's start), counted on rank 0's barriers. A
// stage's bands 0-1 hold V of CTA 0's keys, which PV is done with first, bands
// 2-3 that of CTA 1's; the rope's place holds P on its way until the end.
__device__ void load_keys(const WideArgs& a, const WidePart& w, uint8_t* smem, WideCtl* ctl,
                          uint32_t rank, const CUtensorMap* tm_kv, const CUtensorMap* tm_kvr,
                          const CUtensorMap* tm_q, const CUtensorMap* tm_qr) {
  const int lane = threadIdx.x & 31;
  const long long n = w.end - w.begin;
  Pages pages(a, w, true);
  int block = (int)(w.begin / w.tiles), tile = (int)(w.begin % w.tiles);
  const uint32_t q_bar = tc::map_rank(&ctl->q_full, 0);
  uint32_t x = 0;                                  // blocks whose Q was requested
  bool ok = true;
  for (long long i = 0; ok && i < n; ++i) {
    const int st = i & 1;
    const uint32_t ph = (uint32_t)((i >> 1) - 1) & 1;
    const int cur = pages.take(i + 1 < n);
    const int p0 = __shfl_sync(0xffffffffu, cur, 2 * rank);
    const int p1 = __shfl_sync(0xffffffffu, cur, 2 * rank + 1);
    if (lane == 0) {
      const uint32_t bar = tc::map_rank(&ctl->k_full[st], 0);
      uint8_t* stage = smem + st * kStageBytes;
      if (i >= 2) ok = w_wait(&ctl->pv_half[st], ph, ctl, a.status);
      if (ok) {
        tc::remote_arrive_expect_tx(bar, ((p0 >= 0) + (p1 >= 0)) * dec::kPageBytes);
        for (int h = 0; h < 2; ++h)
          for (int c = 0; c < 2; ++c)
            if ((h ? p1 : p0) >= 0)
              tc::tma_load_2d_pair(stage + c * kChunkBytes + h * (kChunkBytes / 2), tm_kv, bar,
                                   c * 128, (h ? p1 : p0) * kPage);
      }
      if (ok && (i == 0 || tile == 0)) {           // a new block
        if (x > 0) ok = w_wait(&ctl->q_empty, (x - 1) & 1, ctl, a.status);
        if (ok) {
          uint8_t* q = smem + kOffQ;
          const int row = block * kRows + (int)rank * 64;
          tc::remote_arrive_expect_tx(q_bar, kQBytes);
          for (int c = 0; c < 4; ++c)
            tc::tma_load_2d_pair(q + c * kQChunk, tm_q, q_bar, c * 128, row);
          tc::tma_load_2d_pair(q + 4 * kQChunk, tm_qr, q_bar, 512, row);
        }
        ++block;
        ++x;
      }
      if (ok && i >= 2) ok = w_wait(&ctl->pv_done[st], ph, ctl, a.status);
      if (ok) {
        for (int h = 0; h < 2; ++h) {
          const int id = h ? p1 : p0;
          if (id < 0) continue;
          for (int c = 2; c < 4; ++c)
            tc::tma_load_2d_pair(stage + c * kChunkBytes + h * (kChunkBytes / 2), tm_kv, bar,
                                 c * 128, id * kPage);
          tc::tma_load_2d_pair(stage + 4 * kChunkBytes + h * (kRopeBytes / 2), tm_kvr, bar, 512,
                               id * kPage);
        }
      }
    }
    if (++tile == w.tiles) tile = 0;
    ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
  }
}

// The other CTA's keys of the own value dims, over the bands S is done with.
__device__ void load_values(const WideArgs& a, const WidePart& w, uint8_t* smem, WideCtl* ctl,
                            uint32_t rank, const CUtensorMap* tm_kv) {
  const int lane = threadIdx.x & 31;
  const long long n = w.end - w.begin;
  const uint32_t other = 1 - rank;
  Pages pages(a, w, false);
  bool ok = true;
  for (long long i = 0; ok && i < n; ++i) {
    const int st = i & 1;
    const int cur = pages.take(i + 1 < n);
    const int p0 = __shfl_sync(0xffffffffu, cur, 2 * other);
    const int p1 = __shfl_sync(0xffffffffu, cur, 2 * other + 1);
    if (lane == 0 && (ok = w_wait(&ctl->s_full[st], (uint32_t)(i >> 1) & 1, ctl, a.status))) {
      uint8_t* stage = smem + st * kStageBytes;
      tc::mbar_arrive_expect_tx(&ctl->v_full[st], ((p0 >= 0) + (p1 >= 0)) * 2 * kPage * 128);
      for (int h = 0; h < 2; ++h)
        for (int d = 0; d < 2; ++d)
          if ((h ? p1 : p0) >= 0)
            tc::tma_load_2d(stage + (2 * other + d) * kChunkBytes + h * (kChunkBytes / 2), tm_kv,
                            &ctl->v_full[st], (2 * rank + d) * 128, (h ? p1 : p0) * kPage);
    }
    ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
  }
}

// Rank 1 tells rank 0's PV issuer what is complete here: V of each tile, and P of
// CTA 0's keys each time it is written (twice for a tile that PV sent back; the
// last tile's PV ends it).
__device__ void relay_values(const WideArgs& a, const WidePart& w, WideCtl* ctl) {
  for (long long i = 0; i < w.end - w.begin; ++i) {
    if (!w_wait(&ctl->v_full[i & 1], (uint32_t)(i >> 1) & 1, ctl, a.status)) return;
    tc::remote_arrive(tc::map_rank(&ctl->v_peer[i & 1], 0));
  }
}
__device__ void relay_p(const WideArgs& a, const WidePart& w, WideCtl* ctl) {
  const long long n = w.end - w.begin, last = n - 1;
  const uint32_t to = tc::map_rank(&ctl->p_peer[0], 0);
  for (long long k = 0;; ++k) {
    tc::mbar_arrive_expect_tx(&ctl->p_in, 128 * kPRow);
    const unsigned long long t0 = tc::globaltimer_ns();
    while (!tc::mbar_try_wait(&ctl->p_in, (uint32_t)k & 1)) {
      // Every tile's last write has been told of: its PV ends this.
      if (k - peek(&ctl->moved) >= n && tc::mbar_test_wait(&ctl->pv_done[last & 1], (uint32_t)(last >> 1) & 1)) return;
      const bool expired = tc::globaltimer_ns() - t0 > kTimeoutNs;
      if (*reinterpret_cast<volatile int*>(&ctl->abort_flag) || expired) {
        *reinterpret_cast<volatile int*>(&ctl->abort_flag) = 1;
        if (expired && a.status) atomicOr(a.status, MLA_FAULT_WAIT_TIMEOUT);
        return;
      }
    }
    tc::remote_arrive(to);
  }
}

// ---------------------------------------------------------------- MMAs (rank 0)
// S and PV are issued by a thread each: neither waits on the other's inputs.
__device__ __forceinline__ void mma_drain(uint64_t* bar) {
  tc::mma_commit_pair(bar);                        // every MMA done before TMEM is released
  const unsigned long long t0 = tc::globaltimer_ns();
  while (!tc::mbar_try_wait(bar, 0) && tc::globaltimer_ns() - t0 < kTimeoutNs) {
  }
}

__device__ void issue_s(const WideArgs& a, const WidePart& w, uint8_t* smem, WideCtl* ctl,
                        uint32_t tmem) {
  const uint32_t s_kv = tc::smem_u32(smem), s_q = tc::smem_u32(smem + kOffQ);
  const long long n = w.end - w.begin;
  int tile = (int)(w.begin % w.tiles);
  uint32_t x = 0;
  for (long long i = 0; i < n; ++i) {
    const int st = i & 1;
    if (i == 0 || tile == 0) {                     // a new block: its Q in both CTAs
      if (!w_wait(&ctl->q_full, x & 1, ctl, a.status)) break;
      ++x;
    }
    // The S buffer of tile i - 2 is free: its stage was refilled after its PV,
    // whose P the softmax wrote after it had read that S.
    if (!w_wait(&ctl->k_full[st], (uint32_t)(i >> 1) & 1, ctl, a.status)) break;
    tc::fence_after_sync();
    const uint32_t kv = s_kv + st * kStageBytes, d = tmem + kSCol + st * kRows;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        tc::mma_f8_pair(d, tc::smem_desc(kv + c * kChunkBytes + kk * 32, 16, 1024, tc::kSw128),
                        tc::smem_desc(s_q + c * kQChunk + kk * 32, 16, 1024, tc::kSw128), kIdescS,
                        (c | kk) != 0);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
      tc::mma_f8_pair(d, tc::smem_desc(kv + 4 * kChunkBytes + kk * 32, 16, 512, tc::kSw64),
                      tc::smem_desc(s_q + 4 * kQChunk + kk * 32, 16, 512, tc::kSw64), kIdescS, true);
    tc::mma_commit_pair(&ctl->s_full[st]);
    if (++tile == w.tiles) tile = 0;
    if (tile == 0) tc::mma_commit_pair(&ctl->q_empty);
  }
  mma_drain(&ctl->drain[0]);
}

__device__ void issue_pv(const WideArgs& a, const WidePart& w, uint8_t* smem, WideCtl* ctl,
                         uint32_t tmem) {
  const uint32_t s_kv = tc::smem_u32(smem), s_p = tc::smem_u32(smem + kOffP);
  const long long n = w.end - w.begin;
  int tile = (int)(w.begin % w.tiles);
  bool first = true;                               // the pair's first tile of the block
  uint32_t votes = 0, ps = 0;                      // votes before this tile, writes of P
  bool ok = true;
  for (long long i = 0; ok && i < n; ++i) {
    const int st = i & 1;
    const uint32_t ph = (uint32_t)(i >> 1) & 1;
    tc::mbar_arrive_expect_tx(&ctl->p_in, 128 * kPRow);
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      ok = ok && w_wait(bar, parity, ctl, a.status);
    };
    auto half = [&](int kh, bool fresh) {
      tc::fence_after_sync();
      const uint32_t kv = s_kv + st * kStageBytes;
#pragma unroll
      for (int d = 0; d < 2; ++d)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint64_t va = tc::smem_desc(kv + (kh * 2 + d) * kChunkBytes + kk * 32 * 128,
                                            kChunkBytes, 1024, tc::kSw128);
          const uint32_t pk = s_p + (kh * 128 + kk * 32) * kPRow;
          tc::mma_f8_pair(tmem + d * kRows, va, tc::smem_desc(pk, kPBytes, 1024, tc::kSw128), kIdescHi,
                          !(fresh && kk == 0));
          tc::mma_f8_pair(tmem + d * kRows, va, tc::smem_desc(pk + 64, kPBytes, 1024, tc::kSw128),
                          kIdescLo, true);
        }
    };
    // P of CTA 0's keys and V for it, in both CTAs. The first half waits for CTA
    // 1's softmax too (and with it the second half's P) where that touches what
    // the half writes or reads: O (read out before a block's first tile, scaled
    // where the maxima moved) or V (keys past a block's end are cleared).
    bool both = first || tile == w.tiles - 1;
    wait(&ctl->p_own, ps & 1);
    if (!first) wait(&ctl->votes[votes & 1], (votes >> 1) & 1);
    if (!first && ok) {
      const int b = votes++ & 1;
      if (peek(&ctl->vote[0][b]) | peek(&ctl->vote[1][b])) {
        // A row moved: that P is void, another follows.
        wait(&ctl->p_peer[0], ps & 1);
        wait(&ctl->p_peer[1], ps & 1);
        wait(&ctl->p_in, ps & 1);
        if (!ok) break;
        ++ps;
        tc::mbar_arrive_expect_tx(&ctl->p_in, 128 * kPRow);
        for (int c = 0; c < 2; ++c) *reinterpret_cast<volatile uint32_t*>(&ctl->vote[c][b]) = 0;
        const uint32_t count = peek(&ctl->moved) + 1;
        tc::remote_st(tc::map_rank(&ctl->moved, 1), count);
        *reinterpret_cast<volatile uint32_t*>(&ctl->moved) = count;
        wait(&ctl->p_own, ps & 1);
        both = true;
      }
    }
    wait(&ctl->p_peer[0], ps & 1);
    wait(&ctl->v_peer[st], ph);
    if (both) wait(&ctl->p_peer[1], ps & 1);
    if (!ok) break;
    half(0, first);
    tc::mma_commit_pair(&ctl->pv_half[st]);
    wait(&ctl->v_full[st], ph);
    wait(&ctl->p_in, ps & 1);
    if (!both) wait(&ctl->p_peer[1], ps & 1);
    if (!ok) break;
    half(1, false);
    tc::mma_commit_pair(&ctl->pv_done[st]);
    ++ps;
    if (++tile == w.tiles) tile = 0;
    first = tile == 0;
  }
  mma_drain(&ctl->drain[1]);
}

// ---------------------------------------------------------------- softmax
// Every wait here is bounded, barriers among the softmax warps included: a
// thread whose wait runs out leaves, and the others' next one ends by the abort
// flag.
struct Soft {
  const WideArgs& a;
  WideCtl* ctl;
  uint32_t tmem, rank;
  int quarter, part, lane, gt;                     // rows 32 part .. 32 part + 31
  uint32_t swaps = 0, votes = 0, syncs = 0, sends = 0, moves = 0;
  bool ok = true;                                  // warp-uniform

  __device__ Soft(const WideArgs& a_, WideCtl* c, uint32_t t, uint32_t r)
      : a(a_), ctl(c), tmem(t), rank(r) {
    const int warp = threadIdx.x >> 5;
    quarter = warp & 3;
    gt = threadIdx.x - 128;
    part = gt >> 7;
    lane = threadIdx.x & 31;
  }
  __device__ uint32_t lanes() const { return (uint32_t)(quarter * 32) << 16; }
  __device__ void wait(uint64_t* bar, uint32_t parity) {
    const bool got = ok && w_wait(bar, parity, ctl, a.status);
    ok = __all_sync(0xffffffffu, got);
  }
  // Barrier of `warps` warps on `bar`, its `count`-th use.
  __device__ void meet(uint64_t* bar, uint32_t count) {
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bar);
    wait(bar, count & 1);
  }
  __device__ void sync() { meet(&ctl->sync, syncs++); }
  // Row value `v` of threads gt < 128 (row gt) to the other CTA; returns its value.
  __device__ float swap(float v) {
    const int b = swaps & 1;
    const uint32_t ph = (swaps >> 1) & 1;
    ++swaps;
    float got = v;
    if (gt < kRows) {
      if (gt == 0) tc::mbar_arrive_expect_tx(&ctl->swap_bar[b], kRows * 4);
      tc::remote_st_async(tc::map_rank(&ctl->swap[b][gt], 1 - rank), __float_as_uint(v),
                          tc::map_rank(&ctl->swap_bar[b], 1 - rank));
      wait(&ctl->swap_bar[b], ph);
      got = *reinterpret_cast<volatile float*>(&ctl->swap[b][gt]);
    }
    return got;
  }
  static __device__ __forceinline__ float at_most_9(float d) {    // NaN stays
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(d), "f"(9.f));
    return r;
  }
  static __device__ __forceinline__ uint16_t f16x2_to_e5m2x2(uint32_t h) {
    uint16_t r;
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
    return r;
  }
  // The weights of two rows of this thread's key.
  __device__ __forceinline__ void pair(uint64_t raw, uint64_t neg_max, bool valid, float& most,
                                       float& p0, float& p1) const {
    float d0, d1;
    unpack_f32x2(fma_f32x2(raw, pack_f32x2(a.bmm1_log2, a.bmm1_log2), neg_max), d0, d1);
    most = fmaxf(most, fmaxf(d0, d1));
    p0 = valid ? ex2(at_most_9(d0)) : 0.f;
    p1 = valid ? ex2(at_most_9(d1)) : 0.f;
  }
  // P of the tile: codes of this thread's key in its 32 rows; lp gathers the row
  // sums. Returns the largest score above its row's max; more than 9 count as 9
  // (more than 8 has the tile done again).
  __device__ float weigh(int st, bool valid, uint64_t (&lp)[16], uint32_t (&hi)[8],
                         uint32_t (&lo)[8]) const {
    float most = -INFINITY;
    const ulonglong2* m4 = reinterpret_cast<const ulonglong2*>(&ctl->neg_max[part * 32]);
#pragma unroll
    for (int c = 0; c < 32; c += 16) {
      uint32_t raw[16];
      tc::tmem_ld16(tmem + lanes() + kSCol + st * kRows + part * 32 + c, raw);
      tc::tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        const int i = c + e;
        const ulonglong2 m = m4[i / 4];
        float p[4];
        pair(pack_f32x2(__uint_as_float(raw[e]), __uint_as_float(raw[e + 1])), m.x, valid, most, p[0],
             p[1]);
        pair(pack_f32x2(__uint_as_float(raw[e + 2]), __uint_as_float(raw[e + 3])), m.y, valid, most, p[2],
             p[3]);
        lp[i / 2] = add_f32x2(lp[i / 2], pack_f32x2(p[0], p[1]));
        lp[i / 2 + 1] = add_f32x2(lp[i / 2 + 1], pack_f32x2(p[2], p[3]));
        const uint32_t h01 = dec::f32x2_to_f16x2(p[0], p[1]), h23 = dec::f32x2_to_f16x2(p[2], p[3]);
        const uint16_t e01 = dec::f16x2_to_e4m3x2(h01), e23 = dec::f16x2_to_e4m3x2(h23);
        const uint16_t l01 = f16x2_to_e5m2x2(dec::f16x2_sub(h01, e4m3x2_to_f16x2(e01)));
        const uint16_t l23 = f16x2_to_e5m2x2(dec::f16x2_sub(h23, e4m3x2_to_f16x2(e23)));
        hi[i / 4] = (uint32_t)e01 | ((uint32_t)e23 << 16);
        lo[i / 4] = (uint32_t)l01 | ((uint32_t)l23 << 16);
      }
    }
    return valid ? most : -INFINITY;
  }
  // Takes back what weigh added (the same values bit for bit).
  __device__ void unweigh(int st, bool valid, uint64_t (&lp)[16]) const {
    uint32_t raw[32];
    tc::tmem_ld32(tmem + lanes() + kSCol + st * kRows + part * 32, raw);
    tc::tmem_wait_ld();
    const uint64_t* m2 = reinterpret_cast<const uint64_t*>(&ctl->neg_max[part * 32]);
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      float most = 0.f, p0, p1;
      pair(pack_f32x2(__uint_as_float(raw[i]), __uint_as_float(raw[i + 1])), m2[i / 2], valid, most, p0,
           p1);
      lp[i / 2] = add_f32x2(lp[i / 2], pack_f32x2(-p0, -p1));
    }
  }
  // Rows whose max grew by more than 8: the new max, 2 below the tile's, agreed
  // with the other CTA; row sums and O follow. `last`: the pair's previous tile
  // if O holds something of this block, else -1.
  __device__ void move(int st, bool valid, uint64_t (&lp)[16], long long last) {
    {
      uint32_t raw[32];
      float v[32];
      tc::tmem_ld32(tmem + lanes() + kSCol + st * kRows + part * 32, raw);
      tc::tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 32; ++i)
        v[i] = valid ? __uint_as_float(raw[i]) * a.bmm1_log2 : -INFINITY;
      dec::transpose_reduce32<true>(v, lane);
      ctl->red[quarter][part * 32 + lane] = v[0];
    }
    sync();
    if (gt < kRows) {
      const float own = fmaxf(fmaxf(ctl->red[0][gt], ctl->red[1][gt]),
                              fmaxf(ctl->red[2][gt], ctl->red[3][gt]));
      const float tm = fmaxf(own, swap(own));
      const float mo = -ctl->neg_max[gt];
      const float mn = tm > mo + 8.f ? tm - dec::kMaxLead : mo;
      ctl->vec[gt] = mo == -INFINITY ? 0.f : ex2(mo - mn);
      ctl->neg_max[gt] = -mn;
    } else {
      ++swaps;
    }
    sync();
#pragma unroll
    for (int i = 0; i < 16; ++i)
      lp[i] = fma_f32x2(lp[i], *reinterpret_cast<const uint64_t*>(&ctl->vec[part * 32 + 2 * i]),
                        pack_f32x2(0.f, 0.f));
    if (last >= 0) {
      wait(&ctl->pv_done[last & 1], (uint32_t)(last >> 1) & 1);
      tc::fence_after_sync();
#pragma unroll 1
      for (int d = 0; d < 2; ++d) {                // the two blocks of dims
        uint32_t raw[32];
        const uint32_t at = tmem + lanes() + d * kRows + part * 32;
        tc::tmem_ld32(at, raw);
        tc::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e)
          raw[e] = __float_as_uint(__uint_as_float(raw[e]) * ctl->vec[part * 32 + e]);
        tc::tmem_st32(at, raw);
      }
      tc::tmem_wait_st();
    }
  }
  // The codes of this thread's key to their place; rows for the other CTA by way
  // of `put`, from which the two warps that hold a key's 64 rows send them.
  __device__ void write_p(uint8_t* put, int key, bool away, const uint32_t (&hi)[8],
                          const uint32_t (&lo)[8]) const {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int at = (part & 1) * 2 + j;
      *reinterpret_cast<uint4*>(put + ((at ^ (key & 7)) << 4)) =
          make_uint4(hi[4 * j], hi[4 * j + 1], hi[4 * j + 2], hi[4 * j + 3]);
      *reinterpret_cast<uint4*>(put + (((4 + at) ^ (key & 7)) << 4)) =
          make_uint4(lo[4 * j], lo[4 * j + 1], lo[4 * j + 2], lo[4 * j + 3]);
    }
  }
  __device__ void send_p(const uint8_t* put, const uint8_t* place, bool away) {
    tc::fence_proxy_async_smem();
    tc::fence_before_sync();
    if (away) {
      meet(&ctl->pair[quarter], sends++);
      if (lane == 0 && (part & 1) == 0 && ok)
        tc::bulk_copy_to(tc::map_rank(place, 1 - rank), put, 32 * kPRow,
                         tc::map_rank(&ctl->p_in, 1 - rank));
    }
    __syncwarp();
    if (lane == 0) {
      if (rank == 0)
        tc::mbar_arrive(&ctl->p_own);
      else
        tc::remote_arrive(tc::map_rank(&ctl->p_peer[1], 0));
    }
  }
  // This warp's vote on a tile, to the PV issuer: CTA 0's go with its P.
  __device__ void cast(bool moved) {
    const bool any = __any_sync(0xffffffffu, moved);
    if (lane == 0) {
      uint32_t* word = &ctl->vote[rank][votes & 1];
      if (rank == 0) {
        if (any) *reinterpret_cast<volatile uint32_t*>(word) = 1;
      } else {
        if (any) {
          tc::remote_st(tc::map_rank(word, 0), 1);
          tc::fence_cluster();
        }
        tc::remote_arrive(tc::map_rank(&ctl->votes[votes & 1], 0));
      }
    }
    ++votes;
  }
  // Waits until PV of the previous tile is done with `bar`'s part, or has sent the
  // tile back (true) instead of beginning.
  __device__ bool moved_or(uint64_t* bar, uint32_t parity) {
    bool back = false;
    if (ok) {
      const unsigned long long t0 = tc::globaltimer_ns();
      while (!tc::mbar_try_wait(bar, parity)) {
        if (peek(&ctl->moved) != moves) {
          back = true;
          break;
        }
        const bool expired = tc::globaltimer_ns() - t0 > kTimeoutNs;
        if (*reinterpret_cast<volatile int*>(&ctl->abort_flag) || expired) {
          *reinterpret_cast<volatile int*>(&ctl->abort_flag) = 1;
          if (expired && a.status) atomicOr(a.status, MLA_FAULT_WAIT_TIMEOUT);
          ok = false;
          break;
        }
      }
    }
    ok = __all_sync(0xffffffffu, ok);
    back = __any_sync(0xffffffffu, back);
    moves += back ? 1 : 0;
    return back;
  }
};

__device__ void softmax(const WideArgs& a, const WidePart& w, uint8_t* smem, WideCtl* ctl,
                        uint32_t tmem, uint32_t rank) {
  Soft s(a, ctl, tmem, rank);
  const int tl = s.quarter * 32 + s.lane;          // key of this CTA's half tile / dim of a block
  const long long n = w.end - w.begin;
  int block = (int)(w.begin / w.tiles), first_tile = (int)(w.begin % w.tiles);
  uint64_t lp[16];                                 // this key's share of its rows' sums, in pairs
  // Where this key's rows go, the P half of CTA part / 2: rows of 128 bytes in
  // 16-byte pieces, piece j of key k at j ^ (k & 7). Rows for the other CTA wait
  // here for a bulk copy: 64 keys in the stage's rope slot, which S is done with,
  // 64 behind P; both are free again once PV of the tile is done.
  const int key = (int)rank * 128 + tl;
  const bool away = (s.part >> 1) != (int)rank;
  uint8_t* const place = smem + kOffP + key * kPRow;
  auto put_at = [&](int st) {
    return !away ? place
                 : smem + (tl < 64 ? st * kStageBytes + 4 * kChunkBytes + tl * kPRow
                                   : kOffStage + (tl - 64) * kPRow);
  };
  uint32_t hi[8], lo[8];
  uint32_t ps = 0;                                 // writes of P before this tile's
  // Tile g's P again, with new maxima, agreed after both CTAs' first copies of it
  // have landed (they wait for p_in before they exchange row maxima).
  auto again = [&](long long g, bool valid) {
    s.unweigh(g & 1, valid, lp);
    s.wait(&ctl->p_in, (ps - 1) & 1);
    s.sync();                                      // everyone has read the old maxima
    s.move(g & 1, valid, lp, g - 1);
    s.weigh(g & 1, valid, lp, hi, lo);
    uint8_t* put = put_at(g & 1);
    s.write_p(put, key, away, hi, lo);
    s.send_p(put, place, away);
    ++ps;
  };
  long long g = 0;
  while (g < n) {
    const int nt = (int)min((long long)(w.tiles - first_tile), n - g);
    s.sync();                                      // the previous block's readers are done
    if (s.gt < kRows) ctl->neg_max[s.gt] = INFINITY;
#pragma unroll
    for (int i = 0; i < 16; ++i) lp[i] = 0;
    s.sync();
    bool valid = true;
    for (int t = 0; t < nt; ++t, ++g) {
      const int st = g & 1;
      const uint32_t ph = (uint32_t)(g >> 1) & 1;
      const int key0 = (first_tile + t) * kKeys;
      valid = key0 + key < w.len;
      s.wait(&ctl->s_full[st], ph);
      if (!s.ok) return;
      tc::fence_after_sync();
      if (t == 0) {
        s.move(st, valid, lp, -1);
        s.weigh(st, valid, lp, hi, lo);
      } else {
        s.cast(s.weigh(st, valid, lp, hi, lo) > 8.f);
        // The place of P of these keys is free once PV of the previous tile is
        // done with it; if that tile came back it is done again first. (The votes on
        // this one were then cast on maxima that only grew since: at worst it comes
        // back for nothing.)
        uint64_t* bar = rank == 0 ? &ctl->pv_half[(g - 1) & 1] : &ctl->pv_done[(g - 1) & 1];
        const uint32_t bph = (uint32_t)((g - 1) >> 1) & 1;
        if (s.moved_or(bar, bph)) {
          s.unweigh(st, valid, lp);
          again(g - 1, true);
          s.weigh(st, valid, lp, hi, lo);
          s.wait(bar, bph);
        }
      }
      if (t == 0 && g > 0)
        s.wait(rank == 0 ? &ctl->pv_half[(g - 1) & 1] : &ctl->pv_done[(g - 1) & 1],
               (uint32_t)((g - 1) >> 1) & 1);
      if (!s.ok) return;
      uint8_t* put = put_at(st);
      s.write_p(put, key, away, hi, lo);
      // Keys past the end: their V must be finite (0), a slot of each part.
      if (key0 + kKeys > w.len) {
        s.wait(&ctl->v_full[st], ph);
        if (key0 + (s.part >> 1) * 128 + tl >= w.len) {
          uint4* v =
              reinterpret_cast<uint4*>(smem + st * kStageBytes + s.part * kChunkBytes + tl * 128);
#pragma unroll
          for (int u = 0; u < 8; ++u) v[u] = make_uint4(0, 0, 0, 0);
        }
      }
      s.send_p(put, place, away);
      ++ps;
    }
    const int last = (int)((g - 1) & 1);
    const uint32_t last_ph = (uint32_t)((g - 1) >> 1) & 1;
    if (s.moved_or(&ctl->pv_done[last], last_ph)) {
      again(g - 1, valid);
      s.wait(&ctl->pv_done[last], last_ph);
    }
    // Row sums over both CTAs' keys, 1 / l and the LSE, then this CTA's dims.
    {
      float v[32];
#pragma unroll
      for (int i = 0; i < 16; ++i) unpack_f32x2(lp[i], v[2 * i], v[2 * i + 1]);
      dec::transpose_reduce32<false>(v, s.lane);
      ctl->red[s.quarter][s.part * 32 + s.lane] = v[0];
    }
    s.sync();
    const size_t slot = (size_t)(w.unit + block) * kRows;
    const int rows = (int)min((long long)kRows, a.N - (long long)block * kRows);
    if (s.gt < kRows) {
      const float own = ctl->red[0][s.gt] + ctl->red[1][s.gt] + ctl->red[2][s.gt] + ctl->red[3][s.gt];
      const float l = own + s.swap(own);
      ctl->vec[s.gt] = l > 0.f ? 1.f / l : 0.f;
      if (rank == 0 && s.gt < rows)
        a.part_lse[slot + s.gt] = l == 0.f ? -INFINITY : __log2f(l) - ctl->neg_max[s.gt];
    } else {
      ++s.swaps;
    }
    s.sync();
    if (!s.ok) return;
    tc::fence_after_sync();
#pragma unroll 1
    for (int d = 0; d < 2; ++d) {                  // the two blocks of dims
      uint32_t raw[32];
      tc::tmem_ld32(tmem + s.lanes() + d * kRows + s.part * 32, raw);
      tc::tmem_wait_ld();
      float* dst = a.part_o + (slot + s.part * 32) * kDv + rank * 256 + d * 128 + tl;
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (s.part * 32 + e < rows)
          dst[(size_t)e * kDv] = __uint_as_float(raw[e]) * ctl->vec[s.part * 32 + e];
    }
    tc::fence_before_sync();
    ++block;
    first_tile = 0;
  }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
wide_kernel(const WideArgs a, const __grid_constant__ CUtensorMap tm_kv,
            const __grid_constant__ CUtensorMap tm_kvr, const __grid_constant__ CUtensorMap tm_q,
            const __grid_constant__ CUtensorMap tm_qr) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  WideCtl* ctl = reinterpret_cast<WideCtl*>(smem + kOffCtl);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = tc::cluster_rank();
  if (threadIdx.x == 0) {
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&ctl->k_full[b], 2);
      tc::mbar_init(&ctl->v_full[b], 1);
      tc::mbar_init(&ctl->s_full[b], 1);
      tc::mbar_init(&ctl->pv_half[b], 1);
      tc::mbar_init(&ctl->pv_done[b], 1);
      tc::mbar_init(&ctl->v_peer[b], 1);
      tc::mbar_init(&ctl->votes[b], kSoftWarps);
      tc::mbar_init(&ctl->swap_bar[b], 1);
      tc::mbar_init(&ctl->drain[b], 1);
      ctl->vote[0][b] = ctl->vote[1][b] = 0;
    }
    ctl->moved = 0;
    tc::mbar_init(&ctl->sync, kSoftWarps);
    for (int q = 0; q < 4; ++q) tc::mbar_init(&ctl->pair[q], 2);
    tc::mbar_init(&ctl->p_own, kSoftWarps);
    tc::mbar_init(&ctl->p_in, 1);
    tc::mbar_init(&ctl->p_peer[0], 1);
    tc::mbar_init(&ctl->p_peer[1], kSoftWarps);
    tc::mbar_init(&ctl->q_full, 2);
    tc::mbar_init(&ctl->q_empty, 1);
    ctl->abort_flag = 0;
    tc::fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tc::prefetch_tmap(&tm_kv);
    tc::prefetch_tmap(&tm_kvr);
    tc::prefetch_tmap(&tm_q);
    tc::prefetch_tmap(&tm_qr);
  }
  if (warp == 1) {
    tc::tmem_alloc_pair(&ctl->tmem_base, kTmemCols);
    tc::tmem_relinquish_pair();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();      // both CTAs' barriers and TMEM are there
  tc::fence_after_sync();
  const uint32_t tmem = ctl->tmem_base;

  grid_dep_wait();
  grid_dep_launch();
  const WidePart w = wide_part(a, (int)(blockIdx.x >> 1), threadIdx.x == 0);
  if (w.begin == w.end) {
    // No tiles for this pair.
  } else if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == 0) {
      load_keys(a, w, smem, ctl, rank, &tm_kv, &tm_kvr, &tm_q, &tm_qr);
    } else if (warp == 3) {
      load_values(a, w, smem, ctl, rank, &tm_kv);
    } else if (lane == 0) {
      if (rank == 0 && warp == 1)
        issue_s(a, w, smem, ctl, tmem);
      else if (rank == 0)
        issue_pv(a, w, smem, ctl, tmem);
      else if (warp == 1)
        relay_values(a, w, ctl);
      else
        relay_p(a, w, ctl);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    softmax(a, w, smem, ctl, tmem, rank);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (ctl->abort_flag)     // a wait ran out: what is still in flight here or to the other CTA lands
    for (const unsigned long long t0 = tc::globaltimer_ns(); tc::globaltimer_ns() - t0 < 1000000;) {
    }
  tc::cluster_sync();      // no CTA leaves while the other's MMAs or stores may reach it
  tc::fence_after_sync();
  if (warp == 1) tc::tmem_dealloc_pair(tmem, kTmemCols);
}

}  // namespace

cudaError_t launch_wide(const WideArgs& a, const uint8_t* q, const uint8_t* kv, cudaStream_t st) {
  CUtensorMap tkv, tkvr, tq, tqr;
  const cuuint64_t kv_dims[2] = {(cuuint64_t)kDqk, (cuuint64_t)a.num_pages * kPage};
  const cuuint64_t q_dims[2] = {(cuuint64_t)kDqk, (cuuint64_t)a.N};
  const cuuint64_t str[1] = {(cuuint64_t)kDqk};
  const cuuint32_t box[2] = {128, 64}, boxr[2] = {64, 64};     // a page's keys, or 64 query rows
  if (!dec::encode(&tkv, kv, 2, kv_dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !dec::encode(&tkvr, kv, 2, kv_dims, str, boxr, CU_TENSOR_MAP_SWIZZLE_64B) ||
      !dec::encode(&tq, q, 2, q_dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !dec::encode(&tqr, q, 2, q_dims, str, boxr, CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  static bool attr_set[64] = {};
  cudaError_t e = dec::set_smem(wide_kernel, kSmemBytes, attr_set);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * a.units));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, wide_kernel, a, tkv, tkvr, tq, tqr);
}

}  // namespace mlafold
