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
// computed on the assumption that no row moves, scout warps meanwhile look
// for a row that moves and exchange a flag, and only then is the tile done again
// with new maxima.
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
// Four warpgroups: the TMA warp, the MMA (or relay) warp and two idle ones; four
// scout warps; two groups of softmax warps. The softmax threads hold 64 row
// sums and 32 words of codes: registers move to them from the others (the
// launch's 4 x 128 a thread: 64 + 64 + 2 x 192).
constexpr int kScout = 128;                   // scouts: a key and all 128 rows each
constexpr int kSoft = 256;                    // softmax threads: a key and 64 rows each
constexpr int kThreads = 128 + kScout + kSoft;
constexpr int kRegsIssue = 64, kRegsScout = 64, kRegsSoft = 192;
static_assert(kRegsIssue + kRegsScout + 2 * kRegsSoft <= 4 * (65536 / kThreads), "register pool");
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
  uint64_t k_full[2];      // TMA -> MMA (rank 0), relay (rank 1): own keys landed
  uint64_t k_peer[2];      // rank 0: the other CTA's keys landed
  uint64_t v_full[2];      // TMA -> MMA, relay: the other CTA's keys of the own dims landed
  uint64_t s_full[2];      // MMA -> softmax, scouts, TMA: S of a tile done
  uint64_t p_own;          // softmax -> MMA, relay: P of the own keys written or under way
  uint64_t p_in;           // softmax of the other CTA -> MMA, relay: P of its keys landed
  uint64_t p_peer[2];      // rank 0: P of CTA i's keys (and V for it) complete in rank 1
  uint64_t pv_half[2];     // MMA -> softmax of rank 0, TMA: O holds CTA 0's keys of the tile
  uint64_t pv_done[2];     // MMA -> softmax, TMA: O holds the tile; P and the stage are free
  uint64_t q_full, q_peer, q_empty;
  uint64_t vote_bar[2];    // the other CTA's flag is in vote_peer
  uint64_t told[2];        // scouts -> softmax: verdict
  uint64_t swap_bar[2];    // the other CTA's row values are in swap
  uint64_t drain;
  uint32_t vote_peer[2];
  uint32_t vote[2];        // bits of this CTA's scouts: kMoved, kFailed
  uint32_t verdict[2];     // of the pair's scouts
  uint32_t soft_word[2];   // kFailed of softmax threads; kMoved, kFailed of the verdict
  uint32_t moves;          // how often new maxima came into m_run
  uint32_t tmem_base;
  int abort_flag;
  alignas(16) float m_run[kRows];   // running row max (base-2 scores), read four at a time
  float vec[kRows];        // rescale factors, then 1 / l
  float red[4][kRows];
  float swap[2][kRows];
};
static_assert(offsetof(WideCtl, m_run) % 16 == 0, "float4 reads");
constexpr int kSmemBytes = kOffCtl + (int)sizeof(WideCtl) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");
constexpr uint32_t kMoved = 1, kFailed = 2;

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
__device__ __forceinline__ void soft_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kSoft) : "memory");
}
__device__ __forceinline__ void scout_sync() {
  asm volatile("bar.sync 2, %0;" ::"n"(kScout) : "memory");
}
// Waits, as bounded as w_wait, until the maxima have moved `count` times.
__device__ __forceinline__ bool wait_moves(uint32_t count, WideCtl* ctl, int32_t* status) {
  const unsigned long long t0 = tc::globaltimer_ns();
  while (*reinterpret_cast<volatile uint32_t*>(&ctl->moves) < count) {
    if (*reinterpret_cast<volatile int*>(&ctl->abort_flag)) return false;
    if (tc::globaltimer_ns() - t0 > kTimeoutNs) {
      *reinterpret_cast<volatile int*>(&ctl->abort_flag) = 1;
      if (status) atomicOr(status, MLA_FAULT_WAIT_TIMEOUT);
      return false;
    }
  }
  __threadfence_block();
  return true;
}
__device__ __forceinline__ uint32_t peek(const uint32_t* p) {
  return *reinterpret_cast<const volatile uint32_t*>(p);
}

// ---------------------------------------------------------------- producer
// One warp; lane l < 4 holds the id of page l of a tile. Three kinds of load,
// each issued as soon as what it overwrites is free.
__device__ void producer(const WideArgs& a, const WidePart& w, uint8_t* smem, WideCtl* ctl,
                         uint32_t rank, const CUtensorMap* tm_kv, const CUtensorMap* tm_kvr,
                         const CUtensorMap* tm_q, const CUtensorMap* tm_qr) {
  const int lane = threadIdx.x & 31;
  const long long n = w.end - w.begin;             // tiles of this pair
  const int pages_all = (int)cdiv(w.len, kPage);
  int tile = (int)(w.begin % w.tiles);             // within its block, of the next page_ids()
  int block = (int)(w.begin / w.tiles);            // of the next Q
  auto page_ids = [&]() {                          // lane l: page l of the next tile
    const int p = tile * (kKeys / kPage) + lane;
    if (++tile == w.tiles) tile = 0;
    return lane < kKeys / kPage && p < pages_all ? a.prefix_table[p] : -1;
  };
  // Next tile: own keys' bands 0-1, their bands 2-3 and rope, other keys' values.
  long long nk = 0, nk2 = 0, nv = 0;
  long long q_at = 0, q_step = w.tiles - tile;     // first tile of the next block
  uint32_t x = 0;                                  // blocks whose Q was requested
  int ids[2] = {-1, -1}, next = page_ids();
  unsigned long long t0 = 0;
  bool ok = true;
  while (nv < n) {
    uint32_t can = 0;                              // lane 0 looks, all lanes act
    if (lane == 0) {
      if (q_at <= nk && q_at < n && (x == 0 || tc::mbar_test_wait(&ctl->q_empty, (x - 1) & 1)))
        can |= 1;
      // A stage's bands 0-1 hold V of CTA 0's keys, which PV is done with first;
      // bands 2-3 that of CTA 1's. The rope's place holds P until the end.
      if (nk < n && nk <= nk2 + 1 && nk < nv + 2 &&
          (nk < 2 || tc::mbar_test_wait(&ctl->pv_half[nk & 1], (uint32_t)((nk >> 1) - 1) & 1)))
        can |= 2;
      if (nv < nk2 && tc::mbar_test_wait(&ctl->s_full[nv & 1], (uint32_t)(nv >> 1) & 1)) can |= 4;
      if (nk2 < nk &&
          (nk2 < 2 || tc::mbar_test_wait(&ctl->pv_done[nk2 & 1], (uint32_t)((nk2 >> 1) - 1) & 1)))
        can |= 8;
    }
    can = __shfl_sync(0xffffffffu, can, 0);
    if (can & 1) {
      if (lane == 0) {
        uint8_t* q = smem + kOffQ;
        const int row = block * kRows + (int)rank * 64;
        tc::mbar_arrive_expect_tx(&ctl->q_full, kQBytes);
        for (int c = 0; c < 4; ++c)
          tc::tma_load_2d(q + c * kQChunk, tm_q, &ctl->q_full, c * 128, row);
        tc::tma_load_2d(q + 4 * kQChunk, tm_qr, &ctl->q_full, 512, row);
      }
      q_at += q_step;
      q_step = w.tiles;
      ++block;
      ++x;
    }
    if (can & 8) {
      const int st = nk2 & 1, cur = st ? ids[1] : ids[0];
      const int p0 = __shfl_sync(0xffffffffu, cur, 2 * rank);
      const int p1 = __shfl_sync(0xffffffffu, cur, 2 * rank + 1);
      if (lane == 0) {
        uint8_t* stage = smem + st * kStageBytes;
        for (int h = 0; h < 2; ++h) {
          const int id = h ? p1 : p0;
          if (id < 0) continue;
          for (int c = 2; c < 4; ++c)
            tc::tma_load_2d(stage + c * kChunkBytes + h * (kChunkBytes / 2), tm_kv,
                            &ctl->k_full[st], c * 128, id * kPage);
          tc::tma_load_2d(stage + 4 * kChunkBytes + h * (kRopeBytes / 2), tm_kvr, &ctl->k_full[st],
                          512, id * kPage);
        }
      }
      ++nk2;
    }
    if (can & 4) {
      const int st = nv & 1, cur = st ? ids[1] : ids[0];
      const uint32_t other = 1 - rank;
      const int p0 = __shfl_sync(0xffffffffu, cur, 2 * other);
      const int p1 = __shfl_sync(0xffffffffu, cur, 2 * other + 1);
      if (lane == 0) {
        uint8_t* stage = smem + st * kStageBytes;
        tc::mbar_arrive_expect_tx(&ctl->v_full[st], ((p0 >= 0) + (p1 >= 0)) * 2 * kPage * 128);
        for (int h = 0; h < 2; ++h) {
          const int id = h ? p1 : p0;
          if (id < 0) continue;
          for (int i = 0; i < 2; ++i)              // own dims of the other CTA's keys
            tc::tma_load_2d(stage + (2 * other + i) * kChunkBytes + h * (kChunkBytes / 2), tm_kv,
                            &ctl->v_full[st], (2 * rank + i) * 128, id * kPage);
        }
      }
      ++nv;
    }
    if (can & 2) {
      const int st = nk & 1;
      int cur = next;
      if (cur >= a.num_pages || (cur < 0 && lane < kKeys / kPage &&
                                 ((tile ? tile : w.tiles) - 1) * (kKeys / kPage) + lane < pages_all)) {
        if (a.status) atomicOr(a.status, MLA_FAULT_PAGE_RANGE);
        cur = -1;
      }
      if (st) ids[1] = cur; else ids[0] = cur;
      const int p0 = __shfl_sync(0xffffffffu, cur, 2 * rank);
      const int p1 = __shfl_sync(0xffffffffu, cur, 2 * rank + 1);
      if (lane == 0) {
        uint8_t* stage = smem + st * kStageBytes;
        tc::mbar_arrive_expect_tx(&ctl->k_full[st], ((p0 >= 0) + (p1 >= 0)) * dec::kPageBytes);
        for (int h = 0; h < 2; ++h) {
          const int id = h ? p1 : p0;
          if (id < 0) continue;
          for (int c = 0; c < 2; ++c)
            tc::tma_load_2d(stage + c * kChunkBytes + h * (kChunkBytes / 2), tm_kv,
                            &ctl->k_full[st], c * 128, id * kPage);
        }
      }
      next = nk + 1 < n ? page_ids() : -1;         // in flight until the next tile
      ++nk;
    }
    if (can) {
      t0 = 0;
      continue;
    }
    const unsigned long long now = tc::globaltimer_ns();
    if (t0 == 0) t0 = now;
    bool stop = false;
    if (lane == 0) {
      const bool expired = now - t0 > kTimeoutNs;
      if (expired) {
        *reinterpret_cast<volatile int*>(&ctl->abort_flag) = 1;
        if (a.status) atomicOr(a.status, MLA_FAULT_WAIT_TIMEOUT);
      }
      stop = *reinterpret_cast<volatile int*>(&ctl->abort_flag) != 0;
    }
    if (__shfl_sync(0xffffffffu, (int)stop, 0)) {
      ok = false;
      break;
    }
  }
  if (lane == 0 && !ok) {                          // never leave with copies in flight
    const unsigned long long t1 = tc::globaltimer_ns();
    auto drain = [&](uint64_t* bar, uint32_t parity) {
      while (!tc::mbar_try_wait(bar, parity) && tc::globaltimer_ns() - t1 < kTimeoutNs) {
      }
    };
    // A tile whose second part was never requested does not complete: its first
    // part has landed well before the wait below gives up.
    for (long long i = nk2 < 2 ? 0 : nk2 - 2; i < nk; ++i)
      drain(&ctl->k_full[i & 1], (uint32_t)(i >> 1) & 1);
    for (long long i = nv < 2 ? 0 : nv - 2; i < nv; ++i)
      drain(&ctl->v_full[i & 1], (uint32_t)(i >> 1) & 1);
    if (x > 0) drain(&ctl->q_full, (x - 1) & 1);
  }
}

// ---------------------------------------------------------------- relay (rank 1)
// Tells rank 0's MMA thread what is complete here.
__device__ void relay(const WideArgs& a, const WidePart& w, WideCtl* ctl) {
  const long long n = w.end - w.begin;
  long long nk = 0, np0 = 0, np1 = 0;              // next tile: keys, P of CTA 0's and CTA 1's keys
  uint32_t x = 0;
  unsigned long long t0 = 0;
  int tile = (int)(w.begin % w.tiles);             // of the next keys, within its block
  tc::mbar_arrive_expect_tx(&ctl->p_in, 128 * kPRow);
  while (np0 < n || np1 < n) {
    bool progress = false;
    if (np0 < nk && tc::mbar_test_wait(&ctl->p_in, (uint32_t)np0 & 1) &&
        tc::mbar_test_wait(&ctl->v_full[np0 & 1], (uint32_t)(np0 >> 1) & 1)) {
      tc::remote_arrive(tc::map_rank(&ctl->p_peer[0], 0));
      if (++np0 < n) tc::mbar_arrive_expect_tx(&ctl->p_in, 128 * kPRow);
      progress = true;
    }
    if (np1 < nk && tc::mbar_test_wait(&ctl->p_own, (uint32_t)np1 & 1)) {
      tc::remote_arrive(tc::map_rank(&ctl->p_peer[1], 0));
      ++np1;
      progress = true;
    }
    if (nk < n && nk <= np1 + 1 && tc::mbar_test_wait(&ctl->k_full[nk & 1], (uint32_t)(nk >> 1) & 1)) {
      bool q = true;
      if (nk == 0 || tile == 0) {
        q = tc::mbar_test_wait(&ctl->q_full, x & 1);
        if (q) {
          tc::remote_arrive(tc::map_rank(&ctl->q_peer, 0));
          ++x;
        }
      }
      if (q) {
        tc::remote_arrive(tc::map_rank(&ctl->k_peer[nk & 1], 0));
        if (++tile == w.tiles) tile = 0;
        ++nk;
        progress = true;
      }
    }
    if (progress) {
      t0 = 0;
      continue;
    }
    const unsigned long long now = tc::globaltimer_ns();
    if (t0 == 0) t0 = now;
    const bool expired = now - t0 > kTimeoutNs;
    if (*reinterpret_cast<volatile int*>(&ctl->abort_flag) || expired) {
      *reinterpret_cast<volatile int*>(&ctl->abort_flag) = 1;
      if (expired && a.status) atomicOr(a.status, MLA_FAULT_WAIT_TIMEOUT);
      return;
    }
  }
}

// ---------------------------------------------------------------- MMA issuer (rank 0)
__device__ void mma_issuer(const WideArgs& a, const WidePart& w, uint8_t* smem, WideCtl* ctl,
                           uint32_t tmem) {
  const uint32_t s_kv = tc::smem_u32(smem), s_q = tc::smem_u32(smem + kOffQ);
  const uint32_t s_p = tc::smem_u32(smem + kOffP);
  const long long n = w.end - w.begin;
  long long ns = 0, block_end = 0;                 // next S; tile at which the next block begins
  long long npv = 0;                               // next PV: half tiles, CTA 0's keys first
  int pv_tile = (int)(w.begin % w.tiles);          // PV's tile within its block
  bool pv_first = true;                            // the pair's first of the block
  uint32_t votes = 0;                              // verdicts the scouts gave before it
  uint32_t x = 0;
  bool q_ready = false;
  unsigned long long t0 = 0;
  tc::mbar_arrive_expect_tx(&ctl->p_in, 128 * kPRow);
  while (npv < 2 * n) {
    bool progress = false;
    const long long tp = npv >> 1;
    const int kh = (int)(npv & 1);
    const uint32_t pp = (uint32_t)tp & 1;
    if (tp < ns) {
      // P of CTA kh's keys and V for it, in both CTAs. The first half waits for
      // CTA 1's softmax too (and with it the second half's P) where that touches
      // what the half writes or reads: O (read out before a block's first tile,
      // scaled where the maxima moved) or V (keys past a block's end are cleared).
      bool ready = tc::mbar_test_wait(&ctl->p_peer[kh], pp);
      if (kh == 0) {
        ready = ready && tc::mbar_test_wait(&ctl->p_own, pp);
        if (ready && (pv_first || pv_tile == w.tiles - 1 || (peek(&ctl->verdict[votes & 1]) & kMoved)))
          ready = tc::mbar_test_wait(&ctl->p_peer[1], pp) && tc::mbar_test_wait(&ctl->p_in, pp) &&
                  tc::mbar_test_wait(&ctl->v_full[tp & 1], (uint32_t)(tp >> 1) & 1);
      } else {
        ready = ready && tc::mbar_test_wait(&ctl->p_in, pp) &&
                tc::mbar_test_wait(&ctl->v_full[tp & 1], (uint32_t)(tp >> 1) & 1);
      }
      if (ready) {
        tc::fence_after_sync();
        const uint32_t kv = s_kv + (tp & 1) * kStageBytes;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t va = tc::smem_desc(kv + (kh * 2 + i) * kChunkBytes + kk * 32 * 128,
                                              kChunkBytes, 1024, tc::kSw128);
            const uint32_t pk = s_p + (kh * 128 + kk * 32) * kPRow;
            tc::mma_f8_pair(tmem + i * kRows, va, tc::smem_desc(pk, kPBytes, 1024, tc::kSw128),
                            kIdescHi, !(pv_first && kh == 0 && kk == 0));
            tc::mma_f8_pair(tmem + i * kRows, va, tc::smem_desc(pk + 64, kPBytes, 1024, tc::kSw128),
                            kIdescLo, true);
          }
        tc::mma_commit_pair(kh == 0 ? &ctl->pv_half[tp & 1] : &ctl->pv_done[tp & 1]);
        if (kh == 1) {
          if (tp + 1 < n) tc::mbar_arrive_expect_tx(&ctl->p_in, 128 * kPRow);
          if (!pv_first) ++votes;
          if (++pv_tile == w.tiles) pv_tile = 0;
          pv_first = pv_tile == 0;
        }
        ++npv;
        progress = true;
      }
    }
    if (ns < n && ns <= (npv >> 1) + 1) {
      const int st = ns & 1;
      const uint32_t ph = (uint32_t)(ns >> 1) & 1;
      if (ns == block_end) {                       // a new block: its Q in both CTAs
        if (!q_ready)
          q_ready = tc::mbar_test_wait(&ctl->q_full, x & 1) &&
                    tc::mbar_test_wait(&ctl->q_peer, x & 1);
      }
      if ((ns != block_end || q_ready) && tc::mbar_test_wait(&ctl->k_full[st], ph) &&
          tc::mbar_test_wait(&ctl->k_peer[st], ph)) {
        // The S buffer of tile ns - 2 is free: its stage was refilled after its
        // PV, whose P the softmax wrote after it had read that S.
        tc::fence_after_sync();
        if (ns == block_end) {
          block_end += w.tiles - (w.begin + ns) % w.tiles;
          q_ready = false;
          ++x;
        }
        const uint32_t kv = s_kv + st * kStageBytes, d = tmem + kSCol + st * kRows;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc::mma_f8_pair(d, tc::smem_desc(kv + c * kChunkBytes + kk * 32, 16, 1024, tc::kSw128),
                            tc::smem_desc(s_q + c * kQChunk + kk * 32, 16, 1024, tc::kSw128),
                            kIdescS, (c | kk) != 0);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
          tc::mma_f8_pair(d, tc::smem_desc(kv + 4 * kChunkBytes + kk * 32, 16, 512, tc::kSw64),
                          tc::smem_desc(s_q + 4 * kQChunk + kk * 32, 16, 512, tc::kSw64), kIdescS,
                          true);
        tc::mma_commit_pair(&ctl->s_full[st]);
        ++ns;
        if (ns == block_end || ns == n) tc::mma_commit_pair(&ctl->q_empty);
        progress = true;
      }
    }
    if (progress) {
      t0 = 0;
    } else {
      const unsigned long long now = tc::globaltimer_ns();
      if (t0 == 0) t0 = now;
      const bool expired = now - t0 > kTimeoutNs;
      if (*reinterpret_cast<volatile int*>(&ctl->abort_flag) || expired) {
        *reinterpret_cast<volatile int*>(&ctl->abort_flag) = 1;
        if (expired && a.status) atomicOr(a.status, MLA_FAULT_WAIT_TIMEOUT);
        break;
      }
    }
  }
  tc::mma_commit_pair(&ctl->drain);                // every MMA done before TMEM is released
  const unsigned long long t1 = tc::globaltimer_ns();
  while (!tc::mbar_try_wait(&ctl->drain, 0) && tc::globaltimer_ns() - t1 < kTimeoutNs) {
  }
}

// ---------------------------------------------------------------- scouts
// Whether a score exceeds its row's max by more than 8, tile by tile, agreed
// between the pair's CTAs while the softmax computes P as if none did.
__device__ void scout(const WideArgs& a, const WidePart& w, WideCtl* ctl, uint32_t tmem,
                      uint32_t rank) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, tl = quarter * 32 + lane;
  const long long n = w.end - w.begin;
  int tile = (int)(w.begin % w.tiles);
  uint32_t votes = 0, moves = 0;
  bool ok = true, fresh = true;                    // fresh: the block's first tile
  for (long long g = 0; g < n; ++g) {
    const int st = g & 1, key0 = tile * kKeys;
    if (++tile == w.tiles) tile = 0;
    if (fresh) {                                   // its maxima come from the tile itself
      fresh = tile == 0;
      ok = __all_sync(0xffffffffu, ok && wait_moves(++moves, ctl, a.status));
      continue;
    }
    const int b = votes & 1;
    const uint32_t ph = (votes >> 1) & 1;
    ++votes;
    if (ok) ok = w_wait(&ctl->s_full[st], (uint32_t)(g >> 1) & 1, ctl, a.status);
    ok = __all_sync(0xffffffffu, ok);
    tc::fence_after_sync();
    const bool valid = key0 + (int)rank * 128 + tl < w.len;
    float most = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      uint32_t raw[32];
      tc::tmem_ld32(tmem + ((uint32_t)(quarter * 32) << 16) + kSCol + st * kRows + c * 32, raw);
      tc::tmem_wait_ld();
      const float4* m4 = reinterpret_cast<const float4*>(&ctl->m_run[c * 32]);
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        const float4 m = m4[i / 4];
        most = fmaxf(most, fmaf(__uint_as_float(raw[i]), a.bmm1_log2, -m.x));
        most = fmaxf(most, fmaf(__uint_as_float(raw[i + 1]), a.bmm1_log2, -m.y));
        most = fmaxf(most, fmaf(__uint_as_float(raw[i + 2]), a.bmm1_log2, -m.z));
        most = fmaxf(most, fmaf(__uint_as_float(raw[i + 3]), a.bmm1_log2, -m.w));
      }
    }
    tc::fence_before_sync();
    const bool any = __any_sync(0xffffffffu, valid && most > 8.f);
    if (lane == 0 && (any || !ok)) atomicOr(&ctl->vote[b], (any ? kMoved : 0) | (ok ? 0 : kFailed));
    scout_sync();
    if (quarter == 0) {
      uint32_t mine = peek(&ctl->vote[b]);
      __syncwarp();
      if (lane == 0) {
        ctl->vote[b] = 0;
        tc::mbar_arrive_expect_tx(&ctl->vote_bar[b], 4);
        tc::remote_st_async(tc::map_rank(&ctl->vote_peer[b], 1 - rank), mine & kMoved,
                            tc::map_rank(&ctl->vote_bar[b], 1 - rank));
        if (!w_wait(&ctl->vote_bar[b], ph, ctl, a.status)) mine |= kFailed;
        mine |= peek(&ctl->vote_peer[b]);
        *reinterpret_cast<volatile uint32_t*>(&ctl->verdict[b]) = mine;
        tc::mbar_arrive(&ctl->told[b]);
      }
    }
    scout_sync();
    const uint32_t verdict = peek(&ctl->verdict[b]);
    if (verdict & kFailed) return;                 // all of them
    if (verdict & kMoved) {
      ok = __all_sync(0xffffffffu, ok && wait_moves(++moves, ctl, a.status));
    }
    fresh = tile == 0;
  }
}

// ---------------------------------------------------------------- softmax
struct Soft {
  const WideArgs& a;
  WideCtl* ctl;
  uint32_t tmem, rank;
  int quarter, half, lane, gt;
  uint32_t swaps = 0, votes = 0, words = 0;
  bool ok = true;                                  // warp-uniform

  __device__ Soft(const WideArgs& a_, WideCtl* c, uint32_t t, uint32_t r)
      : a(a_), ctl(c), tmem(t), rank(r) {
    const int warp = threadIdx.x >> 5;
    quarter = warp & 3;
    gt = threadIdx.x - 128 - kScout;
    half = gt >> 7;
    lane = threadIdx.x & 31;
  }
  __device__ uint32_t lanes() const { return (uint32_t)(quarter * 32) << 16; }
  // A thread that gave up a wait goes on through the barriers, so that every
  // thread reaches each of them, until verdict() makes all of them leave.
  __device__ void wait(uint64_t* bar, uint32_t parity) {
    const bool got = ok && w_wait(bar, parity, ctl, a.status);
    ok = __all_sync(0xffffffffu, got);
  }
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
  // P of the tile: codes of this thread's key in 64 rows; lp gathers the row
  // sums. Scores more than 9 above a row's max count as 9: the scouts' verdict
  // has such a tile done again.
  __device__ void weigh(int st, bool valid, float (&lp)[64], uint32_t (&hi)[16],
                        uint32_t (&lo)[16]) const {
    uint32_t raw[2][32];
    const uint32_t at = tmem + lanes() + kSCol + st * kRows + half * 64;
    tc::tmem_ld32(at, raw[0]);
    tc::tmem_ld32(at + 32, raw[1]);
    tc::tmem_wait_ld();
    const float4* m4 = reinterpret_cast<const float4*>(&ctl->m_run[half * 64]);
#pragma unroll
    for (int i = 0; i < 64; i += 4) {
      const float4 mm = m4[i / 4];
      const float m[4] = {mm.x, mm.y, mm.z, mm.w};
      float p[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float s = __uint_as_float(raw[i >> 5][(i & 31) + u]);
        p[u] = valid ? ex2(at_most_9(fmaf(s, a.bmm1_log2, -m[u]))) : 0.f;
        lp[i + u] += p[u];
      }
      const uint32_t h01 = dec::f32x2_to_f16x2(p[0], p[1]), h23 = dec::f32x2_to_f16x2(p[2], p[3]);
      const uint16_t e01 = dec::f16x2_to_e4m3x2(h01), e23 = dec::f16x2_to_e4m3x2(h23);
      const uint16_t l01 = f16x2_to_e5m2x2(dec::f16x2_sub(h01, e4m3x2_to_f16x2(e01)));
      const uint16_t l23 = f16x2_to_e5m2x2(dec::f16x2_sub(h23, e4m3x2_to_f16x2(e23)));
      hi[i / 4] = (uint32_t)e01 | ((uint32_t)e23 << 16);
      lo[i / 4] = (uint32_t)l01 | ((uint32_t)l23 << 16);
    }
  }
  // Takes back what weigh added (the same values bit for bit).
  __device__ void unweigh(int st, bool valid, float (&lp)[64]) const {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t raw[32];
      tc::tmem_ld32(tmem + lanes() + kSCol + st * kRows + half * 64 + c * 32, raw);
      tc::tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float d =
            fmaf(__uint_as_float(raw[i]), a.bmm1_log2, -ctl->m_run[half * 64 + c * 32 + i]);
        lp[c * 32 + i] -= valid ? ex2(at_most_9(d)) : 0.f;
      }
    }
  }
  // Rows whose max grew by more than 8: the new max, 2 below the tile's, agreed
  // with the other CTA; row sums and O follow. `last`: the pair's previous tile
  // if O holds something of this block, else -1.
  __device__ void move(int st, bool valid, float (&lp)[64], long long last) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t raw[32];
      float v[32];
      tc::tmem_ld32(tmem + lanes() + kSCol + st * kRows + half * 64 + c * 32, raw);
      tc::tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 32; ++i)
        v[i] = valid ? __uint_as_float(raw[i]) * a.bmm1_log2 : -INFINITY;
      dec::transpose_reduce32<true>(v, lane);
      ctl->red[quarter][half * 64 + c * 32 + lane] = v[0];
    }
    soft_sync();
    if (gt < kRows) {
      const float own = fmaxf(fmaxf(ctl->red[0][gt], ctl->red[1][gt]),
                              fmaxf(ctl->red[2][gt], ctl->red[3][gt]));
      const float tm = fmaxf(own, swap(own));
      const float mo = ctl->m_run[gt];
      const float mn = tm > mo + 8.f ? tm - dec::kMaxLead : mo;
      ctl->vec[gt] = mo == -INFINITY ? 0.f : ex2(mo - mn);
      ctl->m_run[gt] = mn;
    } else {
      ++swaps;
    }
    soft_sync();
    if (gt == 0) {
      __threadfence_block();
      *reinterpret_cast<volatile uint32_t*>(&ctl->moves) += 1;
    }
#pragma unroll
    for (int i = 0; i < 64; ++i) lp[i] *= ctl->vec[half * 64 + i];
    if (last >= 0) {
      wait(&ctl->pv_done[last & 1], (uint32_t)(last >> 1) & 1);
      tc::fence_after_sync();
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {                // two blocks of dims, 32 rows at a time
        uint32_t raw[32];
        const int row = half * 64 + (i & 1) * 32;
        const uint32_t at = tmem + lanes() + (i >> 1) * kRows + row;
        tc::tmem_ld32(at, raw);
        tc::tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e)
          raw[e] = __float_as_uint(__uint_as_float(raw[e]) * ctl->vec[row + e]);
        tc::tmem_st32(at, raw);
      }
      tc::tmem_wait_st();
    }
  }
  // The scouts' verdict on the tile, the same for every thread; kFailed also
  // once any softmax thread gave up a wait.
  __device__ uint32_t verdict() {
    const int v = votes & 1, b = words & 1;
    const uint32_t ph = (votes >> 1) & 1;
    ++votes;
    ++words;
    if (gt < 32) {
      wait(&ctl->told[v], ph);
      if (lane == 0) atomicOr(&ctl->soft_word[b], (ok ? peek(&ctl->verdict[v]) : kFailed));
    } else if (!ok && lane == 0) {
      atomicOr(&ctl->soft_word[b], kFailed);
    }
    soft_sync();
    const uint32_t word = peek(&ctl->soft_word[b]);
    // The other word was last read before this barrier.
    if (gt == 0) *reinterpret_cast<volatile uint32_t*>(&ctl->soft_word[b ^ 1]) = 0;
    return word;
  }
};

__device__ void softmax(const WideArgs& a, const WidePart& w, uint8_t* smem, WideCtl* ctl,
                        uint32_t tmem, uint32_t rank) {
  Soft s(a, ctl, tmem, rank);
  const int tl = s.quarter * 32 + s.lane;          // key of this CTA's half tile / dim of a block
  const long long n = w.end - w.begin;
  int block = (int)(w.begin / w.tiles), first_tile = (int)(w.begin % w.tiles);
  float lp[64];                                    // this key's share of its rows' sums
  // Where this key's 64 rows go, the P half of CTA `half`: rows of 128 bytes in
  // 16-byte pieces, piece j of key k at j ^ (k & 7). Rows for the other CTA wait
  // here for a bulk copy: 64 keys in the stage's rope slot, which S is done with,
  // 64 behind P; both are free again once PV of the tile is done.
  const int key = (int)rank * 128 + tl;
  const bool away = s.half != (int)rank;
  long long g = 0;
  while (g < n) {
    const int nt = (int)min((long long)(w.tiles - first_tile), n - g);
    soft_sync();                                   // the previous block's readers are done
    if (s.gt < kRows) ctl->m_run[s.gt] = -INFINITY;
#pragma unroll
    for (int i = 0; i < 64; ++i) lp[i] = 0.f;
    soft_sync();
    for (int t = 0; t < nt; ++t, ++g) {
      const int st = g & 1;
      const uint32_t ph = (uint32_t)(g >> 1) & 1;
      const int key0 = (first_tile + t) * kKeys;
      const bool valid = key0 + key < w.len;
      uint32_t hi[16], lo[16];
      s.wait(&ctl->s_full[st], ph);
      tc::fence_after_sync();
      if (t == 0) {
        s.move(st, valid, lp, -1);
        s.weigh(st, valid, lp, hi, lo);
      } else {
        s.weigh(st, valid, lp, hi, lo);
        const uint32_t verdict = s.verdict();
        if (verdict & kFailed) return;             // all of them
        if (verdict & kMoved) {
          s.unweigh(st, valid, lp);
          soft_sync();                             // everyone has read the old maxima
          s.move(st, valid, lp, g - 1);
          s.weigh(st, valid, lp, hi, lo);
        }
      }
      // The place of P of these keys is free once PV of the previous tile is done
      // with it.
      if (g > 0)
        s.wait(rank == 0 ? &ctl->pv_half[(g - 1) & 1] : &ctl->pv_done[(g - 1) & 1],
               (uint32_t)((g - 1) >> 1) & 1);
      uint8_t* put = smem + (!away ? kOffP + key * kPRow
                             : tl < 64 ? st * kStageBytes + 4 * kChunkBytes + tl * kPRow
                                       : kOffStage + (tl - 64) * kPRow);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        *reinterpret_cast<uint4*>(put + ((j ^ (key & 7)) << 4)) =
            make_uint4(hi[4 * j], hi[4 * j + 1], hi[4 * j + 2], hi[4 * j + 3]);
        *reinterpret_cast<uint4*>(put + (((4 + j) ^ (key & 7)) << 4)) =
            make_uint4(lo[4 * j], lo[4 * j + 1], lo[4 * j + 2], lo[4 * j + 3]);
      }
      // Keys past the end: their V must be finite (0), in both halves' slots.
      if (key0 + kKeys > w.len) {
        s.wait(&ctl->v_full[st], ph);
#pragma unroll
        for (int kh = 0; kh < 2; ++kh)
          if (key0 + kh * 128 + tl >= w.len) {
            uint4* v = reinterpret_cast<uint4*>(smem + st * kStageBytes +
                                                (kh * 2 + s.half) * kChunkBytes + tl * 128);
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = make_uint4(0, 0, 0, 0);
          }
      }
      tc::fence_proxy_async_smem();
      tc::fence_before_sync();
      __syncwarp();
      if (s.lane == 0) {
        if (away)                                  // this warp's 32 keys
          tc::bulk_copy_to(tc::map_rank(smem + kOffP + key * kPRow, 1 - rank), put, 32 * kPRow,
                           tc::map_rank(&ctl->p_in, 1 - rank));
        tc::mbar_arrive(&ctl->p_own);
      }
    }
    // Row sums over both CTAs' keys, 1 / l and the LSE, then this CTA's dims.
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = lp[c * 32 + i];
      dec::transpose_reduce32<false>(v, s.lane);
      ctl->red[s.quarter][s.half * 64 + c * 32 + s.lane] = v[0];
    }
    soft_sync();
    const size_t slot = (size_t)(w.unit + block) * kRows;
    const int rows = (int)min((long long)kRows, a.N - (long long)block * kRows);
    if (s.gt < kRows) {
      const float own = ctl->red[0][s.gt] + ctl->red[1][s.gt] + ctl->red[2][s.gt] + ctl->red[3][s.gt];
      const float l = own + s.swap(own);
      ctl->vec[s.gt] = l > 0.f ? 1.f / l : 0.f;
      if (rank == 0 && s.gt < rows)
        a.part_lse[slot + s.gt] = l == 0.f ? -INFINITY : ctl->m_run[s.gt] + __log2f(l);
    } else {
      ++s.swaps;
    }
    soft_sync();
    s.wait(&ctl->pv_done[(g - 1) & 1], (uint32_t)((g - 1) >> 1) & 1);
    tc::fence_after_sync();
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {                  // two blocks of dims, 32 rows at a time
      uint32_t raw[32];
      const int row0 = s.half * 64 + (i & 1) * 32;
      tc::tmem_ld32(tmem + s.lanes() + (i >> 1) * kRows + row0, raw);
      tc::tmem_wait_ld();
      float* dst = a.part_o + (slot + row0) * kDv + rank * 256 + (i >> 1) * 128 + tl;
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (row0 + e < rows) dst[(size_t)e * kDv] = __uint_as_float(raw[e]) * ctl->vec[row0 + e];
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
      tc::mbar_init(&ctl->k_full[b], 1);
      tc::mbar_init(&ctl->k_peer[b], 1);
      tc::mbar_init(&ctl->v_full[b], 1);
      tc::mbar_init(&ctl->s_full[b], 1);
      tc::mbar_init(&ctl->p_peer[b], 1);
      tc::mbar_init(&ctl->pv_half[b], 1);
      tc::mbar_init(&ctl->pv_done[b], 1);
      tc::mbar_init(&ctl->vote_bar[b], 1);
      tc::mbar_init(&ctl->told[b], 1);
      tc::mbar_init(&ctl->swap_bar[b], 1);
      ctl->vote[b] = 0;
      ctl->soft_word[b] = 0;
    }
    tc::mbar_init(&ctl->p_own, kSoft / 32);
    tc::mbar_init(&ctl->p_in, 1);
    ctl->moves = 0;
    tc::mbar_init(&ctl->q_full, 1);
    tc::mbar_init(&ctl->q_peer, 1);
    tc::mbar_init(&ctl->q_empty, 1);
    tc::mbar_init(&ctl->drain, 1);
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
      producer(a, w, smem, ctl, rank, &tm_kv, &tm_kvr, &tm_q, &tm_qr);
    } else if (warp == 1 && lane == 0) {
      if (rank == 0)
        mma_issuer(a, w, smem, ctl, tmem);
      else
        relay(a, w, ctl);
    }
  } else if (warp < 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsScout));
    scout(a, w, ctl, tmem, rank);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    softmax(a, w, smem, ctl, tmem, rank);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (ctl->abort_flag)     // let stores in flight to the other CTA land before it may leave
    for (const unsigned long long t0 = tc::globaltimer_ns(); tc::globaltimer_ns() - t0 < 100000;) {
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
