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
// computed on the assumption that no row moves, the CTAs exchange a flag, and
// only where one of them saw a row move is the tile done again with new maxima.
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
constexpr int kSoft = 256;                    // softmax threads: a key and 64 rows each
constexpr int kThreads = 64 + kSoft;
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
  uint64_t s_full[2];      // MMA -> softmax, TMA: S of a tile done
  uint64_t p_full;         // softmax of both CTAs -> MMA (rank 0), relay (rank 1): this CTA's
                           // rows of P written
  uint64_t p_peer;         // rank 0: P and V complete in the other CTA
  uint64_t pv_done[2];     // MMA -> softmax, TMA: O holds the tile; P and the stage are free
  uint64_t q_full, q_peer, q_empty;
  uint64_t vote_bar[2];    // the other CTA's flag is in vote_peer
  uint64_t swap_bar[2];    // the other CTA's row values are in swap
  uint64_t drain;
  uint32_t vote_peer[2];
  uint32_t vote[2];        // bits of this CTA's threads: kMoved, kFailed
  uint32_t decision;
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
  long long nk = 0, nv = 0;                        // next tile: own keys, other keys' values
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
      if (nk < n && (nk < 2 || tc::mbar_test_wait(&ctl->pv_done[nk & 1], (uint32_t)((nk >> 1) - 1) & 1)))
        can |= 2;
      if (nv < nk && tc::mbar_test_wait(&ctl->s_full[nv & 1], (uint32_t)(nv >> 1) & 1)) can |= 4;
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
          for (int c = 0; c < 4; ++c)
            tc::tma_load_2d(stage + c * kChunkBytes + h * (kChunkBytes / 2), tm_kv,
                            &ctl->k_full[st], c * 128, id * kPage);
          tc::tma_load_2d(stage + 4 * kChunkBytes + h * (kRopeBytes / 2), tm_kvr, &ctl->k_full[st],
                          512, id * kPage);
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
    for (long long i = nk < 2 ? 0 : nk - 2; i < nk; ++i)
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
  long long nk = 0, np = 0;                        // next tile: keys, P
  uint32_t x = 0;
  unsigned long long t0 = 0;
  while (np < n) {
    bool progress = false;
    if (np < nk && tc::mbar_test_wait(&ctl->p_full, (uint32_t)np & 1) &&
        tc::mbar_test_wait(&ctl->v_full[np & 1], (uint32_t)(np >> 1) & 1)) {
      tc::remote_arrive(tc::map_rank(&ctl->p_peer, 0));
      ++np;
      progress = true;
    }
    if (nk < n && nk <= np + 1 && tc::mbar_test_wait(&ctl->k_full[nk & 1], (uint32_t)(nk >> 1) & 1)) {
      bool q = true;
      if (nk == 0 || (w.begin + nk) % w.tiles == 0) {
        q = tc::mbar_test_wait(&ctl->q_full, x & 1);
        if (q) {
          tc::remote_arrive(tc::map_rank(&ctl->q_peer, 0));
          ++x;
        }
      }
      if (q) {
        tc::remote_arrive(tc::map_rank(&ctl->k_peer[nk & 1], 0));
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
  long long ns = 0, npv = 0, block_end = 0;        // tile at which the next block begins
  uint32_t x = 0;
  bool q_ready = false;
  unsigned long long t0 = 0;
  while (npv < n) {
    bool progress = false;
    if (npv < ns && tc::mbar_test_wait(&ctl->p_full, (uint32_t)npv & 1) &&
        tc::mbar_test_wait(&ctl->p_peer, (uint32_t)npv & 1) &&
        tc::mbar_test_wait(&ctl->v_full[npv & 1], (uint32_t)(npv >> 1) & 1)) {
      tc::fence_after_sync();
      const uint32_t kv = s_kv + (npv & 1) * kStageBytes;
      const bool first = npv == 0 || (w.begin + npv) % w.tiles == 0;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int kh = 0; kh < 2; ++kh)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t va = tc::smem_desc(kv + (kh * 2 + i) * kChunkBytes + kk * 32 * 128,
                                              kChunkBytes, 1024, tc::kSw128);
            const uint32_t pk = s_p + (kh * 128 + kk * 32) * kPRow;
            tc::mma_f8_pair(tmem + i * kRows, va, tc::smem_desc(pk, kPBytes, 1024, tc::kSw128),
                            kIdescHi, !(first && kh == 0 && kk == 0));
            tc::mma_f8_pair(tmem + i * kRows, va, tc::smem_desc(pk + 64, kPBytes, 1024, tc::kSw128),
                            kIdescLo, true);
          }
      tc::mma_commit_pair(&ctl->pv_done[npv & 1]);
      ++npv;
      progress = true;
    }
    if (ns < n && ns <= npv + 1) {
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

// ---------------------------------------------------------------- softmax
struct Soft {
  const WideArgs& a;
  uint8_t* smem;
  WideCtl* ctl;
  uint32_t tmem, rank;
  int quarter, half, lane, gt;
  uint32_t swaps = 0, votes = 0;
  bool ok = true;                                  // warp-uniform

  __device__ Soft(const WideArgs& a_, uint8_t* s, WideCtl* c, uint32_t t, uint32_t r)
      : a(a_), smem(s), ctl(c), tmem(t), rank(r) {
    const int warp = threadIdx.x >> 5;
    quarter = warp & 3;
    half = (warp - 2) >> 2;
    lane = threadIdx.x & 31;
    gt = threadIdx.x - 64;
  }
  __device__ uint32_t lanes() const { return (uint32_t)(quarter * 32) << 16; }
  // A thread that gave up a wait goes on through the barriers, so that every
  // thread reaches each of them, until the next vote makes all of them leave.
  __device__ void wait(uint64_t* bar, uint32_t parity) {
    const bool got = ok && w_wait(bar, parity, ctl, a.status);
    ok = __all_sync(0xffffffffu, got);
  }
  // Scores of 32 rows of this thread's key, in base 2 (-inf for keys past the end).
  __device__ void scores(int st, int c, bool valid, float (&v)[32]) const {
    uint32_t raw[32];
    tc::tmem_ld32(tmem + lanes() + kSCol + st * kRows + half * 64 + c * 32, raw);
    tc::tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i)
      v[i] = valid ? __uint_as_float(raw[i]) * a.bmm1_log2 : -INFINITY;
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
  // P of the tile: codes of this thread's key in 64 rows; lp gathers the row
  // sums; returns the largest score above a row's max. Scores more than 9 above
  // it count as 9: such a tile is done again.
  __device__ float weigh(int st, bool valid, float (&lp)[64], uint32_t (&hi)[16],
                         uint32_t (&lo)[16]) const {
    float most = -INFINITY;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t raw[32];
      tc::tmem_ld32(tmem + lanes() + kSCol + st * kRows + half * 64 + c * 32, raw);
      tc::tmem_wait_ld();
      const float4* m4 = reinterpret_cast<const float4*>(&ctl->m_run[half * 64 + c * 32]);
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        const float4 mm = m4[i / 4];
        const float m[4] = {mm.x, mm.y, mm.z, mm.w};
        float p[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float d =
              valid ? fmaf(__uint_as_float(raw[i + u]), a.bmm1_log2, -m[u]) : -INFINITY;
          most = fmaxf(most, d);
          p[u] = ex2(at_most_9(d));
          lp[c * 32 + i + u] += p[u];
        }
        const uint32_t h01 = dec::f32x2_to_f16x2(p[0], p[1]), h23 = dec::f32x2_to_f16x2(p[2], p[3]);
        const uint16_t e01 = dec::f16x2_to_e4m3x2(h01), e23 = dec::f16x2_to_e4m3x2(h23);
        const uint16_t l01 = f16x2_to_e5m2x2(dec::f16x2_sub(h01, e4m3x2_to_f16x2(e01)));
        const uint16_t l23 = f16x2_to_e5m2x2(dec::f16x2_sub(h23, e4m3x2_to_f16x2(e23)));
        hi[c * 8 + i / 4] = (uint32_t)e01 | ((uint32_t)e23 << 16);
        lo[c * 8 + i / 4] = (uint32_t)l01 | ((uint32_t)l23 << 16);
      }
    }
    return most;
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
        const float d = valid ? fmaf(__uint_as_float(raw[i]), a.bmm1_log2,
                                     -ctl->m_run[half * 64 + c * 32 + i])
                              : -INFINITY;
        lp[c * 32 + i] -= ex2(at_most_9(d));
      }
    }
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
  // Rows whose max grew by more than 8: the new max, 2 below the tile's, agreed
  // with the other CTA; row sums and O follow. `last`: the pair's previous tile
  // if O holds something of this block, else -1.
  __device__ void move(int st, bool valid, float (&lp)[64], long long last) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float v[32];
      scores(st, c, valid, v);
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
  // Whether any row of the pair moved; false with ok unset once any thread here
  // gave up a wait.
  __device__ bool vote(bool moved) {
    const int b = votes & 1;
    const uint32_t ph = (votes >> 1) & 1;
    ++votes;
    const bool any = __any_sync(0xffffffffu, moved);
    if (lane == 0 && (any || !ok))
      atomicOr(&ctl->vote[b], (any ? kMoved : 0) | (ok ? 0 : kFailed));
    soft_sync();
    if (gt < 32) {
      uint32_t mine = *reinterpret_cast<volatile uint32_t*>(&ctl->vote[b]);
      if (lane == 0) {
        ctl->vote[b ^ 1] = 0;                      // read by all before this barrier
        tc::mbar_arrive_expect_tx(&ctl->vote_bar[b], 4);
        tc::remote_st_async(tc::map_rank(&ctl->vote_peer[b], 1 - rank), mine & kMoved,
                            tc::map_rank(&ctl->vote_bar[b], 1 - rank));
      }
      wait(&ctl->vote_bar[b], ph);
      if (!ok) mine |= kFailed;
      if (lane == 0)
        ctl->decision = mine | *reinterpret_cast<volatile uint32_t*>(&ctl->vote_peer[b]);
    }
    soft_sync();
    const uint32_t d = *reinterpret_cast<volatile uint32_t*>(&ctl->decision);
    if (d & kFailed) ok = false;
    return (d & kMoved) != 0;
  }
};

__device__ void softmax(const WideArgs& a, const WidePart& w, uint8_t* smem, WideCtl* ctl,
                        uint32_t tmem, uint32_t rank) {
  Soft s(a, smem, ctl, tmem, rank);
  const int tl = s.quarter * 32 + s.lane;          // key of this CTA's half tile / dim of a block
  const long long n = w.end - w.begin;
  float lp[64];                                    // this key's share of its rows' sums
  long long g = 0;
  while (g < n) {
    const int block = (int)((w.begin + g) / w.tiles), first_tile = (int)((w.begin + g) % w.tiles);
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
      const bool valid = key0 + (int)rank * 128 + tl < w.len;
      uint32_t hi[16], lo[16];
      s.wait(&ctl->s_full[st], ph);
      tc::fence_after_sync();
      if (t == 0) {
        s.move(st, valid, lp, -1);
        s.weigh(st, valid, lp, hi, lo);
      } else {
        const float most = s.weigh(st, valid, lp, hi, lo);
        const bool moved = s.vote(most > 8.f);
        if (!s.ok) return;
        if (moved) {
          s.unweigh(st, valid, lp);
          soft_sync();                             // everyone has read the old maxima
          s.move(st, valid, lp, g - 1);
          s.weigh(st, valid, lp, hi, lo);
        }
      }
      // P is free once PV of the previous tile is done with it.
      if (g > 0) s.wait(&ctl->pv_done[(g - 1) & 1], (uint32_t)((g - 1) >> 1) & 1);
      // This key's 64 rows: the P half of CTA `half`, rows of 128 bytes in 16-byte
      // pieces, piece j of key k at j ^ (k & 7). Rows for the other CTA wait here
      // for a bulk copy: 64 keys in the stage's rope slot, which S is done with,
      // 64 behind P; both are free again once PV of this tile is done.
      const int key = (int)rank * 128 + tl;
      const bool away = s.half != (int)rank;
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
                           tc::map_rank(&ctl->p_full, 1 - rank));
        // One warp also announces what the other CTA's 128 keys bring.
        if (s.gt == 0)
          tc::mbar_arrive_expect_tx(&ctl->p_full, 128 * kPRow);
        else
          tc::mbar_arrive(&ctl->p_full);
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
      tc::mbar_init(&ctl->pv_done[b], 1);
      tc::mbar_init(&ctl->vote_bar[b], 1);
      tc::mbar_init(&ctl->swap_bar[b], 1);
      ctl->vote[b] = 0;
    }
    tc::mbar_init(&ctl->p_full, kSoft / 32);
    tc::mbar_init(&ctl->p_peer, 1);
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
  } else if (warp == 0) {
    producer(a, w, smem, ctl, rank, &tm_kv, &tm_kvr, &tm_q, &tm_qr);
  } else if (warp == 1) {
    if (lane == 0) {
      if (rank == 0)
        mma_issuer(a, w, smem, ctl, tmem);
      else
        relay(a, w, ctl);
    }
  } else {
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
