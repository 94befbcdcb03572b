// Blocks of 128 query rows against the keys they share: all rows against the
// prefix's, a request's rows against its own (prefix.h says in which order and by
// which CTAs; prefix.cu joins the partial results).
//
// Bound by the FP8 tensor pipe: 2 * 1088 FLOP per (row, key) beside 576 bytes
// per key; with few rows per request by what two stages of keys per CTA can
// stream from HBM. What sets the shape is TMEM: a 512-dim FP32 accumulator of 128 rows
// fills an SM's 512 columns. A pair of CTAs (tcgen05 cta_group::2) therefore
// shares a block of 128 rows, 64 in each CTA: an MMA of M = 128 over the pair
// keeps a CTA's 64 rows in all 128 lanes (lanes 0-63 its first N / 2 columns,
// lanes 64-127 the others), so O takes 256 columns beside two S buffers of 128,
// and at N = 256 runs at the pipe's full rate (66 cycles per instruction
// measured; an M = 128, N = 64 MMA of one CTA takes 50 for a quarter of it).
//
//   S[128 rows, 256 keys]  = Q[128, 576] . K[256, 576]^T      18 MMAs
//   O[128 rows, 512 dims] += P[128, 256] . V[256, 512]        2 dim halves x 16 MMAs
//
// Rows never leave their CTA: softmax, maxima and sums are its own. B is split
// over the pair: CTA c brings keys 128 c .. 128 c + 127 of a 256-key tile to S,
// and dims 256 c .. 256 c + 255 of all 256 keys to PV. A KV stage holds the CTA's
// own keys (four 128-dim bands and the rope); once S is done with them, its two
// bands of the other CTA's dims are overwritten with the other CTA's keys of its
// own dims, so that V of (dim half i, keys of CTA h) lies in slot 2 h + i in both
// CTAs, as the pair's MMA wants, and two stages fit.
//
// P enters the product as an E4M3 and an E5M2 term: hi = e4m3(p), lo = e5m2(p - hi).
// E5M2's range keeps the second term where hi is subnormal (p < 2^-6, absolute step
// 2^-9), so hi + lo is p to 2^-8 relative or 2^-14 absolute. With a second E4M3 term, as in
// the decode of every request on its own, it is 2^-9 or 2^-10: modelled over 4,096 keys
// (tests/test_prefix_p_precision.py), outputs of broad rows (values of deviation 0.5) are off
// by 9e-4 of theirs against 5e-4, those of peaked rows (deviation 1) by 7e-4 against 2 - 3e-3.
// The running max is lazy (moved when 32 weights of a row sum to more than 2^8, to 2 below
// the tile's); P is computed as if no row moved and once more where one did.
//
// With plan and merge: 128 x 7 x 64 behind 16k 1.13 - 1.18 ms (power cap), 2.0 PFLOP/s
// (0.52 of twice the BF16 rate); 24 x 1 x 64 behind 64k 111 us (0.51); 64 x 7 x 8 behind 16k
// 99 us (0.37); 32 x 4 x 8 behind 4k 27 - 30 us by its lengths; 2 x 4 x 8 behind 300 18 us. The
// second term of P makes the tensor pipe's work 1.47 times the algorithmic. A tile takes
// 4,110 cycles against the MMAs' 3,300: from S to PV 2,380 (weights 1,100, vote 280, wait
// for P's place 320, stores 490) and from PV to the next band of keys 1,420, with two stages
// to hide them behind. From a piece's last P to the next piece's first S it takes 11,000:
// the last PV and the row sums 3,000 - 4,000, partial rows out 6,200. Tried and
// slower: the softmax in two halves of warps, so that PV begins on the first (by CTA's
// keys: only two of four schedulers work, 4,385 cycles; by 64 keys of each: 4,397); P
// written before the vote (112 -> 120 us); barriers per 32 rows (112 -> 116); V of CTA
// 0's keys as soon as S leaves its bands (112 -> 114).
#include "decode_common.cuh"
#include "formats.cuh"
#include "internal.h"
#include "pair.cuh"
#include "prefix.h"
#include "ptx.cuh"
#include "tc.cuh"

namespace mlafold {
namespace {

using dec::kChunkBytes;      // 128 keys x 128 dims
using dec::kRopeBytes;       // 128 keys x 64 dims
using dec::kStageBytes;

constexpr int kRows = kWideRows;              // query rows per block, half of them per CTA
constexpr int kKeys = kWideKeys;              // keys per tile
constexpr int kSoft = 512;                    // softmax threads: a row and 32 keys each
constexpr int kThreads = 128 + kSoft;         // + two TMA warps, the S and the PV warp
constexpr int kQChunk = 64 * 128;             // this CTA's 64 rows x 128 dims
constexpr int kQBytes = 64 * kDqk;
constexpr int kPChunk = 64 * 128;             // 64 rows x 128 keys of one term
constexpr int kOffQ = 2 * kStageBytes;
constexpr int kOffP = kOffQ + kQBytes;        // hi of CTA 0's and CTA 1's keys, then lo
constexpr int kOffCtl = kOffP + 4 * kPChunk;
constexpr uint32_t kTmemCols = 512;
constexpr int kSCol = 256;                    // S buffers after O's two halves of 128 columns
constexpr unsigned long long kWaitLimitNs = 2000000000ull;
constexpr uint32_t kIdescS = tc::idesc_e4m3_f32(kRows, kKeys, false, false);
constexpr uint32_t kIdescHi = tc::idesc_e4m3_f32(kRows, 256, false, true);
constexpr uint32_t kIdescLo = kIdescHi | (1u << 7);       // A in E5M2
static_assert(kOffQ % 1024 == 0 && kOffP % 1024 == 0, "swizzle atoms need 1 KB alignment");

struct WideCtl {
  uint64_t k_full[2];      // rank 0: TMA of both CTAs -> S: bands 0, 1 and the rope of both
                           // CTAs' keys landed
  uint64_t k_band[2][2];   // rank 0: TMA of both CTAs -> S: bands 2 and 3, by stage and band
  uint64_t v_full[2];      // rank 0: TMA of both CTAs -> PV: V complete in both
  uint64_t v_tail[2];      // TMA -> softmax, TMA warp: V of a block's last tile landed here
  uint64_t s_full[2];      // MMA -> softmax, TMA: S of a tile done
  uint64_t p_full[2];      // rank 0: softmax of both CTAs -> PV: P of CTA h's keys written
  uint64_t pv_first[2];    // MMA -> TMA: O's first dim half holds CTA 0's keys of the tile
  uint64_t pv_half[2];     // MMA -> softmax, TMA: all of O does
  uint64_t pv_most[2];     // MMA -> TMA: and the first dim half of CTA 1's
  uint64_t pv_done[2];     // MMA -> softmax, TMA: O holds the tile; P and the stage are free
  uint64_t q_full;         // rank 0: TMA of both CTAs -> S
  uint64_t q_empty;        // MMA -> TMA
  uint64_t drain[2];
  uint32_t tmem_base;
  int abort_flag;
  alignas(16) float red[8][64];     // row values of the eight threads that share a row
};
// Behind the control block: the plan (R + 1 places) and the lengths.
constexpr int kOffPlan = kOffCtl + (int)((sizeof(WideCtl) + 15) / 16 * 16);
constexpr int kSmemBytes = kOffPlan + (2 * kMaxR + 1) * 4 + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

// TEST, through the whole kernel: the instance of the failure-detection test, whose limit is an
// argument (read in the regular instance, it cost the tiles' loops 1 - 2 %).
template <bool TEST>
__device__ __forceinline__ unsigned long long wait_limit(const WideArgs& a) {
  return TEST ? a.wait_limit_ns : kWaitLimitNs;
}
template <bool TEST>
__device__ __forceinline__ bool w_wait(uint64_t* bar, uint32_t parity, WideCtl* ctl,
                                       const WideArgs& a) {
  if (tc::mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = tc::globaltimer_ns();
  while (true) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    if (*reinterpret_cast<volatile int*>(&ctl->abort_flag)) return false;
    if (tc::globaltimer_ns() - t0 > wait_limit<TEST>(a)) {
      *reinterpret_cast<volatile int*>(&ctl->abort_flag) = 1;
      if (a.status) atomicOr(a.status, MLA_FAULT_WAIT_TIMEOUT);
      return false;
    }
  }
}
__device__ __forceinline__ void soft_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kSoft) : "memory");
}
__device__ __forceinline__ bool soft_any(bool pred) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
      " bar.red.or.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)pred), "n"(kSoft)
      : "memory");
  return r != 0;
}

// ---------------------------------------------------------------- loads
// The page ids of a piece's tiles, in lanes 0-3 of a warp: asked for a tile ahead,
// checked when used. One outside the cache becomes the first page behind it, which a
// copy fills with zeros: no stale keys take its place.
struct Pages {
  const WideArgs& a;
  const int32_t* table = nullptr;
  int page = 0, end = 0, next = 0, lane;           // page: this lane's of the next tile
  bool there = false;                              // it is one of the keys' pages
  __device__ explicit Pages(const WideArgs& a_) : a(a_), lane(threadIdx.x & 31) {}
  __device__ void ask() {
    there = lane < kKeys / kPage && page < end;
    if (there) next = table[page];
    page += kKeys / kPage;
  }
  __device__ void begin(const WidePiece& p) {
    table = p.table;
    page = p.tile * (kKeys / kPage) + lane;
    end = (int)cdiv(p.len, kPage);
    ask();
  }
  __device__ int take(bool more, bool report) {    // -1: no such page
    int cur = there ? next : -1;
    if (there && (cur < 0 || cur >= a.num_pages)) {
      if (report && a.status) atomicOr(a.status, MLA_FAULT_PAGE_RANGE);
      cur = a.num_pages;
    }
    if (more) ask();
    return cur;
  }
};

// Own keys (and Q at each piece's start). A stage's bands hold V in the order in
// which PV is done with it (CTA 0's keys of the first dim half, of the second, CTA
// 1's keys): each is refilled as it becomes free, so that little is left to load once
// PV is done.
template <bool TEST>
__device__ void load_keys(const WideArgs& a, WideWalk walk, uint8_t* smem, WideCtl* ctl,
                          uint32_t rank, const CUtensorMap* tm_kv, const CUtensorMap* tm_kvr,
                          const CUtensorMap* tm_q, const CUtensorMap* tm_qr) {
  const int lane = threadIdx.x & 31;
  Pages pages(a);
  const uint32_t q_bar = tc::map_rank(&ctl->q_full, 0);
  uint32_t x = 0, i = 0;                           // pieces, tiles
  bool ok = true;
  WidePiece piece;
  while (ok && walk.next(piece)) {
    pages.begin(piece);
    auto load_q = [&] {
      uint8_t* q = smem + kOffQ;
      const int row = piece.row0 + (int)rank * 64;
      tc::remote_arrive_expect_tx(q_bar, kQBytes);
      for (int c = 0; c < 4; ++c)
        tc::tma_load_2d_pair(q + c * kQChunk, tm_q, q_bar, c * 128, row);
      tc::tma_load_2d_pair(q + 4 * kQChunk, tm_qr, q_bar, 512, row);
    };
    // While the first page ids are under way. Failure-detection test: never, in CTA 0.
    if (x == 0 && lane == 0 && !(TEST && blockIdx.x == 0)) load_q();
    __syncwarp();
    for (int t = 0; ok && t < piece.count; ++t, ++i) {
      const int st = i & 1;
      const uint32_t ph = ((i >> 1) - 1) & 1;
      const int cur = pages.take(t + 1 < piece.count, true);
      const int p0 = __shfl_sync(0xffffffffu, cur, 2 * rank);
      const int p1 = __shfl_sync(0xffffffffu, cur, 2 * rank + 1);
      if (lane == 0) {
        const uint32_t bar = tc::map_rank(&ctl->k_full[st], 0);
        const uint32_t bar2 = tc::map_rank(&ctl->k_band[st][0], 0);
        const uint32_t bar3 = tc::map_rank(&ctl->k_band[st][1], 0);
        const uint32_t live = (p0 >= 0) + (p1 >= 0);
        uint8_t* stage = smem + st * kStageBytes;
        if (i >= 2) ok = w_wait<TEST>(&ctl->pv_first[st], ph, ctl, a);
        auto band = [&](int c, uint32_t to) {
          for (int h = 0; h < 2; ++h)
            if ((h ? p1 : p0) >= 0)
              tc::tma_load_2d_pair(stage + c * kChunkBytes + h * (kChunkBytes / 2), tm_kv, to,
                                   c * 128, (h ? p1 : p0) * kPage);
        };
        if (ok) {
          tc::remote_arrive_expect_tx(bar, live * (kPage * (2 * 128 + 64)));
          tc::remote_arrive_expect_tx(bar2, live * (kPage * 128));
          tc::remote_arrive_expect_tx(bar3, live * (kPage * 128));
          band(0, bar);
          for (int h = 0; h < 2; ++h)
            if ((h ? p1 : p0) >= 0)
              tc::tma_load_2d_pair(stage + 4 * kChunkBytes + h * (kRopeBytes / 2), tm_kvr, bar, 512,
                                   (h ? p1 : p0) * kPage);
        }
        if (ok && t == 0 && x > 0) {
          ok = w_wait<TEST>(&ctl->q_empty, (x - 1) & 1, ctl, a);
          if (ok) load_q();
        }
        if (ok && i >= 2) ok = w_wait<TEST>(&ctl->pv_half[st], ph, ctl, a);
        if (ok) band(1, bar);
        if (ok && i >= 2) ok = w_wait<TEST>(&ctl->pv_most[st], ph, ctl, a);
        if (ok) band(2, bar2);
        if (ok && i >= 2) ok = w_wait<TEST>(&ctl->pv_done[st], ph, ctl, a);
        if (ok) band(3, bar3);
      }
      ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
    }
    ++x;
  }
}

// Whether keys of the piece's tile t lie past the end.
__device__ __forceinline__ bool ragged(const WidePiece& p, int t) {
  return (long long)(p.tile + t + 1) * kKeys > p.len;
}

// The other CTA's keys of the own value dims, over the bands S is done with. Where
// the softmax clears V behind the last key, that must have landed here before
// rank 0 hears of it.
template <bool TEST>
__device__ void load_values(const WideArgs& a, WideWalk walk, uint8_t* smem, WideCtl* ctl,
                            uint32_t rank, const CUtensorMap* tm_kv) {
  const int lane = threadIdx.x & 31;
  const uint32_t other = 1 - rank;
  Pages pages(a);
  uint32_t tails = 0, i = 0;                       // parity of each stage's tails so far; tiles
  bool ok = true;
  WidePiece piece;
  while (ok && walk.next(piece)) {
    pages.begin(piece);
    for (int t = 0; ok && t < piece.count; ++t, ++i) {
      const int st = i & 1;
      const int cur = pages.take(t + 1 < piece.count, false);
      const int p0 = __shfl_sync(0xffffffffu, cur, 2 * other);
      const int p1 = __shfl_sync(0xffffffffu, cur, 2 * other + 1);
      const bool tail = ragged(piece, t);
      if (lane == 0 && (ok = w_wait<TEST>(&ctl->s_full[st], (i >> 1) & 1, ctl, a))) {
        uint8_t* stage = smem + st * kStageBytes;
        const uint32_t there = tc::map_rank(&ctl->v_full[st], 0);
        const uint32_t bar = tail ? tc::map_rank(&ctl->v_tail[st], rank) : there;
        tc::remote_arrive_expect_tx(bar, ((p0 >= 0) + (p1 >= 0)) * 2 * kPage * 128);
        for (int h = 0; h < 2; ++h)
          for (int d = 0; d < 2; ++d)
            if ((h ? p1 : p0) >= 0)
              tc::tma_load_2d_pair(stage + (2 * other + d) * kChunkBytes + h * (kChunkBytes / 2),
                                   tm_kv, bar, (2 * rank + d) * 128, (h ? p1 : p0) * kPage);
        if (tail) {
          ok = w_wait<TEST>(&ctl->v_tail[st], (tails >> st) & 1, ctl, a);
          tc::remote_arrive(there);
        }
      }
      if (tail) tails ^= 1u << st;
      ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
    }
  }
}

// ---------------------------------------------------------------- MMAs (rank 0)
// S and PV are issued by a thread each: neither waits on the other's inputs.
template <bool TEST>
__device__ __forceinline__ void mma_drain(uint64_t* bar, const WideArgs& a) {
  tc::mma_commit_pair(bar);                        // every MMA done before TMEM is released
  const unsigned long long t0 = tc::globaltimer_ns();
  while (!tc::mbar_try_wait(bar, 0) && tc::globaltimer_ns() - t0 < wait_limit<TEST>(a)) {
  }
}

template <bool TEST>
__device__ void issue_s(const WideArgs& a, WideWalk walk, uint8_t* smem, WideCtl* ctl,
                        uint32_t tmem) {
  const uint32_t s_kv = tc::smem_u32(smem), s_q = tc::smem_u32(smem + kOffQ);
  uint32_t x = 0, i = 0;                           // pieces, tiles
  bool ok = true;
  WidePiece piece;
  while (ok && walk.next(piece)) {
    if (!(ok = w_wait<TEST>(&ctl->q_full, x & 1, ctl, a))) break;     // Q in both CTAs
    ++x;
    for (int t = 0; t < piece.count; ++t, ++i) {
      const int st = i & 1;
      // The S buffer of tile i - 2 is free: the bands were refilled after PV had begun,
      // and no P of a tile is written before every thread of its CTA has read its S (the
      // vote). Bands 2 and 3 follow as PV leaves them; the others' MMAs cover their flight.
      if (!(ok = w_wait<TEST>(&ctl->k_full[st], (i >> 1) & 1, ctl, a))) break;
      tc::fence_after_sync();
      const uint32_t kv = s_kv + st * kStageBytes, d = tmem + kSCol + st * 128;
      auto band = [&](int c) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          tc::mma_f8_pair(d, tc::smem_desc(s_q + c * kQChunk + kk * 32, 16, 1024, tc::kSw128),
                          tc::smem_desc(kv + c * kChunkBytes + kk * 32, 16, 1024, tc::kSw128),
                          kIdescS, (c | kk) != 0);
      };
      band(0);
      band(1);
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
        tc::mma_f8_pair(d, tc::smem_desc(s_q + 4 * kQChunk + kk * 32, 16, 512, tc::kSw64),
                        tc::smem_desc(kv + 4 * kChunkBytes + kk * 32, 16, 512, tc::kSw64), kIdescS,
                        true);
      for (int c = 2; c < 4 && ok; ++c) {
        if (!(ok = w_wait<TEST>(&ctl->k_band[st][c - 2], (i >> 1) & 1, ctl, a))) break;
        tc::fence_after_sync();
        band(c);
      }
      if (!ok) break;
      tc::mma_commit_pair(&ctl->s_full[st]);
    }
    if (ok) tc::mma_commit_pair(&ctl->q_empty);
  }
  mma_drain<TEST>(&ctl->drain[0], a);
}

template <bool TEST>
__device__ void issue_pv(const WideArgs& a, WideWalk walk, uint8_t* smem, WideCtl* ctl,
                         uint32_t tmem) {
  const uint32_t s_kv = tc::smem_u32(smem), s_p = tc::smem_u32(smem + kOffP);
  uint32_t i = 0;
  bool ok = true;
  WidePiece piece;
  while (ok && walk.next(piece)) {
    for (int t = 0; ok && t < piece.count; ++t, ++i) {
      const int st = i & 1;
      ok = w_wait<TEST>(&ctl->v_full[st], (i >> 1) & 1, ctl, a) &&
           w_wait<TEST>(&ctl->p_full[0], i & 1, ctl, a);
      if (!ok) break;
      tc::fence_after_sync();
      const uint32_t kv = s_kv + st * kStageBytes;
      auto product = [&](int kh, int d) {            // CTA kh's keys, dim half d
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint64_t v = tc::smem_desc(kv + (kh * 2 + d) * kChunkBytes + kk * 32 * 128,
                                           kChunkBytes, 1024, tc::kSw128);
          const uint32_t p = s_p + kh * kPChunk + kk * 32;
          tc::mma_f8_pair(tmem + d * 128, tc::smem_desc(p, 16, 1024, tc::kSw128), v, kIdescHi,
                          !(t == 0 && kh == 0 && kk == 0));
          tc::mma_f8_pair(tmem + d * 128, tc::smem_desc(p + 2 * kPChunk, 16, 1024, tc::kSw128), v,
                          kIdescLo, true);
        }
      };
      product(0, 0);
      tc::mma_commit_pair(&ctl->pv_first[st]);
      product(0, 1);
      tc::mma_commit_pair(&ctl->pv_half[st]);
      if (!(ok = w_wait<TEST>(&ctl->p_full[1], i & 1, ctl, a))) break;
      tc::fence_after_sync();
      product(1, 0);
      tc::mma_commit_pair(&ctl->pv_most[st]);
      product(1, 1);
      tc::mma_commit_pair(&ctl->pv_done[st]);
    }
  }
  mma_drain<TEST>(&ctl->drain[1], a);
}

// ---------------------------------------------------------------- softmax
// p - h for an FP16 h, in FP32.
__device__ __forceinline__ float less_f16(float p, uint16_t h) {
  float r;
  asm("fma.rn.f32.f16 %0, %1, %2, %3;" : "=f"(r) : "h"(h), "h"((uint16_t)0xbc00), "f"(p));
  return r;
}
__device__ __forceinline__ uint16_t f32x2_to_e5m2x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// P of 32 keys of a row from their scores: the codes of both terms and the sum.
// Returns whether they sum to more than 2^8: the tile is then done again.
__device__ __forceinline__ bool weigh(const uint32_t (&raw)[32], float scale, float neg_max,
                                      float& sum, uint32_t (&hi)[8], uint32_t (&lo)[8]) {
  const uint64_t scale2 = pack_f32x2(scale, scale), neg2 = pack_f32x2(neg_max, neg_max);
  uint64_t sums[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    uint64_t d01 = pack_f32x2(__uint_as_float(raw[i]), __uint_as_float(raw[i + 1]));
    uint64_t d23 = pack_f32x2(__uint_as_float(raw[i + 2]), __uint_as_float(raw[i + 3]));
    d01 = fma_f32x2(d01, scale2, neg2);
    d23 = fma_f32x2(d23, scale2, neg2);
    float p[4];
    unpack_f32x2(d01, p[0], p[1]);
    unpack_f32x2(d23, p[2], p[3]);
#pragma unroll
    for (int u = 0; u < 4; ++u) p[u] = ex2(p[u]);
    sums[0] = add_f32x2(sums[0], pack_f32x2(p[0], p[1]));
    sums[1] = add_f32x2(sums[1], pack_f32x2(p[2], p[3]));
    const uint16_t e01 = f32x2_to_e4m3x2(p[0], p[1]), e23 = f32x2_to_e4m3x2(p[2], p[3]);
    const uint32_t h01 = e4m3x2_to_f16x2(e01), h23 = e4m3x2_to_f16x2(e23);
    const uint16_t l01 = f32x2_to_e5m2x2(less_f16(p[0], (uint16_t)h01),
                                         less_f16(p[1], (uint16_t)(h01 >> 16)));
    const uint16_t l23 = f32x2_to_e5m2x2(less_f16(p[2], (uint16_t)h23),
                                         less_f16(p[3], (uint16_t)(h23 >> 16)));
    hi[i / 4] = (uint32_t)e01 | ((uint32_t)e23 << 16);
    lo[i / 4] = (uint32_t)l01 | ((uint32_t)l23 << 16);
  }
  float a, b;
  unpack_f32x2(add_f32x2(sums[0], sums[1]), a, b);
  sum = a + b;
  return sum > 256.f;
}

// Thread (row, 32 keys): TMEM lane l holds row l % 64, keys of CTA l / 64; the
// four warps of a lane quarter take 32 of its columns each. A thread that gave up
// a wait goes on through the barriers, so that every thread reaches each of
// them, until the next vote has all of them leave.
template <bool TEST>
__device__ void softmax(const WideArgs& a, WideWalk walk, uint8_t* smem, WideCtl* ctl,
                        uint32_t tmem, uint32_t rank) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, group = (warp - 4) >> 2;
  const int row = (quarter & 1) * 32 + lane, kh = quarter >> 1;
  const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
  const int col0 = group * 32;                     // of S: keys; of a half of O: dims
  float* const mine = &ctl->red[kh * 4 + group][row];
  uint32_t tails = 0, g = 0;                       // parity of each stage's tails so far; tiles
  bool ok = true;                                  // warp-uniform
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const bool got = ok && w_wait<TEST>(bar, parity, ctl, a);
    ok = __all_sync(0xffffffffu, got);
  };
  // The eight threads' values of this row, joined.
  auto row_max = [&](float v) {
    *mine = v;
    soft_sync();
    for (int j = 0; j < 8; ++j) v = fmaxf(v, ctl->red[j][row]);
    return v;
  };
  auto row_sum = [&](float v) {
    *mine = v;
    soft_sync();
    v = 0.f;
    for (int j = 0; j < 8; ++j) v += ctl->red[j][row];
    return v;
  };
  WidePiece piece;
  while (walk.next(piece)) {
    float m = -INFINITY, l = 0.f;                  // the row's max; this thread's share of its sum
    for (int t = 0; t < piece.count; ++t, ++g) {
      const int st = g & 1;
      const uint32_t ph = (g >> 1) & 1;
      const int key0 = (piece.tile + t) * kKeys;
      const bool tail = ragged(piece, t);
      wait(&ctl->s_full[st], ph);
      tc::fence_after_sync();
      uint32_t raw[32], hi[8], lo[8];
      tc::tmem_ld32(tmem + lanes + kSCol + st * 128 + col0, raw);
      tc::tmem_wait_ld();
      if (tail) {                                  // keys past the end
        const int left = piece.len - (key0 + kh * 128 + col0);
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i >= left) raw[i] = 0xff800000u;     // -inf
      }
      float sum;
      bool moved = t == 0;
      if (t > 0) {
        const bool over = weigh(raw, a.bmm1_log2, m == -INFINITY ? 0.f : -m, sum, hi, lo);
        if (soft_any(over || !ok)) {
          if (soft_any(!ok)) return;               // all of them
          moved = true;
        }
      }
      if (moved) {
        // Rows whose max grew by more than 3 (or begin; 32 weights that sum to more
        // than 2^8 hold one above 2^3): the new max is 2 below the tile's; the sum and
        // O follow.
        float v = -INFINITY;
#pragma unroll
        for (int i = 0; i < 32; ++i) v = fmaxf(v, __uint_as_float(raw[i]) * a.bmm1_log2);
        const float tm = row_max(v);
        const float mn = tm > m + 3.f ? tm - dec::kMaxLead : m;
        const float f = m == -INFINITY ? 0.f : ex2(m - mn);
        m = mn;
        l *= f;
        if (t > 0) {
          wait(&ctl->pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1);
          tc::fence_after_sync();
#pragma unroll 1
          for (int d = 0; d < 2; ++d) {
            uint32_t o[32];
            const uint32_t at = tmem + lanes + d * 128 + col0;
            tc::tmem_ld32(at, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tc::tmem_st32(at, o);
          }
          tc::tmem_wait_st();
          tc::fence_before_sync();
        }
        soft_sync();                               // O is scaled before any P of this CTA counts
        weigh(raw, a.bmm1_log2, m == -INFINITY ? 0.f : -m, sum, hi, lo);
      }
      l += sum;
      // P of these keys is free once PV of the previous tile is done with it.
      if (g > 0)
        wait(kh == 0 ? &ctl->pv_half[(g - 1) & 1] : &ctl->pv_done[(g - 1) & 1],
             ((g - 1) >> 1) & 1);
      // Rows of 128 bytes (128 keys) in 16-byte pieces, piece j of row r at j ^ (r & 7).
      uint8_t* p = smem + kOffP + kh * kPChunk + row * 128;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int at = ((group * 2 + j) ^ (row & 7)) << 4;
        *reinterpret_cast<uint4*>(p + at) =
            make_uint4(hi[4 * j], hi[4 * j + 1], hi[4 * j + 2], hi[4 * j + 3]);
        *reinterpret_cast<uint4*>(p + 2 * kPChunk + at) =
            make_uint4(lo[4 * j], lo[4 * j + 1], lo[4 * j + 2], lo[4 * j + 3]);
      }
      if (tail) {
        // V behind the last key must be finite (0): 256 keys x this CTA's 256 dims,
        // half a band row per thread.
        wait(&ctl->v_tail[st], (tails >> st) & 1);
        for (int z = threadIdx.x - 128; z < kKeys * 2; z += kSoft) {
          const int key = z >> 1, slot = (key >> 7) * 2 + (z & 1);
          if (key0 + key >= piece.len) {
            uint4* v = reinterpret_cast<uint4*>(smem + st * kStageBytes + slot * kChunkBytes +
                                                (key & 127) * 128);
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = make_uint4(0, 0, 0, 0);
          }
        }
        tails ^= 1u << st;
      }
      tc::fence_proxy_async_smem();
      tc::fence_before_sync();
      if (tail) soft_sync();                       // V is clear before any P of this CTA counts
      __syncwarp();
      if (lane == 0) tc::remote_arrive(tc::map_rank(&ctl->p_full[kh], 0));
    }
    // The row's sum, its LSE, and the row itself.
    soft_sync();                                   // red[] is free
    const float z = row_sum(l);
    const float inv = z > 0.f ? 1.f / z : 0.f;
    const size_t first_row = (size_t)piece.slot + rank * 64;
    const int live = min(64, piece.row_end - piece.row0 - (int)rank * 64);
    if (row < live && kh == 0 && group == 0)
      a.part_lse[first_row + row] = z == 0.f ? -INFINITY : m + __log2f(z);
    wait(&ctl->pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1);
    tc::fence_after_sync();
    // Through 2 KB of P's place per warp, 16 of its rows of 128 bytes at a time: lane l
    // then stores 16-byte piece l % 8 of rows l / 8, l / 8 + 4, ..., whole lines. Piece c
    // of row r lies at c ^ (r & 7).
    float4* const stage = reinterpret_cast<float4*>(smem + kOffP) + (warp - 4) * 128;
    float* const dst = a.part_o + (first_row + (quarter & 1) * 32 + (lane >> 3)) * kDv + kh * 256 +
                       col0 + (lane & 7) * 4;
    const int rows = live - (quarter & 1) * 32 - (lane >> 3);      // of this lane, 4 apart
    if ((quarter & 1) * 32 < live) {               // else: a warp without live rows
#pragma unroll 1
      for (int d = 0; d < 2; ++d) {
        uint32_t o[32];
        tc::tmem_ld32(tmem + lanes + d * 128 + col0, o);
        tc::tmem_wait_ld();
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
          if (lane >> 4 == pass) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              stage[(lane & 15) * 8 + (j ^ (lane & 7))] =
                  make_float4(__uint_as_float(o[4 * j]) * inv, __uint_as_float(o[4 * j + 1]) * inv,
                              __uint_as_float(o[4 * j + 2]) * inv,
                              __uint_as_float(o[4 * j + 3]) * inv);
          }
          __syncwarp();
          float4 v[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int r = (lane >> 3) + 4 * u;
            v[u] = stage[r * 8 + ((lane & 7) ^ (r & 7))];
          }
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (pass * 16 + 4 * u < rows)
              *reinterpret_cast<float4*>(dst + (pass * 16 + 4 * u) * kDv + d * 128) = v[u];
          __syncwarp();
        }
      }
    }
    soft_sync();                                   // P's place and O are free
    tc::fence_before_sync();
  }
}

template <bool TEST>
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
      tc::mbar_init(&ctl->k_band[b][0], 2);
      tc::mbar_init(&ctl->k_band[b][1], 2);
      tc::mbar_init(&ctl->v_full[b], 2);
      tc::mbar_init(&ctl->v_tail[b], 1);
      tc::mbar_init(&ctl->s_full[b], 1);
      tc::mbar_init(&ctl->p_full[b], 2 * kSoft / 64);   // the warps of one key half, both CTAs
      tc::mbar_init(&ctl->pv_first[b], 1);
      tc::mbar_init(&ctl->pv_half[b], 1);
      tc::mbar_init(&ctl->pv_most[b], 1);
      tc::mbar_init(&ctl->pv_done[b], 1);
      tc::mbar_init(&ctl->drain[b], 1);
    }
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
  int32_t* plan = reinterpret_cast<int32_t*>(smem + kOffPlan);
  int32_t* lens = plan + kMaxR + 1;
  const int prefix_len = *a.prefix_len;
  bool cut = blockIdx.x == 0 && threadIdx.x == 0 && prefix_len > (long long)a.prefix_pages * kPage;
  const int begin = a.plan[0];
  int flaw = threadIdx.x == 0 ? wide_ends_flaw(begin, a.plan[a.R], a.own_most) : 0;
  for (int i = threadIdx.x; i < a.R; i += kThreads) {
    const int first = i > 0 ? a.plan[i] : 0, after = a.plan[i + 1], len = a.seq_lens[i];
    plan[i + 1] = after;
    lens[i] = wide_len(len, a.max_pages);
    cut |= blockIdx.x == 0 && len > lens[i] && len > 0;
    flaw |= wide_flaw(first, after, lens[i], a.own_blocks, a.own_tiles);
  }
  if (threadIdx.x == 0) plan[0] = 0;
  if (cut && a.status) atomicOr(a.status, MLA_FAULT_PAGE_RANGE);
  if ((flaw & kPlanNone) && blockIdx.x == 0 && a.status) atomicOr(a.status, MLA_FAULT_WORK_ITEM);
  flaw = __syncthreads_or(flaw);
  // Other CTAs may read the word before or after: 0 and kPlanAnew are one to them. A word
  // that is neither stays, so that all of them see it.
  if (blockIdx.x == 0 && threadIdx.x == 0 && begin == (flaw ? 0 : kPlanAnew))
    a.plan[0] = flaw ? kPlanAnew : 0;
  if (flaw) {                          // a scan that takes few registers: unrolled, the tiles' loops
    if (warp == 0) {                   // of the whole kernel took 1 - 2 % longer
      int sum = 0;
#pragma unroll 1
      for (int base = 0; base < a.R; base += 32) {
        int v = base + lane < a.R ? wide_places(lens[base + lane], a.own_blocks) : 0;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
          const int t = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v += t;
        }
        if (base + lane < a.R) plan[base + lane + 1] = sum + v;
        sum += __shfl_sync(0xffffffffu, v, 31);
      }
    }
    __syncthreads();
  }
  const WideWalk walk(a, plan, lens, prefix_len, (int)(blockIdx.x >> 1));
  if (walk.pos >= walk.end) {
    // Nothing for this pair.
  } else if (warp == 0) {
    load_keys<TEST>(a, walk, smem, ctl, rank, &tm_kv, &tm_kvr, &tm_q, &tm_qr);
  } else if (warp == 3) {
    load_values<TEST>(a, walk, smem, ctl, rank, &tm_kv);
  } else if (warp >= 4) {
    softmax<TEST>(a, walk, smem, ctl, tmem, rank);
  } else if (rank == 0 && lane == 0) {
    if (warp == 1)
      issue_s<TEST>(a, walk, smem, ctl, tmem);
    else
      issue_pv<TEST>(a, walk, smem, ctl, tmem);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (ctl->abort_flag)     // a wait ran out: what is still in flight here or to the other CTA lands
    for (const unsigned long long t0 = tc::globaltimer_ns(); tc::globaltimer_ns() - t0 < 1000000;) {
    }
  tc::cluster_sync();      // no CTA leaves while the other's MMAs or arrivals may reach it
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
  static bool attr_set[2][64] = {};
  const bool test = a.wait_limit_ns != 0;
  auto* kernel = test ? wide_kernel<true> : wide_kernel<false>;
  cudaError_t e = dec::set_smem(kernel, kSmemBytes, attr_set[test]);
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
  return cudaLaunchKernelEx(&cfg, kernel, a, tkv, tkvr, tq, tqr);
}

}  // namespace mlafold
