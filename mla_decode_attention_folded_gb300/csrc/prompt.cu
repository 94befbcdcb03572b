// Attention over whole prompts, packed: the expanded form of the latent attention.
//
//   s[i][h][j] = sm_scale (q[i][h][0:128] . k_nope[j][h / G] + q[i][h][128:192] . k_rope[j])
//   out[i][h]  = softmax_j(s[i][h]) v[j][h / G],   lse[i][h] = log2 sum_j 2^(s log2 e)
//
// over the keys j of token i's request that it sees (causal: up to its own place, counted
// from the end). The rope dims of a key are one vector for all heads.
//
// Bound by the BF16 tensor pipe: 640 FLOP per (query, key, head) against 644 bytes per (query,
// head). A pair of CTAs takes 512 query rows of one head as two halves of 256, each the M of
// its MMAs (cta_group::2: 128 rows in each CTA): while the softmax of one half runs, the tensor
// pipe multiplies for the other.
//   S[256, 128 keys] = Q K^T, 12 MMAs;  O[256, 128] += P V, 8 MMAs, P from TMEM.
// Requests of up to 256 rows would leave a half empty: theirs are the rows of two heads, on the same
// keys (grouped heads) or on tiles of K and V that come by turns, one for each half.
//
// Each CTA loads half of a tile of K (64 keys) and of V (64 dims), 40 KB: three tiles are in
// flight where a CTA on its own has room for little more than one, and waits for it (64 heads of
// 8k tokens: 1130 us by single CTAs, 942 by pairs). TMEM holds both halves' S and O (4 x 128
// columns); P (BF16) takes the place of the S it was made from.
// Warp 0 loads by TMA; warps 1 and 2 of the first CTA issue the halves' MMAs (one warp for both:
// 1320 us, 1172 with two); warp 3 tells them that V is there, and clears what lies behind a
// request's last key; eight warps each are the softmax of the halves: two threads to a row, 64 keys
// each (1172 -> 1130 us). The maximum that P is relative to moves only when a score exceeds it by
// 2^8 (O and the sum are then rescaled), so that the two threads need no more than a barrier's vote
// in most tiles; P leaves in two halves, the first multiplied while the second is made (117 -> 112 us for
// the grouped prompts below); P is rounded to BF16 (2^-8, as the inputs are), its sum is of the FP32 values.
// Registers are short (96 a thread): a few words that the loading warp or a softmax thread spills cost 1
// to 5 %. So the loading warp makes its plan again for each piece and leaves the next one in shared
// memory, the softmax keeps little of a piece and rescales O eight columns at a time.
//
// How the work is shared out is in prompt.h. The order of a half's MMAs is PV(t) before S(t + 1),
// so that S may overwrite P and its completion tells that O is final.
//
// Measured (graph replays; in brackets with L2 flushed before each call): 64 heads of 8,192 tokens 867 to
// 926 us (885), 1,485 to 1,585 TFLOP/s (the pipe's peak in a burst is 1,874, and 1,690 under the power
// cap); 4 x 32 heads of 900 to 1,500 tokens, grouped, without a mask 112 us (116), 1,088 TFLOP/s; 24
// prompts of up to 2,048 tokens and 8 heads 122 us (125), 720; 512 tokens on 16k keys, 8 heads 42.6 to
// 43.6 us (46.7), 990; two short prompts 8.5 us (10.6).
// Dropped: V given back after S (1130 -> 1258 us); the MMAs' lock before the wait for P (912 -> 963);
// weights made while the vote on the maximum runs (935 -> 1016); masks per 32 columns (spills, 916
// -> 1173); registers moved from the four first warps to the softmax (24 prompts 128 -> 136 us, again
// 122 -> 135 at the end); votes by the two warps that share rows instead of a half's eight (equal).
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "checks.h"
#include "decode_common.cuh"
#include "formats.cuh"
#include "internal.h"
#include "pair.cuh"
#include "prompt.h"
#include "ptx.cuh"
#include "tc.cuh"

namespace mlafold {
namespace {

using namespace prompt;

constexpr int kNope = 128, kRope = 64, kV = 128;
constexpr int kBlock = 128 * 128;                // bytes: 128 rows of 64 BF16
constexpr int kQBlocks = 3;                      // 192 dims
constexpr int kMine = 128;                       // a CTA's rows of a half
constexpr int kStages = 3;                       // tiles of K and of V in flight
constexpr int kKBlock = 64 * 128, kKBytes = 3 * kKBlock;   // 64 keys of 64 dims; 192 dims
constexpr int kVBytes = kBlock;                  // 128 keys of 64 dims
constexpr int kOffK = 2 * kQBlocks * kBlock;
constexpr int kOffV = kOffK + kStages * kKBytes;
constexpr int kOffCtl = kOffV + kStages * kVBytes;
constexpr int kSoft = 256;                       // softmax threads of a half: two to a row
constexpr int kThreads = 128 + 2 * kSoft;
constexpr uint32_t kTmemCols = 512, kColO = 256;
constexpr unsigned long long kWaitLimitNs = 2000000000ull;   // 2 s
constexpr uint32_t kIdescS = tc::idesc_bf16_f32(kHalf, kKeys);   // M = 256 over the pair
constexpr uint32_t kIdescO = tc::idesc_bf16_f32(kHalf, kV) | (1u << 16);   // V is MN-major
constexpr float kLazy = 8.f;
constexpr float kLowest = -FLT_MAX;               // a piece's LSE: keys seen, all scores -infinity

// A run of tiles of one item.
struct Piece {
  int row0, rows;                // first query row (of all), rows of the item
  int head, key0, m;             // head, first key (of all), keys of the request
  int lim0;                      // keys that row 0 would see, before it is cut to 0 .. m
  int t0, t1;                    // tiles, t1 <= what the last row sees
  int slot;                      // of its FP32 rows; -1: the whole item, straight to out
  int causal;
  int twin;                      // 1: the halves are the rows of head and head + 1; 2: of K and V each
};
// First of the item's rows in half h.
__device__ __forceinline__ int half_row(const Piece& p, int h) { return p.twin ? 0 : h * kHalf; }
__device__ __forceinline__ int row_limit(const Piece& p, int j) {
  const int e = p.causal ? p.lim0 + j : p.m;
  return e < 0 ? 0 : e < p.m ? e : p.m;
}
// Tiles of the piece that half h multiplies.
__device__ __forceinline__ int half_tiles(const Piece& p, int h) {
  const int row = half_row(p, h), rows = min(p.rows - row, kHalf);
  if (rows <= 0) return 0;
  const int last = tiles_of(row_limit(p, row + rows - 1));
  return max(min(p.t1, last) - p.t0, 0);
}

// The pair's barriers: those that MMAs wait for count on the first CTA, those that MMAs arrive on
// in both.
struct PromptCtl {
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[kStages], k_empty[kStages];
  uint64_t v_land[kStages];      // this CTA's copies of V
  uint64_t v_full[kStages], v_empty[kStages];
  uint64_t s_full[2], p_half[2], p_full[2], o_full[2];
  uint64_t job_full[2], job_empty[2];
  uint64_t claim_full[2], claim_empty[2];   // first CTA -> second: claimed items; and back
  uint64_t drain[2];
  Piece job[2];
  Piece staged;                  // the loading warp's: the next one
  long long claim[2];
  float row[2][kMine];           // [half][row]: what the two threads of a row tell one another
  // Values that are no numbers (below): by piece and dim, (piece + 1, ~ the first such key). Four
  // pieces' worth: who notes them waits until both CTAs' softmaxes have done with the fourth before.
  unsigned long long bad[4][2][kV];   // [][half]
  uint32_t bad_piece[4];         // piece + 1, where there are any
  uint32_t v_piece;              // the other CTA's: pieces that its V warp has taken
  uint32_t tmem_base;
  uint32_t lock;                 // held by the half whose MMAs are being issued
  int abort_flag;
};
constexpr int kSmemBytes = kOffCtl + (int)sizeof(PromptCtl) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

struct PromptArgs {
  const int32_t* cu;             // [R + 1]
  const int32_t* cu_keys;        // [R + 1], or null: cu
  uint16_t* out;                 // [T][H][128]
  float* lse;                    // [T][H], or null
  Plan* plan;
  long long* first_place;        // [R + 1]
  long long* first_item;         // [R + 1]
  Join* joins;                   // [pairs]
  float* part_o;                 // [slots][32][512][4]
  float* part_lse;               // [slots][512]
  int32_t* status;
  float scale_log2;
  int R, T, Tk, H, group, causal, pairs;
  int twins;                     // short requests have two heads to an item
  int planned;                   // the plan kernel has run; else every CTA plans for itself (R <= 32)
  unsigned long long wait_limit_ns;
  int withhold;                  // failure-detection test: CTA 0 never loads its first keys
};

// Rows [first, first + count) of request r; offsets that are none give no rows.
__device__ __forceinline__ bool span(const int32_t* cu, int r, int most, int& first, int& count) {
  const int a = cu[r], b = cu[r + 1];
  const bool ok = a >= 0 && b >= a && b <= most;
  first = ok ? a : 0;
  count = ok ? b - a : 0;
  return ok;
}
__device__ __forceinline__ Request request(const PromptArgs& a, int r, int& row0, int& key0, bool& ok) {
  Request q;
  ok = span(a.cu, r, a.T, row0, q.n);
  ok = span(a.cu_keys ? a.cu_keys : a.cu, r, a.Tk, key0, q.m) && ok;
  if (!ok) q.n = q.m = 0;
  q.causal = a.causal;
  return q;
}

// ---------------------------------------------------------------- plan
constexpr int kPlanThreads = kMaxR;

__global__ void __launch_bounds__(kPlanThreads) prompt_plan_kernel(const PromptArgs a) {
  __shared__ long long sums[2][32];
  __shared__ int most[32];
  const int r = threadIdx.x, lane = r & 31, warp = r >> 5;
  grid_dep_wait();
  grid_dep_launch();
  int row0, key0, longest = 0;
  long long w = 0, it = 0;
  if (r < a.R) {
    bool ok;
    const Request q = request(a, r, row0, key0, ok);
    if (!ok && a.status) atomicOr(a.status, MLA_FAULT_WORK_ITEM);
    const int I = items(q);
    w = places(q) * units(q, a.H, a.twins);
    it = (long long)I * units(q, a.H, a.twins);
    if (I) longest = max(item_tiles(q, I - 1), I > 1 ? item_tiles(q, I - 2) : 0);
  }
  long long sw = w, si = it;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, sw, o), v = __shfl_up_sync(0xffffffffu, si, o);
    if (lane >= o) sw += u, si += v;
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 31) sums[0][warp] = sw, sums[1][warp] = si;
  if (lane == 0) most[warp] = longest;
  __syncthreads();
  long long bw = 0, bi = 0, tw = 0, ti = 0;
  for (int i = 0; i < (int)(blockDim.x >> 5); ++i) {
    if (i < warp) bw += sums[0][i], bi += sums[1][i];
    tw += sums[0][i], ti += sums[1][i];
    longest = max(longest, most[i]);
  }
  if (r < a.R) {
    a.first_place[r] = bw + sw - w;
    a.first_item[r] = bi + si - it;
  }
  if (r == 0) {
    a.first_place[a.R] = tw;
    a.first_item[a.R] = ti;
    a.plan->total = tw;
    a.plan->all_items = ti;
    const bool whole = whole_items(tw, longest, a.pairs);
    const long long len = whole ? 0 : cdiv(tw, parts_of(tw, a.pairs));
    a.plan->len = len;
    a.plan->parts = whole ? 0 : (int)cdiv(tw, len);
    a.plan->claimed = 0;
  }
}

// The last r with first[r] <= x, by a warp.
__device__ __forceinline__ int find_request(const long long* first, int R, long long x, int lane) {
  int lo = 0, n = R;
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const bool le = lane * step < n && first[lo + lane * step] <= x;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int hit = m ? 31 - __clz(m) : 0, end = lo + n;
    lo += hit * step;
    n = min(step, end - lo);
  }
  return lo;
}

// ---------------------------------------------------------------- attention
__device__ __forceinline__ bool pr_wait(uint64_t* bar, uint32_t parity, PromptCtl* ctl,
                                        const PromptArgs& a) {
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
// The same for what the other CTA's threads wrote.
__device__ __forceinline__ bool pr_wait_pair(uint64_t* bar, uint32_t parity, PromptCtl* ctl,
                                             const PromptArgs& a) {
  const unsigned long long t0 = tc::globaltimer_ns();
  while (true) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(done)
        : "r"(tc::smem_u32(bar)), "r"(parity)
        : "memory");
    if (done) return true;
    if (*reinterpret_cast<volatile int*>(&ctl->abort_flag)) return false;
    if (tc::globaltimer_ns() - t0 > a.wait_limit_ns) {
      *reinterpret_cast<volatile int*>(&ctl->abort_flag) = 1;
      if (a.status) atomicOr(a.status, MLA_FAULT_WAIT_TIMEOUT);
      return false;
    }
  }
}
// Until the other CTA's V warp has taken `pieces` of them.
__device__ __forceinline__ bool wait_v_piece(PromptCtl* ctl, uint32_t pieces, const PromptArgs& a) {
  const unsigned long long t0 = tc::globaltimer_ns();
  while (true) {
    uint32_t v;
    asm volatile("ld.acquire.cluster.shared::cta.u32 %0, [%1];"
                 : "=r"(v)
                 : "r"(tc::smem_u32(&ctl->v_piece))
                 : "memory");
    if (v >= pieces) return true;
    if (*reinterpret_cast<volatile int*>(&ctl->abort_flag)) return false;
    if (tc::globaltimer_ns() - t0 > a.wait_limit_ns) {
      *reinterpret_cast<volatile int*>(&ctl->abort_flag) = 1;
      if (a.status) atomicOr(a.status, MLA_FAULT_WAIT_TIMEOUT);
      return false;
    }
  }
}
// The next piece, for a whole warp; false at the end, or where the wait ran out.
__device__ __forceinline__ bool take(PromptCtl* ctl, uint32_t seq, const PromptArgs& a, Piece& p, bool read) {
  const int b = seq & 1;
  if (!__all_sync(0xffffffffu, pr_wait(&ctl->job_full[b], (seq >> 1) & 1, ctl, a))) return false;
  p = ctl->job[b];
  __syncwarp();
  if (read) tc::mbar_arrive(&ctl->job_empty[b]);
  return p.rows > 0;
}
// One half's MMAs at a time.
__device__ __forceinline__ bool lock(PromptCtl* ctl, const PromptArgs& a) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (atomicCAS(&ctl->lock, 0u, 1u) == 0) return true;
  const unsigned long long t0 = tc::globaltimer_ns();
  while (atomicCAS(&ctl->lock, 0u, 1u) != 0) {
    if (*reinterpret_cast<volatile int*>(&ctl->abort_flag)) return false;
    if (tc::globaltimer_ns() - t0 > a.wait_limit_ns) {
      *reinterpret_cast<volatile int*>(&ctl->abort_flag) = 1;
      if (a.status) atomicOr(a.status, MLA_FAULT_WAIT_TIMEOUT);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ void unlock(PromptCtl* ctl) { atomicExch(&ctl->lock, 0u); }
// One lane of a whole warp, always the same.
__device__ __forceinline__ bool elect() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void mma_bf16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                              uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_bf16_ts_pair(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                                 uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* m, uint32_t bar, int x,
                                                 int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// A barrier of a half's softmax threads; whether any of them, or all, say so.
__device__ __forceinline__ bool half_any(int h, bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
      " barrier.cta.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(1 + h), "n"(kSoft)
      : "memory");
  return r != 0;
}
// 32 bytes, a sector of its own, at a 32-byte boundary.
__device__ __forceinline__ void st_32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ uint32_t f32x2_to_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
               : "memory");
}
// 1 / x to 2^-23, beside the 2^-8 of the BF16 that it scales: the exact division is a call, for which
// the softmax threads would have to spare registers.
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
prompt_kernel(const PromptArgs a, const __grid_constant__ CUtensorMap tm_q,
              const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_r,
              const __grid_constant__ CUtensorMap tm_v) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  PromptCtl* ctl = reinterpret_cast<PromptCtl*>(smem + kOffCtl);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = tc::cluster_rank();
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&ctl->q_full[i], 2);
      tc::mbar_init(&ctl->q_empty[i], 1);
      tc::mbar_init(&ctl->s_full[i], 1);
      tc::mbar_init(&ctl->p_half[i], 2 * kSoft / 32);
      tc::mbar_init(&ctl->p_full[i], 2 * kSoft / 32);
      tc::mbar_init(&ctl->o_full[i], 1);
      tc::mbar_init(&ctl->job_full[i], 1);
      tc::mbar_init(&ctl->job_empty[i], (rank ? 1 : 3) + 2 * kSoft / 32);
      tc::mbar_init(&ctl->claim_full[i], 1);
      tc::mbar_init(&ctl->claim_empty[i], 1);
      tc::mbar_init(&ctl->drain[i], 1);
    }
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(&ctl->k_full[i], 2);
      tc::mbar_init(&ctl->k_empty[i], 2);
      tc::mbar_init(&ctl->v_land[i], 1);
      tc::mbar_init(&ctl->v_full[i], 2);
      tc::mbar_init(&ctl->v_empty[i], 2);
    }
    ctl->abort_flag = 0;
    ctl->lock = 0;
    for (int i = 0; i < 4; ++i) ctl->bad_piece[i] = 0;
    ctl->v_piece = 0;
    tc::fence_barrier_init();
    tc::prefetch_tmap(&tm_q);
    tc::prefetch_tmap(&tm_k);
    tc::prefetch_tmap(&tm_r);
    tc::prefetch_tmap(&tm_v);
  }
  for (int i = threadIdx.x; i < 4 * 2 * kV; i += kThreads) (&ctl->bad[0][0][0])[i] = 0;
  if (warp == 1) {
    tc::tmem_alloc_pair(&ctl->tmem_base, kTmemCols);
    tc::tmem_relinquish_pair();
  }
  tc::fence_before_sync();
  tc::cluster_sync();            // both CTAs' barriers and TMEM are there
  tc::fence_after_sync();
  const uint32_t tmem = ctl->tmem_base;
  grid_dep_wait();               // the waits' limit counts from the end of the kernel before
  grid_dep_launch();

  if (warp < 4) {
    if (warp == 0) {
      // ------------------------------------------------------------ pieces and copies
      // So far: pieces, tiles, queries of the halves, claims.
      uint32_t seq = 0, n = 0, xq0 = 0, xq1 = 0, claims = 0;
      bool ok = true;
      const int pair = blockIdx.x >> 1;
      const bool withheld = a.withhold && blockIdx.x == 0;
      if (rank == 0 && lane == 0) a.joins[pair].rows = 0;
      // The plan: read, or made here with a request to a lane (and made again for each piece, so that
      // it takes no registers meanwhile).
      struct Lane {
        Request q;
        int row0, key0;
        long long place, item, total, all;       // before this lane's; of all
      };
      auto lanes_plan = [&](Lane& l, bool report) {
        l.q = {0, 0, false};
        l.row0 = l.key0 = 0;
        l.place = l.item = 0;
        if (lane < a.R) {
          bool good;
          l.q = request(a, lane, l.row0, l.key0, good);
          if (report && !good && a.status && blockIdx.x == 0) atomicOr(a.status, MLA_FAULT_WORK_ITEM);
          l.place = places(l.q) * units(l.q, a.H, a.twins);
          l.item = (long long)items(l.q) * units(l.q, a.H, a.twins);
        }
        const long long w = l.place, it = l.item;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long u = __shfl_up_sync(0xffffffffu, l.place, o);
          const long long v = __shfl_up_sync(0xffffffffu, l.item, o);
          if (lane >= o) l.place += u, l.item += v;
        }
        l.total = __shfl_sync(0xffffffffu, l.place, 31);
        l.all = __shfl_sync(0xffffffffu, l.item, 31);
        l.place -= w;
        l.item -= it;
      };
      Lane plan;
      int parts;
      long long total, all, len;
      if (a.planned) {
        total = a.plan->total;
        all = a.plan->all_items;
        parts = a.plan->parts;
        len = a.plan->len;
      } else {
        lanes_plan(plan, true);
        const int I = items(plan.q);
        const int longest = __reduce_max_sync(
            0xffffffffu, I ? max(item_tiles(plan.q, I - 1), I > 1 ? item_tiles(plan.q, I - 2) : 0) : 0);
        total = plan.total;
        all = plan.all;
        const uint32_t t = (uint32_t)total;
        parts = 0;
        len = 0;
        if (t > 0 && !whole_items(total, longest, a.pairs)) {
          const uint32_t aim = min((t + kMinPart - 1) / kMinPart, (uint32_t)a.pairs), l = (t + aim - 1) / aim;
          len = l;
          parts = (int)((t + l - 1) / l);
        }
      }
      // Whole items: the first by the pair's index, then claimed, or by turns where each CTA plans for
      // itself. Parts: places [at, end).
      long long at = pair, end = 0;
      if (parts > 0) {
        at = pair < parts ? part_at(total, len, pair) : 0;
        end = pair < parts ? part_at(total, len, pair + 1) : 0;
      }
      // Queries are loaded as soon as their half's last S of the piece before is done, whatever else
      // the warp waits for: this piece's, then the next one's. All that is lane 0's.
      struct Load {
        int head, row, due;                      // due: bit h: half h's; bit 2: a head for each half
      } cur = {0, 0, 0}, nxt = {0, 0, 0};
      // The piece at `at`, none (no rows) at the end; moves `at` on.
      auto next = [&](auto first_one) {
        Piece p;
        p.rows = 0;
        while (parts > 0 ? at < end : at < all) {
          int row0, u;
          long long x;
          Request q;
          if (a.planned) {
            const long long* first = parts > 0 ? a.first_place : a.first_item;
            const int r = find_request(first, a.R, at, lane);
            bool good;
            q = request(a, r, row0, p.key0, good);
            x = at - first[r];
          } else {
            if (!decltype(first_one)::value) lanes_plan(plan, false);
            const long long first = parts > 0 ? plan.place : plan.item;
            const int r = 31 - __clz(__ballot_sync(0xffffffffu, lane < a.R && first <= at) | 1);
            q.n = __shfl_sync(0xffffffffu, plan.q.n, r);
            q.m = __shfl_sync(0xffffffffu, plan.q.m, r);
            q.causal = a.causal;
            row0 = __shfl_sync(0xffffffffu, plan.row0, r);
            p.key0 = __shfl_sync(0xffffffffu, plan.key0, r);
            x = at - __shfl_sync(0xffffffffu, first, r);
          }
          p.t0 = 0;
          if (parts > 0) {
            const long long per = places(q);
            p.head = head_at(x, per, units(q, a.H, a.twins));
            const long long rest = x - p.head * per;
            u = item_at(q, rest);
            p.t0 = (int)(rest - before(q, u));
          } else {
            claimed_item(q, units(q, a.H, a.twins), 3 * (int)(gridDim.x >> 1), (int)x, p.head, u);
          }
          p.twin = 0;
          if (twins(q, a.twins)) {
            p.head *= 2;
            if (p.head + 1 < a.H) p.twin = p.head / a.group == (p.head + 1) / a.group ? 1 : 2;
          }
          const int tiles = item_tiles(q, u);
          p.t1 = tiles;
          p.slot = -1;
          p.row0 = row0 + u * kRows;
          p.rows = min(q.n - u * kRows, kRows);
          if (parts > 0) {
            const long long left = min(end - at, (long long)(tiles + kExtra - p.t0)), stop = at - p.t0 + tiles;
            at += left;
            if (p.t0 >= tiles) {                   // what an item costs besides its tiles
              p.rows = 0;
              continue;
            }
            p.t1 = (int)min((long long)tiles, p.t0 + left);
            if (p.t0 > 0) {
              p.slot = 2 * pair;
            } else if (p.t1 < tiles) {
              p.slot = 2 * pair + 1;
              int last = pair + 1;
              while (last + 1 < parts && part_at(total, len, last + 1) < stop) ++last;
              if (rank == 0 && lane == 0) a.joins[pair] = {p.row0, p.rows, p.head, last << 1 | (p.twin > 0)};
            }
          }
          p.m = q.m;
          p.causal = q.causal;
          p.lim0 = u * kRows + 1 + q.m - q.n;
          break;
        }
        // It waits in shared memory; what its queries need is kept at hand.
        if (lane == 0) ctl->staged = p;
        Load l = {p.head, p.row0 + (int)rank * kMine, 0};
        if (p.rows > 0) l.due = (half_tiles(p, 0) > 0) | (half_tiles(p, 1) > 0) << 1 | (p.twin > 0) << 2;
        if (decltype(first_one)::value) cur = l;
        else nxt = l;
        __syncwarp();
        if (parts > 0 || p.rows == 0) return;
        if (!a.planned) {
          at += gridDim.x >> 1;
          return;
        }
        // The first CTA claims the item after this and tells the second.
        int got = 1;
        if (lane == 0) {
          const int i = claims & 1;
          const uint32_t phase = claims >> 1 & 1;
          if (rank == 0) {
            at = (long long)(gridDim.x >> 1) + atomicAdd(&a.plan->claimed, 1);
            got = claims < 2 || pr_wait_pair(&ctl->claim_empty[i], phase ^ 1, ctl, a);
            if (got) {
              asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(tc::map_rank(&ctl->claim[i], 1)), "l"(at)
                           : "memory");
              asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                               tc::map_rank(&ctl->claim_full[i], 1))
                           : "memory");
            }
          } else {
            got = pr_wait_pair(&ctl->claim_full[i], phase, ctl, a);
            if (got) {
              at = *reinterpret_cast<volatile long long*>(&ctl->claim[i]);
              asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                               tc::map_rank(&ctl->claim_empty[i], 0))
                           : "memory");
            }
          }
        }
        ++claims;
        at = __shfl_sync(0xffffffffu, at, 0);
        ok = __shfl_sync(0xffffffffu, got, 0) != 0;
      };
      auto load_q = [&](int h, uint32_t& x) {
        const bool now = cur.due >> h & 1;
        if (!now && !(nxt.due >> h & 1)) return;
        if (x > 0 && !tc::mbar_test_wait(&ctl->q_empty[h], (x - 1) & 1)) return;
        int head = now ? cur.head : nxt.head, row = now ? cur.row : nxt.row;
        if (h) {
          if ((now ? cur.due : nxt.due) & 4) ++head;
          else row += kHalf;
        }
        const uint32_t bar = tc::map_rank(&ctl->q_full[h], 0);
        tc::remote_arrive_expect_tx(bar, kQBlocks * kBlock);
#pragma unroll 1
        for (int e = 0; e < kQBlocks; ++e)
          tma_load_3d_pair(smem + (h * kQBlocks + e) * kBlock, &tm_q, bar, e * 128, head, row);
        if (now) cur.due &= ~(1 << h);
        else nxt.due &= ~(1 << h);
        ++x;
      };
      auto load_queries = [&] {
        load_q(0, xq0);
        load_q(1, xq1);
      };
      // Waits for a place in a ring (bar null: for this piece's queries to be asked for).
      auto wait_ring = [&](uint64_t* bar, uint32_t parity) {
        int v = 1;
        if (lane == 0) {
          unsigned long long t0 = 0;
          for (int i = 0;; ++i) {
            if ((cur.due | nxt.due) & 3) load_queries();
            if (bar ? tc::mbar_try_wait(bar, parity) : !(cur.due & 3)) break;
            if (i < 32) continue;
            if (!t0) t0 = tc::globaltimer_ns();
            if (*reinterpret_cast<volatile int*>(&ctl->abort_flag) ||
                tc::globaltimer_ns() - t0 > a.wait_limit_ns) {
              if (atomicExch(&ctl->abort_flag, 1) == 0 && a.status) atomicOr(a.status, MLA_FAULT_WAIT_TIMEOUT);
              v = 0;
              break;
            }
          }
        }
        return __shfl_sync(0xffffffffu, v, 0) != 0;
      };
      next(std::true_type{});
      while (ok) {
        // Hand it on, or an empty one at the end.
        if (seq >= 2 && !(ok = wait_ring(&ctl->job_empty[seq & 1], ((seq >> 1) - 1) & 1))) break;
        const Piece p = ctl->staged;
        __syncwarp();
        if (lane == 0) {
          ctl->job[seq & 1] = p;
          tc::mbar_arrive(&ctl->job_full[seq & 1]);
        }
        if (p.rows == 0) break;
        ++seq;
        // Places of the rings: a tile each, or one for each half.
        const int two = p.twin == 2, nt = max(half_tiles(p, 0), half_tiles(p, 1)) << two;
        const int kvh0 = p.head / a.group, kvh1 = two ? (p.head + 1) / a.group : kvh0;
        const int key0 = p.key0 + p.t0 * kKeys;
#pragma unroll 1
        for (int t = 0; t < nt || t < kStages; ++t) {
          if (t < nt) {
            const int st = n % kStages, key = key0 + (t >> two) * kKeys, kvh = t & two ? kvh1 : kvh0;
            if (n >= kStages && !(ok = wait_ring(&ctl->k_empty[st], (n / kStages - 1) & 1))) break;
            if (lane == 0 && !(withheld && n == 0)) {
              const uint32_t bar = tc::map_rank(&ctl->k_full[st], 0);
              uint8_t* dst = smem + kOffK + st * kKBytes;
              const int mine = key + (int)rank * 64;
              tc::remote_arrive_expect_tx(bar, kKBytes);
              tma_load_3d_pair(dst, &tm_k, bar, 0, kvh, mine);
              tma_load_3d_pair(dst + kKBlock, &tm_k, bar, 128, kvh, mine);
              tc::tma_load_2d_pair(dst + 2 * kKBlock, &tm_r, bar, 0, mine);
            }
            if (lane == 0) load_queries();
            if (n >= kStages && !(ok = wait_ring(&ctl->v_empty[st], (n / kStages - 1) & 1))) break;
            if (lane == 0) {
              tc::mbar_arrive_expect_tx(&ctl->v_land[st], kVBytes);
              tc::tma_load_3d(smem + kOffV + st * kVBytes, &tm_v, &ctl->v_land[st], (int)rank * 128, kvh, key);
            }
            ++n;
          }
          // The next piece is looked up while this one's tiles are multiplied.
          if (t == kStages - 1) {
            next(std::false_type{});
            if (!ok) break;
          }
        }
        if (!ok || !(ok = wait_ring(nullptr, 0))) break;
        cur = nxt;
        nxt.due = 0;
      }
      // Never leave with copies in flight: another role may have given up a wait. V counts here, the
      // pair's K and queries on the first CTA; the CTAs leave together.
      if (lane == 0) {
        const unsigned long long t0 = tc::globaltimer_ns();
        const uint32_t last = ok ? n : n + 1;      // a tile begun when a wait ran out
        for (uint32_t i = n < kStages ? 0 : n - kStages; i < n; ++i)
          while (!tc::mbar_try_wait(&ctl->v_land[i % kStages], (i / kStages) & 1) &&
                 tc::globaltimer_ns() - t0 < a.wait_limit_ns) {
          }
        for (uint32_t i = last < kStages ? 0 : last - kStages; rank == 0 && i < last; ++i)
          while (!tc::mbar_try_wait(&ctl->k_full[i % kStages], (i / kStages) & 1) &&
                 tc::globaltimer_ns() - t0 < a.wait_limit_ns) {
          }
        for (int h = 0; rank == 0 && h < 2; ++h) {
          const uint32_t x = h ? xq1 : xq0;
          while (x > 0 && !tc::mbar_try_wait(&ctl->q_full[h], (x - 1) & 1) &&
                 tc::globaltimer_ns() - t0 < a.wait_limit_ns) {
          }
        }
      }
    } else if (warp <= 2) {
      // ------------------------------------------------------------ MMAs of half h, for both CTAs
      // The whole warp goes through the waits, so that what the MMAs are given is the same in all
      // lanes and stays in uniform registers; one lane issues.
      if (rank == 0) {
        const int h = __shfl_sync(0xffffffffu, warp, 0) - 1;
        const bool one = elect();
        uint32_t n0 = 0, xq = 0, xp = 0;
        const uint32_t s_k = tc::smem_u32(smem + kOffK), s_v = tc::smem_u32(smem + kOffV);
        const uint32_t col_s = tmem + h * kKeys, col_o = tmem + kColO + h * kV;
        const uint64_t qd = tc::smem_desc(tc::smem_u32(smem) + h * kQBlocks * kBlock, 16, 1024, tc::kSw128);
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) { return ok = pr_wait(bar, parity, ctl, a); };
        // What this half does not multiply is given back as it lands: place i of a ring.
        auto give = [&](uint64_t* full, uint64_t* empty, uint32_t i) {
          const uint32_t st = i % kStages;
          if (!wait(full + st, (i / kStages) & 1)) return false;
          if (one) {
            tc::remote_arrive(tc::map_rank(empty + st, 0));
            tc::remote_arrive(tc::map_rank(empty + st, 1));
          }
          return true;
        };
        for (uint32_t seq = 0; ok; ++seq) {
          Piece p;
          if (!take(ctl, seq, a, p, one)) break;
          const int c = __shfl_sync(0xffffffffu, half_tiles(p, h), 0);
          const int two = __shfl_sync(0xffffffffu, p.twin == 2, 0);
          const uint32_t nt = max(c, __shfl_sync(0xffffffffu, half_tiles(p, h ^ 1), 0)) << two;
          // No lane leaves the loop from where only one works, and none waits for the others in it: where a
          // wait runs out they meet behind it.
          // PV of tile t, then S of tile t + 1, under a lock: issued as they come, the halves' MMAs would
          // mingle, both finish late, and both softmaxes then run while the tensor pipe waits. What
          // the copies bring is waited for before P, where it is there by then, so that nothing
          // stands between P and the MMAs.
          auto multiply = [&](auto by_turns) {
            constexpr bool two = decltype(by_turns)::value;
#pragma unroll 1
            for (int t = -1; t < c; ++t) {
              const uint32_t nv = two ? n0 + 2 * t + h : n0 + t, sv = nv % kStages;   // V of tile t
              const uint32_t nk = nv + (two ? 2 : 1), sk = nk % kStages;              // K of tile t + 1
              const bool has_k = t + 1 < c;
              if (t < 0 && c > 0 && !wait(&ctl->q_full[h], xq++ & 1)) break;
              // (Of two tiles by turns this half's comes first, or second.)
              if (two && t >= 1 - h && !give(ctl->v_full, ctl->v_empty, nv - 1)) break;
              if (t >= 0 && !wait(&ctl->v_full[sv], (nv / kStages) & 1)) break;
              if (two && has_k && t + 1 >= 1 - h && !give(ctl->k_full, ctl->k_empty, nk - 1)) break;
              const bool landed = has_k && tc::mbar_test_wait(&ctl->k_full[sk], (nk / kStages) & 1);
              if (t >= 0) {
                // P in two halves of each side's keys: the first is multiplied while the second is made.
                const uint64_t v = tc::smem_desc(s_v + sv * kVBytes, kBlock, 1024, tc::kSw128);
                auto pv = [&](int part) {
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const int kk = (i >> 1) * 4 + part * 2 + (i & 1);
                    mma_bf16_ts_pair(col_o, col_s + (kk >> 2) * 64 + (kk & 3) * 8, v + (kk * 16 * 128 >> 4),
                                     kIdescO, t + part + i != 0);
                  }
                };
                if (!wait(&ctl->p_half[h], xp & 1)) break;
                if (one && (ok = lock(ctl, a))) {
                  tc::fence_after_sync();
                  pv(0);
                }
                if (!wait(&ctl->p_full[h], xp++ & 1)) break;
                if (one) {
                  tc::fence_after_sync();
                  pv(1);
                  tc::mma_commit_pair(&ctl->v_empty[sv]);
                  if (t == c - 1) tc::mma_commit_pair(&ctl->o_full[h]);
                  if (!landed) unlock(ctl);
                }
              }
              if (has_k) {
                if (!landed && !wait(&ctl->k_full[sk], (nk / kStages) & 1)) break;
                if (one && ((t >= 0 && landed) || (ok = lock(ctl, a)))) {
                  tc::fence_after_sync();
                  const uint64_t k = tc::smem_desc(s_k + sk * kKBytes, 16, 1024, tc::kSw128);
#pragma unroll
                  for (int kk = 0; kk < 12; ++kk)
                    mma_bf16_pair(col_s, qd + (((kk >> 2) * kBlock + (kk & 3) * 32) >> 4),
                                  k + (((kk >> 2) * kKBlock + (kk & 3) * 32) >> 4), kIdescS, kk != 0);
                  tc::mma_commit_pair(&ctl->s_full[h]);
                  tc::mma_commit_pair(&ctl->k_empty[sk]);
                  if (t + 1 == c - 1) tc::mma_commit_pair(&ctl->q_empty[h]);
                  unlock(ctl);
                }
              }
            }
          };
          if (two) multiply(std::true_type{});
          else multiply(std::false_type{});
          ok = __all_sync(0xffffffffu, ok);
          // The rest of the other half's, while it finishes: this half goes on to its next piece.
          const uint32_t done = two && c > 0 ? (h ? nt : nt - 1) : c;
          for (uint32_t i = done; ok && i < nt; ++i)
            if (!give(ctl->k_full, ctl->k_empty, n0 + i) || !give(ctl->v_full, ctl->v_empty, n0 + i)) break;
          ok = __all_sync(0xffffffffu, ok);
          n0 += nt;
        }
        if (one) {
          tc::mma_commit_pair(&ctl->drain[h]);       // every MMA done before the CTAs leave
          const unsigned long long t0 = tc::globaltimer_ns();
          while (!tc::mbar_try_wait(&ctl->drain[h], 0) && tc::globaltimer_ns() - t0 < a.wait_limit_ns) {
          }
        }
      }
    } else {
      // ------------------------------------------------------------ V, made fit for the MMAs
      // Weights of keys that a row does not see are 0, and 0 times a value has to be 0. Values behind
      // the request's last key are another's, or nothing's: they are cleared. In tiles that some
      // row sees in part, values that are no numbers are cleared too, and noted by dim, so that the
      // rows that see them get NaN there at the end.
      uint32_t n = 0;
      bool ok = true;
      for (uint32_t seq = 0; ok; ++seq) {
        Piece p;
        if (!take(ctl, seq, a, p, lane == 0)) break;
        // A piece is handed on once this CTA's softmaxes have taken the one two before it, and so have done
        // with the one three before it: what the other CTA has to know before it notes anything.
        if (lane == 0)
          asm volatile("st.release.cluster.shared::cluster.u32 [%0], %1;" ::"r"(tc::map_rank(&ctl->v_piece, rank ^ 1)),
                       "r"(seq + 1)
                       : "memory");
        __syncwarp();
        const int two = p.twin == 2, c0 = half_tiles(p, 0), nt = max(c0, half_tiles(p, 1)) << two;
#pragma unroll 1
        for (int t = 0; t < nt; ++t, ++n) {
          const int st = n % kStages, tile = t >> two, key = (p.t0 + tile) * kKeys, there = min(p.m - key, kKeys);
          uint4* v = reinterpret_cast<uint4*>(smem + kOffV + st * kVBytes);
          if (!(ok = __all_sync(0xffffffffu, pr_wait(&ctl->v_land[st], (n / kStages) & 1, ctl, a)))) break;
          if (there < kKeys) {
            for (int i = there * 8 + lane; i < kKeys * 8; i += 32) v[i] = make_uint4(0, 0, 0, 0);
            tc::fence_proxy_async_smem();
            __syncwarp();
          }
          if (row_limit(p, tile < c0 ? 0 : half_row(p, 1)) < key + there) {
            uint32_t odd = 0;                      // bit 15 of a half: an exponent of ones
#pragma unroll 4
            for (int i = lane; i < kKeys * 8; i += 32) {
              const uint4 x = v[i];
              odd |= ((x.x & 0x7F807F80u) + 0x00800080u) | ((x.y & 0x7F807F80u) + 0x00800080u) |
                     ((x.z & 0x7F807F80u) + 0x00800080u) | ((x.w & 0x7F807F80u) + 0x00800080u);
            }
            if (__any_sync(0xffffffffu, (odd & 0x80008000u) != 0)) {
              // The notes' place was that of piece seq - 4. This CTA's softmaxes have done with it, as have the
              // other's once its piece seq - 1 is handed on. (A half without tiles waits for nothing of
              // the other CTA's, so that one may be pieces behind.)
              if (!(ok = __all_sync(0xffffffffu, wait_v_piece(ctl, seq, a)))) break;
              const int b = seq & 3;
              for (int i = lane; i < kKeys * 64; i += 32) {
                uint16_t* x = reinterpret_cast<uint16_t*>(v) + i;
                if ((*x & 0x7F80u) != 0x7F80u) continue;
                *x = 0;
                // Row i / 64; its 16-byte pieces lie exchanged by the row's place among eight.
                const int key_row = i >> 6, piece = (i >> 3 & 7) ^ (key_row & 7);
                const int dim = (int)rank * 64 + piece * 8 + (i & 7);
                const unsigned long long note = (unsigned long long)(seq + 1) << 32 | ~(uint32_t)(key + key_row);
                for (int c = 0; c < 2; ++c) {
                  for (int h = two ? t & 1 : 0; h < (two ? (t & 1) + 1 : 2); ++h)
                    asm volatile("red.relaxed.cluster.shared::cluster.max.u64 [%0], %1;" ::"r"(
                                     tc::map_rank(&ctl->bad[b][h][dim], c)),
                                 "l"(note)
                                 : "memory");
                  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(tc::map_rank(&ctl->bad_piece[b], c)),
                               "r"(seq + 1)
                               : "memory");
                }
              }
              asm volatile("fence.acq_rel.cluster;" ::: "memory");
              tc::fence_proxy_async_smem();
              __syncwarp();
            }
          }
          if (lane == 0) tc::remote_arrive(tc::map_rank(&ctl->v_full[st], 0));
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax and output
    // Thread (h, side, row): keys 64 side .. of its row of S, dims 64 side .. of its row of O. After a
    // wait that ran out a half's threads go on to the end of the piece without waiting, so that
    // all meet at its barriers, and leave together.
    const int h = (warp - 4) >> 3, side = (warp - 4) >> 2 & 1, quarter = warp & 3, row = quarter * 32 + lane;
    const int in_half = (int)rank * kMine + row, j = h * kHalf + in_half;   // j: row of a slot
    const uint32_t p_half = tc::map_rank(&ctl->p_half[h], 0), p_full = tc::map_rank(&ctl->p_full[h], 0);
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t col_s = lanes + h * kKeys + side * 64;
    const uint32_t col_o = col_s + kColO;
    uint32_t xs = 0, xo = 0;
    Piece p;
    bool ok = true;
    auto all_wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, pr_wait(bar, parity, ctl, a));
    };
    for (uint32_t seq = 0; !half_any(h, !(ok && take(ctl, seq, a, p, lane == 0))); ++seq) {
      const int c = half_tiles(p, h);
      const int i_row = half_row(p, h) + in_half;
      const int lim = i_row < p.rows ? row_limit(p, i_row) : INT_MAX;
      p.row0 += i_row;                           // this thread's own
      p.head += p.twin && h;
      const int lowest = __reduce_min_sync(0xffffffffu, lim);
      int mine = p.t0 * kKeys + side * 64;       // this thread's first key of the tile
      float m = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int t = 0; t < c; ++t) {
        ok = all_wait(&ctl->s_full[h], xs++ & 1) && ok;
        tc::fence_after_sync();
        uint32_t raw[2][32];
        tc::tmem_ld32(col_s, raw[0]);
        tc::tmem_ld32(col_s + 32, raw[1]);
        tc::tmem_wait_ld();
        if (mine + 64 > lowest) {                // keys that some row of the warp does not see
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (mine + i >= lim) raw[i >> 5][i & 31] = 0xFF800000u;
        }
        mine += kKeys;
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 32; e += 2)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            mx[i] = max3(mx[i], __uint_as_float(raw[i][e]), __uint_as_float(raw[i][e + 1]));
        float top = fmaxf(mx[0], mx[1]) * a.scale_log2;
        // The first tile sets the maximum; later ones move it only when they exceed it by 2^8. The
        // barrier also tells that S is read, which P may now overwrite.
        if (half_any(h, top > m + kLazy)) {
          if (side) ctl->row[h][row] = top;
          half_any(h, false);
          if (!side) ctl->row[h][row] = top = fmaxf(top, ctl->row[h][row]);
          half_any(h, false);
          if (side) top = ctl->row[h][row];
          const bool moves = top > m + kLazy;
          const float f = moves ? ex2(m - top) : 1.f;
          if (moves) m = top;
          l *= f;
          if (t > 0 && __any_sync(0xffffffffu, moves)) {
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
              uint32_t o[8];
              tmem_ld8(col_o + 8 * i, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st8(col_o + 8 * i, o);
            }
          }
        }
        const float base = m == -INFINITY ? 0.f : -m;
        const uint64_t c2 = pack_f32x2(a.scale_log2, a.scale_log2), b2 = pack_f32x2(base, base);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float x, y;
            unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(raw[i][2 * e]), __uint_as_float(raw[i][2 * e + 1])),
                                   c2, b2), x, y);
            x = ex2(x);
            y = ex2(y);
            sum[e & 1] = add_f32x2(sum[e & 1], pack_f32x2(x, y));
            pk[e] = f32x2_to_bf16x2(x, y);
          }
          tc::tmem_st16(col_s + 16 * i, pk);
          tc::tmem_wait_st();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::remote_arrive(i ? p_full : p_half);
          __syncwarp();                          // the next store to TMEM is the whole warp's
        }
        float s0, s1;
        unpack_f32x2(add_f32x2(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
      }
      // The rows' sums, of both threads.
      if (side) ctl->row[h][row] = l;
      half_any(h, false);
      if (!side) ctl->row[h][row] = l += ctl->row[h][row];
      if (c > 0) ok = all_wait(&ctl->o_full[h], xo++ & 1) && ok;
      half_any(h, false);
      if (side) l = ctl->row[h][row];
      tc::fence_after_sync();
      float lse = l > 0.f ? m + log2f(l) : l == 0.f ? -INFINITY : l;
      // A row that sees keys and has a sum of 0: all scores are -infinity, the formula 0 / 0. In a piece the
      // others may still have weight: it keeps its O of zeros, and an LSE that tells.
      if (l == 0.f && c > 0 && lim > 0) {
        l = p.slot < 0 ? NAN : 1.f;
        if (p.slot >= 0) lse = kLowest;
      }
      const float inv = l > 0.f ? rcp(l) : l;    // NaN stays
      const bool valid = lim != INT_MAX;
      const size_t at = (size_t)p.row0 * a.H + p.head;
      if (p.slot < 0) {
        if (valid && a.lse && side == 0) a.lse[at] = lse;
      } else if (side == 0) {
        a.part_lse[(size_t)p.slot * kRows + j] = lse;
      }
      const volatile unsigned long long* bad = ctl->bad[seq & 3][h] + side * 64;
      const bool noted = *reinterpret_cast<volatile uint32_t*>(&ctl->bad_piece[seq & 3]) == seq + 1;
#pragma unroll 4
      for (int i = 0; i < 4; ++i) {
        uint32_t o[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = 0;
        if (c > 0) {
          __syncwarp();                          // rows that are none have stored nothing
          tc::tmem_ld16(col_o + 16 * i, o);
          tc::tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = l == 0.f ? 0u : __float_as_uint(__uint_as_float(o[e]) * inv);
        if (noted) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const unsigned long long note = bad[16 * i + e];
            if ((uint32_t)(note >> 32) == seq + 1 && (uint32_t)lim > ~(uint32_t)note) o[e] = 0x7FC00000u;
          }
        }
        if (p.slot < 0) {
          uint32_t w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            w[e] = f32x2_to_bf16x2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
          if (valid && ok) st_32(a.out + at * kV + side * 64 + 16 * i, w);
        } else if (c > 0) {
          uint4* dst =
              reinterpret_cast<uint4*>(a.part_o) + ((size_t)p.slot * 32 + side * 16 + 4 * i) * kRows + j;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            dst[e * kRows] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      }
      tc::fence_before_sync();
    }
  }
  tc::fence_before_sync();
  tc::cluster_sync();            // no CTA leaves while the other's MMAs or arrivals may reach it
  tc::fence_after_sync();
  if (warp == 1) tc::tmem_dealloc_pair(tmem, kTmemCols);
}

// ---------------------------------------------------------------- joining the pieces
// An item that a cut runs through: CTA (p, s) joins 16 rows of the one that begins in part p. A warp
// has 16 rows x 2 quads of dims, 256 bytes in a row; a thread two quads of a row.
constexpr int kJoinRows = 16, kSlices = kRows / kJoinRows;

__global__ void __launch_bounds__(256) prompt_join_kernel(const PromptArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const int4 jn = *reinterpret_cast<const int4*>(a.joins + blockIdx.y);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = blockIdx.x * kJoinRows + (lane & 15);
  // Row j of the slots: of the item, or in half j / 256 a row of that head of two.
  const int part = blockIdx.y, last = jn.w >> 1, twin = jn.w & 1, row_of = twin ? j % kHalf : j;
  if (row_of >= jn.y) return;
  // Pieces: the last of part `part`, then the first of the parts up to `last`.
  auto slot = [&](int p) { return (size_t)(p == part ? 2 * p + 1 : 2 * p); };
  float top = -INFINITY;
#pragma unroll 8
  for (int p = part; p <= last; ++p) top = fmaxf(top, a.part_lse[slot(p) * kRows + j]);
  const float base = top == -INFINITY ? 0.f : top;
  const int quad = (lane >> 4) + 2 * warp;                   // and quad + 16
  float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0}, z = 0.f;
#pragma unroll 4
  for (int p = part; p <= last; ++p) {
    const float l = a.part_lse[slot(p) * kRows + j], w = ex2(l - base);
    const float4* src = reinterpret_cast<const float4*>(a.part_o) + (slot(p) * 32 + quad) * kRows + j;
    float4 v[2] = {src[0], src[16 * kRows]};
    z += w;
    // A piece of which the row sees nothing is perhaps not written. (One whose weight is too small for
    // FP32 is, and its NaN counts.)
    if (l == -INFINITY) v[0] = v[1] = make_float4(0, 0, 0, 0);
    acc[0] += w * v[0].x;
    acc[1] += w * v[0].y;
    acc[2] += w * v[0].z;
    acc[3] += w * v[0].w;
    acc[4] += w * v[1].x;
    acc[5] += w * v[1].y;
    acc[6] += w * v[1].z;
    acc[7] += w * v[1].w;
  }
  const bool lowest = base == kLowest;           // keys seen, and no score above -infinity
  const float inv = lowest ? NAN : z > 0.f ? 1.f / z : z;    // NaN stays
  const size_t row = (size_t)(jn.x + row_of) * a.H + jn.z + (twin ? j / kHalf : 0);
  if (a.lse && threadIdx.x < 16)
    a.lse[row] = z > 0.f && !lowest ? base + log2f(z) : z >= 0.f ? -INFINITY : z;
  uint2* dst = reinterpret_cast<uint2*>(a.out + row * kV) + quad;
  dst[0] = make_uint2(f32x2_to_bf16x2(acc[0] * inv, acc[1] * inv), f32x2_to_bf16x2(acc[2] * inv, acc[3] * inv));
  dst[16] = make_uint2(f32x2_to_bf16x2(acc[4] * inv, acc[5] * inv), f32x2_to_bf16x2(acc[6] * inv, acc[7] * inv));
}

int check_prompt(const mla_prompt_shape* s) {
  if (!s) return MLA_ERR_NULL;
  if (s->R < 1 || s->R > kMaxR || s->tokens < 0 || s->tokens > (1 << 24) || s->keys < 0 ||
      s->keys > (1 << 24) || s->H < 1 || s->H > (1 << 12) || s->kv_heads < 1 ||
      s->H % s->kv_heads != 0 || (s->causal != 0 && s->causal != 1) || s->num_ctas < 1 ||
      s->num_ctas > 2048)
    return MLA_ERR_SHAPE;
  return MLA_OK;
}
size_t prompt_bytes(const mla_prompt_shape* s) {
  const int pairs = pairs_of(s->num_ctas);
  return plan_bytes(s->R, pairs) + lse_bytes(pairs) + 2 * (size_t)pairs * kSlotBytes;
}

int32_t prompt_impl(const mla_prompt_shape* s, const void* q, const void* k_nope, const void* k_rope,
                    const void* v, const int32_t* cu_tokens, const int32_t* cu_keys, float sm_scale,
                    void* workspace, size_t workspace_bytes_given, void* out, float* lse,
                    int32_t* status, mla_stream_t stream, unsigned long long wait_limit_ns,
                    int withhold) {
  int st = check_prompt(s);
  if (st != MLA_OK) return st;
  if (s->q_token_stride < kNope + kRope || s->q_head_stride < kNope + kRope ||
      s->k_token_stride < kNope || s->k_head_stride < kNope || s->v_token_stride < kV ||
      s->v_head_stride < kV || s->rope_stride < kRope)
    return MLA_ERR_SHAPE;
  if (!std::isfinite(sm_scale) || !(sm_scale > 0.f)) return MLA_ERR_SHAPE;
  if (s->tokens == 0) return MLA_OK;
  if (!q || !cu_tokens || !out || !workspace || (s->keys > 0 && (!k_nope || !k_rope || !v)))
    return MLA_ERR_NULL;
  if (!aligned(q, 16) || !aligned(k_nope, 16) || !aligned(k_rope, 16) || !aligned(v, 16) ||
      !aligned(out, 32) || !aligned(lse, 4) || !aligned(cu_tokens, 4) || !aligned(cu_keys, 4) ||
      !aligned(workspace, 256) || !aligned(status, 4) || s->q_token_stride % 8 || s->q_head_stride % 8 ||
      s->k_token_stride % 8 || s->k_head_stride % 8 || s->v_token_stride % 8 || s->v_head_stride % 8 ||
      s->rope_stride % 8)
    return MLA_ERR_ALIGN;
  if (workspace_bytes_given < prompt_bytes(s)) return MLA_ERR_WORKSPACE;
  if ((st = check_device()) != MLA_OK) return st;

  PromptArgs a;
  char* ws = static_cast<char*>(workspace);
  a.cu = cu_tokens;
  a.cu_keys = cu_keys;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.plan = reinterpret_cast<Plan*>(ws);
  a.first_place = reinterpret_cast<long long*>(ws + sizeof(Plan));
  a.first_item = a.first_place + s->R + 1;
  a.joins = reinterpret_cast<Join*>(a.first_item + s->R + 1);
  a.pairs = pairs_of(s->num_ctas);
  a.part_lse = reinterpret_cast<float*>(ws + plan_bytes(s->R, a.pairs));
  a.part_o = reinterpret_cast<float*>(ws + plan_bytes(s->R, a.pairs) + lse_bytes(a.pairs));
  a.status = status;
  a.scale_log2 = (float)((double)sm_scale * 1.4426950408889634);
  a.R = s->R;
  a.T = s->tokens;
  a.Tk = s->keys;
  a.H = s->H;
  a.group = s->H / s->kv_heads;
  a.causal = s->causal;
  a.wait_limit_ns = wait_limit_ns;
  a.withhold = withhold;
  // Without keys the maps of K and V stand on the queries; nothing is read through them.
  CUtensorMap tq, tk, tr, tv;
  const void* kn = s->keys ? k_nope : q;
  const void* kr = s->keys ? k_rope : q;
  const void* kv = s->keys ? v : q;
  const cuuint64_t T = (cuuint64_t)s->tokens, Tk = s->keys ? (cuuint64_t)s->keys : 1;
  const cuuint64_t q_dims[3] = {(kNope + kRope) * 2, (cuuint64_t)s->H, T};
  const cuuint64_t q_str[2] = {(cuuint64_t)s->q_head_stride * 2, (cuuint64_t)s->q_token_stride * 2};
  const cuuint64_t k_dims[3] = {kNope * 2, s->keys ? (cuuint64_t)s->kv_heads : 1, Tk};
  const cuuint64_t k_str[2] = {(cuuint64_t)s->k_head_stride * 2, (cuuint64_t)s->k_token_stride * 2};
  const cuuint64_t v_dims[3] = {kV * 2, s->keys ? (cuuint64_t)s->kv_heads : 1, Tk};
  const cuuint64_t v_str[2] = {(cuuint64_t)s->v_head_stride * 2, (cuuint64_t)s->v_token_stride * 2};
  const cuuint64_t r_dims[2] = {kRope * 2, Tk}, r_str[1] = {(cuuint64_t)s->rope_stride * 2};
  const cuuint32_t box3[3] = {128, 1, 128}, box_k[3] = {128, 1, 64}, box_r[2] = {128, 64};
  if (!dec::encode(&tq, q, 3, q_dims, q_str, box3, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !dec::encode(&tk, kn, 3, k_dims, k_str, box_k, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !dec::encode(&tv, kv, 3, v_dims, v_str, box3, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !dec::encode(&tr, kr, 2, r_dims, r_str, box_r, CU_TENSOR_MAP_SWIZZLE_128B))
    return MLA_ERR_CUDA;
  static bool attr_set[64] = {};
  if (dec::set_smem(prompt_kernel, kSmemBytes, attr_set) != cudaSuccess) return MLA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // A batch of few requests and items has no plan kernel before it: 2 short prompts 11.3 -> 8.8 us,
  // 512 tokens on 16k keys 51.4 -> 48.1, 24 prompts up to 2k the same. Others gain by claimed items,
  // which need one. Offsets that are none may let requests overlap: each may have all rows.
  // Two heads to an item of a short request, unless a head for each pair of CTAs is quicker.
  a.twins = s->keys > kUncut * kKeys || (long long)s->R * s->H > a.pairs;
  const long long items_least = (long long)s->H * cdiv(s->tokens, kRows);
  const long long places_most = items_least * s->R * (1 + kExtra + cdiv(s->keys, kKeys));
  a.planned = s->R > 32 || items_least >= (long long)kWhole * a.pairs || places_most >= (1ll << 31);
  if (a.planned) {
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3((unsigned)(cdiv(s->R, 32) * 32));
    if (cudaLaunchKernelEx(&cfg, prompt_plan_kernel, a) != cudaSuccess) return MLA_ERR_CUDA;
  }
  // No more pairs than the batch can have places.
  const int pairs = (int)(places_most < a.pairs ? places_most : a.pairs);
  cfg.gridDim = dim3(2 * (unsigned)pairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  if (cudaLaunchKernelEx(&cfg, prompt_kernel, a, tq, tk, tr, tv) != cudaSuccess) return MLA_ERR_CUDA;
  // Requests of so few keys that no item can be cut leave nothing to join.
  if (cdiv(s->keys, kKeys) <= kUncut || pairs < 2) return MLA_OK;
  cfg.gridDim = dim3(kSlices, (unsigned)(pairs - 1));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, prompt_join_kernel, a) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace
}  // namespace mlafold

using namespace mlafold;

extern "C" int32_t mla_prompt_workspace_bytes(const mla_prompt_shape* s, size_t* bytes) {
  const int st = check_prompt(s);
  if (st != MLA_OK) return st;
  if (!bytes) return MLA_ERR_NULL;
  *bytes = prompt_bytes(s);
  return MLA_OK;
}

extern "C" int32_t mla_prompt_attention(const mla_prompt_shape* s, const void* q, const void* k_nope,
                                        const void* k_rope, const void* v, const int32_t* cu_tokens,
                                        const int32_t* cu_keys, float sm_scale, void* workspace,
                                        size_t workspace_bytes, void* out, float* lse,
                                        int32_t* status, mla_stream_t stream) {
  return prompt_impl(s, q, k_nope, k_rope, v, cu_tokens, cu_keys, sm_scale, workspace, workspace_bytes,
                     out, lse, status, stream, kWaitLimitNs, 0);
}

extern "C" int32_t mla_prompt_attention_wait_test(const mla_prompt_shape* s, const void* q,
                                                  const void* k_nope, const void* k_rope,
                                                  const void* v, const int32_t* cu_tokens,
                                                  const int32_t* cu_keys, float sm_scale,
                                                  void* workspace, size_t workspace_bytes, void* out,
                                                  float* lse, int32_t* status,
                                                  uint64_t wait_limit_ns, mla_stream_t stream) {
  if (!status) return MLA_ERR_NULL;
  if (wait_limit_ns < 1000000ull || wait_limit_ns > kWaitLimitNs) return MLA_ERR_SHAPE;
  return prompt_impl(s, q, k_nope, k_rope, v, cu_tokens, cu_keys, sm_scale, workspace, workspace_bytes,
                     out, lse, status, stream, wait_limit_ns, 1);
}
