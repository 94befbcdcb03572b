// Absorbed decode queries: the nope part of every (token, head) query times
// that head's W_UK, its rope part turned by the token's position, both as
// E4M3 codes in the layout the decode reads.
//
//   out[t, h, 0:512]   = e4m3((q[t, h, 0:128] . W_UK[h]) / q_scale),  W_UK[h] [128, 512]
//   out[t, h, 512:576] = e4m3(rotate(q[t, h, 128:192], position of t) / q_scale)
//
// The counterpart, before the decode, of the W_UV up-projection after it
// (uv.cu). BF16 products accumulate in FP32 in TMEM; a code is rounded once.
//
// Bound by HBM: W_UK (128 KB per head), 384 B in and 576 B out per (token,
// head) against 131 kFLOP, 137 FLOP/B at most where the tensor pipe's ridge is
// 291. Layout: 128 tokens are the MMA's M, so a thread of the read-back holds
// one token's consecutive latent dims and packs them into codes without a
// transpose (fewer tokens leave rows of the MMA idle, which costs nothing at
// that bound); 128 latent dims (one band) are its N, read MN-major from W_UK's
// latent-contiguous rows. Persistent CTAs walk (head, 128 tokens, band set)
// jobs: warp 0 loads by TMA (Q of a job into a ring of two, W bands into a ring
// of four), warp 1 issues the MMAs into four TMEM accumulators, warps 2-9 read them
// back and store them by TMA, each warp its 32 tokens x 64 dims on its own, from
// two staging tiles, and warps 10-17 turn the rope dims beside them. 128 x 7 x 64:
// 12.5 - 12.8 us, 5.0 TB/s (0.74 of the copy rate; a band takes 1,300 cycles, the time in which
// shared memory, 128 B a cycle, takes in W, feeds A and B to the MMAs, 64 KB, and
// passes the codes on); 16 x 4 x 64 4.2 - 4.4 us, 64 x 7 x 8 3.8 - 4.0 us, 2 x 4 x 8 3.2 - 3.4 us (one
// band per CTA: latency). Pairs of CTAs (M = 256, N = 256) took 16.5 us, twice the
// read-back warps 12.6 and more on the small ones.
#include <cmath>

#include "checks.h"
#include "decode_common.cuh"
#include "formats.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "tc.cuh"

namespace mlafold {
namespace {

constexpr int kNope = 128, kRope = 64;
constexpr int kTok = 128;                       // tokens per job: the MMA's M
constexpr int kBand = 128;                      // latent dims per unit: the MMA's N
constexpr int kBands = kDv / kBand;
constexpr int kWStages = 4, kQStages = 2, kOutStages = 2, kAccs = 4;
constexpr int kChunk = 128 * 128;               // 128 rows of 128 bytes
constexpr int kQBytes = 2 * kChunk;             // 128 tokens x 128 BF16, two 64-dim chunks
constexpr int kWBytes = 2 * kChunk;             // 128 nope rows x 128 BF16, two 64-latent chunks
constexpr int kOutBytes = 32 * 64;              // of a read-back warp: 32 tokens x 64 codes
constexpr int kOffW = 0;
constexpr int kOffQ = kOffW + kWStages * kWBytes;
constexpr int kOffOut = kOffQ + kQStages * kQBytes;
constexpr int kEpi = 256;                       // read-back threads
constexpr int kOffCtl = kOffOut + kEpi / 32 * kOutStages * kOutBytes;
constexpr int kTurn = 256;                      // rope threads: two per token
constexpr int kThreads = 64 + kEpi + kTurn;
constexpr uint32_t kTmemCols = kAccs * kBand;   // 512
// BF16 x BF16 -> FP32, A (queries) K-major, B (W_UK) MN-major.
constexpr uint32_t kIdesc = tc::idesc_bf16_f32(kTok, kBand) | (1u << 16);

struct AbsorbCtl {
  uint64_t w_full[kWStages], w_empty[kWStages];   // TMA -> MMA, MMA -> TMA
  uint64_t q_full[kQStages], q_empty[kQStages];
  uint64_t d_full[kAccs], d_empty[kAccs];         // MMA -> read-back, read-back -> MMA
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
};
constexpr int kSmemBytes = kOffCtl + (int)sizeof(AbsorbCtl) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

struct AbsorbArgs {
  const uint16_t* q;             // [R k] tokens of [H] heads of [192] BF16, strided
  const float* rope;             // [rope_rows][32 cos, 32 sin]
  const int32_t* rope_starts;    // [R]
  uint8_t* out;                  // [R k][H][576]
  int32_t* status;               // may be null
  long long token_stride, head_stride;
  float inv_scale;
  int T, k, H, rope_rows, interleaved;
  int tiles, sets, jobs;         // token tiles, band sets per (head, tile), jobs
  unsigned long long wait_limit_ns;   // bound of every pipeline wait
  int withhold_first_copy;            // failure-detection test: CTA 0 never loads its first
                                      // weights, so one wait must run out
};

// A box of shared memory -> global; the issuing thread commits and waits for its bulk group.
__device__ __forceinline__ void store_box(const CUtensorMap* m, const void* src, int x, int y,
                                          int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(m)),
      "r"(tc::smem_u32(src)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ bool ab_wait(uint64_t* bar, uint32_t parity, AbsorbCtl* ctl,
                                        const AbsorbArgs& a) {
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
// The 64 rope dims of the 128 tokens of a job: two threads per token, 16
// planes each, straight from and to global memory.
__device__ __forceinline__ void turn_rope(const AbsorbArgs& a, int h, int tok0, int gt) {
  const int t = tok0 + (gt >> 1), part = gt & 1;
  if (t >= a.T) return;
  const int r = t / a.k;
  const int start = a.rope_starts[r];
  const long long pos = (long long)start + (t - r * a.k);
  const uint16_t* x = a.q + (long long)t * a.token_stride + (long long)h * a.head_stride + kNope;
  uint8_t* dst = a.out + ((size_t)t * a.H + h) * kDqk + kDv;
  uint32_t lo[4] = {0, 0, 0, 0}, hi[4] = {0, 0, 0, 0};   // 16 codes each
  if (start >= 0 && pos < a.rope_rows) {
    const float4* cs = reinterpret_cast<const float4*>(a.rope + pos * 64 + part * 16);
    float x0[16], x1[16];                                 // the planes' two coordinates
    if (a.interleaved) {
      const uint4* src = reinterpret_cast<const uint4*>(x + part * 32);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float f[8];
        bf16x8_to_f32(src[u], f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x0[4 * u + e] = f[2 * e];
          x1[4 * u + e] = f[2 * e + 1];
        }
      }
    } else {
      const uint4* s0 = reinterpret_cast<const uint4*>(x + part * 16);
      const uint4* s1 = reinterpret_cast<const uint4*>(x + 32 + part * 16);
      bf16x8_to_f32(s0[0], x0);
      bf16x8_to_f32(s0[1], x0 + 8);
      bf16x8_to_f32(s1[0], x1);
      bf16x8_to_f32(s1[1], x1 + 8);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float4 c4 = cs[u], s4 = cs[8 + u];
      const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
      float y0[4], y1[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float p = x0[4 * u + e], q = x1[4 * u + e];
        y0[e] = (p * c[e] - q * s[e]) * a.inv_scale;
        y1[e] = (q * c[e] + p * s[e]) * a.inv_scale;
      }
      if (a.interleaved) {                                // codes 8 u .. 8 u + 7 of 32
        const uint32_t w0 = f32x4_to_e4m3x4(y0[0], y1[0], y0[1], y1[1]);
        const uint32_t w1 = f32x4_to_e4m3x4(y0[2], y1[2], y0[3], y1[3]);
        if (u < 2) {
          lo[2 * u] = w0;
          lo[2 * u + 1] = w1;
        } else {
          hi[2 * u - 4] = w0;
          hi[2 * u - 3] = w1;
        }
      } else {
        lo[u] = f32x4_to_e4m3x4(y0[0], y0[1], y0[2], y0[3]);
        hi[u] = f32x4_to_e4m3x4(y1[0], y1[1], y1[2], y1[3]);
      }
    }
  } else if (start >= 0 && a.status) {
    atomicOr(a.status, MLA_FAULT_ROPE_RANGE);
  }
  const int at = a.interleaved ? part * 2 : part, other = a.interleaved ? at + 1 : at + 2;
  reinterpret_cast<uint4*>(dst)[at] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  reinterpret_cast<uint4*>(dst)[other] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
}

__global__ void __launch_bounds__(kThreads, 1)
absorb_kernel(const AbsorbArgs a, const __grid_constant__ CUtensorMap tm_q,
              const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_o) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  AbsorbCtl* ctl = reinterpret_cast<AbsorbCtl*>(smem + kOffCtl);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kWStages; ++i) {
      tc::mbar_init(&ctl->w_full[i], 1);
      tc::mbar_init(&ctl->w_empty[i], 1);
    }
    for (int i = 0; i < kQStages; ++i) {
      tc::mbar_init(&ctl->q_full[i], 1);
      tc::mbar_init(&ctl->q_empty[i], 1);
    }
    for (int i = 0; i < kAccs; ++i) {
      tc::mbar_init(&ctl->d_full[i], 1);
      tc::mbar_init(&ctl->d_empty[i], kEpi);
    }
    tc::mbar_init(&ctl->drain, 1);
    ctl->abort_flag = 0;
    tc::fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tc::prefetch_tmap(&tm_q);
    tc::prefetch_tmap(&tm_w);
    tc::prefetch_tmap(&tm_o);
  }
  if (warp == 1) {
    tc::tmem_alloc(&ctl->tmem_base, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = ctl->tmem_base;

  const int per = kBands / a.sets;                 // bands per job
  // Job -> head, first token, first band: head-major, so CTAs that run at the
  // same time share a head's W_UK in L2.
  auto head_of = [&](int job) { return job / (a.tiles * a.sets); };
  auto tok_of = [&](int job) { return (job / a.sets) % a.tiles * kTok; };
  auto band_of = [&](int job) { return (job % a.sets) * per; };

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      uint32_t u = 0, x = 0, uq = 0;
      auto withheld = [&](uint32_t at) {
        return a.withhold_first_copy && blockIdx.x == 0 && at == 0;
      };
      auto load_w = [&](int job, int b, uint32_t at) {
        uint64_t* bar = &ctl->w_full[at % kWStages];
        uint8_t* w = smem + kOffW + (at % kWStages) * kWBytes;
        const int y = head_of(job) * kNope, xb = (band_of(job) + b) * kBand * 2;
        if (withheld(at)) return;
        tc::mbar_arrive_expect_tx(bar, kWBytes);
        tc::tma_load_2d(w, &tm_w, bar, xb, y);
        tc::tma_load_2d(w + kChunk, &tm_w, bar, xb + 128, y);
      };
      grid_dep_wait();
      grid_dep_launch();
      for (int job = blockIdx.x; ok && job < a.jobs; job += gridDim.x, ++x) {
        const int qs = x % kQStages;
        if (x >= kQStages &&
            !(ok = ab_wait(&ctl->q_empty[qs], (x / kQStages - 1) & 1, ctl, a)))
          break;
        uint8_t* q = smem + kOffQ + qs * kQBytes;
        tc::mbar_arrive_expect_tx(&ctl->q_full[qs], kQBytes);
        tc::tma_load_3d(q, &tm_q, &ctl->q_full[qs], 0, head_of(job), tok_of(job));
        tc::tma_load_3d(q + kChunk, &tm_q, &ctl->q_full[qs], 128, head_of(job), tok_of(job));
        uq = x + 1;
        for (int b = 0; b < per; ++b, ++u) {
          if (u >= kWStages &&
              !(ok = ab_wait(&ctl->w_empty[u % kWStages], (u / kWStages - 1) & 1, ctl, a)))
            break;
          load_w(job, b, u);
        }
      }
      // Never leave with copies in flight: another role may have given up a wait, then or
      // later, whether this one did or not.
      const unsigned long long t0 = tc::globaltimer_ns();
      for (uint32_t i = u < kWStages ? 0 : u - kWStages; i < u; ++i)
        while (!withheld(i) && !tc::mbar_try_wait(&ctl->w_full[i % kWStages], (i / kWStages) & 1) &&
               tc::globaltimer_ns() - t0 < a.wait_limit_ns) {
        }
      for (uint32_t i = uq < kQStages ? 0 : uq - kQStages; i < uq; ++i)
        while (!tc::mbar_try_wait(&ctl->q_full[i % kQStages], (i / kQStages) & 1) &&
               tc::globaltimer_ns() - t0 < a.wait_limit_ns) {
        }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      grid_dep_wait();       // its waits' limit counts from the end of the preceding kernel
      bool ok = true;
      uint32_t u = 0, x = 0;
      for (int job = blockIdx.x; ok && job < a.jobs; job += gridDim.x, ++x) {
        const int qs = x % kQStages;
        if (!(ok = ab_wait(&ctl->q_full[qs], (x / kQStages) & 1, ctl, a))) break;
        const uint32_t q = tc::smem_u32(smem + kOffQ + qs * kQBytes);
        for (int b = 0; b < per; ++b, ++u) {
          const int ws = u % kWStages, ds = u % kAccs;
          if (!(ok = ab_wait(&ctl->w_full[ws], (u / kWStages) & 1, ctl, a))) break;
          if (u >= kAccs && !(ok = ab_wait(&ctl->d_empty[ds], (u / kAccs - 1) & 1, ctl, a)))
            break;
          tc::fence_after_sync();
          const uint32_t w = tc::smem_u32(smem + kOffW + ws * kWBytes);
#pragma unroll
          for (int kk = 0; kk < kNope / 16; ++kk)
            // A: 16 nope dims (32 bytes) of a 64-dim chunk; B: 16 nope rows of
            // both 64-latent chunks (one chunk apart), 8-row groups 1 KB apart.
            tc::mma_bf16(tmem + ds * kBand,
                         tc::smem_desc(q + (kk >> 2) * kChunk + (kk & 3) * 32, 16, 1024, tc::kSw128),
                         tc::smem_desc(w + kk * 16 * 128, kChunk, 1024, tc::kSw128), kIdesc,
                         kk != 0);
          tc::mma_commit(&ctl->w_empty[ws]);
          if (b == per - 1) tc::mma_commit(&ctl->q_empty[qs]);
          tc::mma_commit(&ctl->d_full[ds]);
        }
      }
      tc::mma_commit(&ctl->drain);                 // every MMA done before TMEM is released
      const unsigned long long t0 = tc::globaltimer_ns();
      while (!tc::mbar_try_wait(&ctl->drain, 0) && tc::globaltimer_ns() - t0 < a.wait_limit_ns) {
      }
    }
  } else if (warp >= 2 + kEpi / 32) {
    grid_dep_wait();
    for (int job = blockIdx.x; job < a.jobs; job += gridDim.x)
      if (band_of(job) == 0) turn_rope(a, head_of(job), tok_of(job), threadIdx.x - 64 - kEpi);
  } else {
    grid_dep_wait();
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    uint32_t u = 0;
    bool ok = true;
    for (int job = blockIdx.x; ok && job < a.jobs; job += gridDim.x) {
      const int h = head_of(job), tok0 = tok_of(job);
      for (int b = 0; ok && b < per; ++b, ++u) {
        const int ds = u % kAccs;
        ok = __all_sync(0xffffffffu, ab_wait(&ctl->d_full[ds], (u / kAccs) & 1, ctl, a));
        if (!ok) break;
        tc::fence_after_sync();
        uint32_t raw[2][32];
        const uint32_t src = tmem + ((uint32_t)(quarter * 32) << 16) + ds * kBand + half * 64;
        tc::tmem_ld32(src, raw[0]);
        tc::tmem_ld32(src + 32, raw[1]);
        tc::tmem_wait_ld();
        tc::fence_before_sync();
        tc::mbar_arrive(&ctl->d_empty[ds]);
        // The warp's staging tile is free once its store of two units back has read it.
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        __syncwarp();
        uint8_t* stage = smem + kOffOut + ((warp - 2) * kOutStages + u % kOutStages) * kOutBytes;
        uint4* dst = reinterpret_cast<uint4*>(stage + lane * 64);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t* f = &raw[j >> 1][(j & 1) * 16 + e * 4];
            w[e] = f32x4_to_e4m3x4(__uint_as_float(f[0]) * a.inv_scale,
                                   __uint_as_float(f[1]) * a.inv_scale,
                                   __uint_as_float(f[2]) * a.inv_scale,
                                   __uint_as_float(f[3]) * a.inv_scale);
          }
          // 64-byte swizzle: 16-byte piece p of row r at piece p ^ ((r >> 1) & 3).
          dst[j ^ ((lane >> 1) & 3)] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        const int tok = tok0 + quarter * 32;
        if (lane == 0 && tok < a.T)
          store_box(&tm_o, stage, (band_of(job) + b) * kBand + half * 64, h, tok);
        if (lane == 0) asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 1) tc::tmem_dealloc(tmem, kTmemCols);
}

}  // namespace
}  // namespace mlafold

using namespace mlafold;

namespace {

constexpr unsigned long long kWaitLimitNs = 2000000000ull;   // 2 s

int32_t absorb_impl(const mla_query_shape* s, const void* q, const void* w_uk, const float* rope,
                    const int32_t* rope_starts, float q_scale, void* out, int32_t* status,
                    mla_stream_t stream, unsigned long long wait_limit_ns, int withhold) {
  if (!s) return MLA_ERR_NULL;
  if (s->R < 1 || s->k < 1 || s->H < 1 || s->rope_rows < 1 ||
      (s->interleaved != 0 && s->interleaved != 1) || s->token_stride < kNope + kRope ||
      s->head_stride < kNope + kRope)
    return MLA_ERR_SHAPE;
  const long long T = (long long)s->R * s->k, tiles = cdiv(T, kTok);
  if (T > (1 << 24) || s->H > (1 << 16) || tiles * s->H > (1 << 24)) return MLA_ERR_SHAPE;
  if (!std::isfinite(q_scale) || !(q_scale > 0.f) || !std::isfinite(1.0f / q_scale))
    return MLA_ERR_SHAPE;
  if (!q || !w_uk || !rope || !rope_starts || !out) return MLA_ERR_NULL;
  if (!aligned(q, 16) || !aligned(w_uk, 16) || !aligned(out, 16) || !aligned(rope, 16) ||
      !aligned(rope_starts, 4) || !aligned(status, 4) || s->token_stride % 8 != 0 ||
      s->head_stride % 8 != 0)
    return MLA_ERR_ALIGN;
  int st = check_device();
  if (st != MLA_OK) return st;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MLA_ERR_CUDA;

  CUtensorMap tq, tw, to;
  const cuuint64_t q_dims[3] = {kNope * 2, (cuuint64_t)s->H, (cuuint64_t)T};
  const cuuint64_t q_str[2] = {(cuuint64_t)s->head_stride * 2, (cuuint64_t)s->token_stride * 2};
  const cuuint64_t w_dims[2] = {kDv * 2, (cuuint64_t)s->H * kNope};
  const cuuint64_t w_str[1] = {kDv * 2};
  const cuuint64_t o_dims[3] = {kDqk, (cuuint64_t)s->H, (cuuint64_t)T};
  const cuuint64_t o_str[2] = {kDqk, (cuuint64_t)s->H * kDqk};
  const cuuint32_t box3[3] = {128, 1, kTok}, box2[2] = {128, kNope}, box_o[3] = {64, 1, 32};
  if (!dec::encode(&tq, q, 3, q_dims, q_str, box3, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !dec::encode(&tw, w_uk, 2, w_dims, w_str, box2, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !dec::encode(&to, out, 3, o_dims, o_str, box_o, CU_TENSOR_MAP_SWIZZLE_64B))
    return MLA_ERR_CUDA;
  static bool attr_set[64] = {};
  if (dec::set_smem(absorb_kernel, kSmemBytes, attr_set) != cudaSuccess) return MLA_ERR_CUDA;

  AbsorbArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.rope = rope;
  a.rope_starts = rope_starts;
  a.out = static_cast<uint8_t*>(out);
  a.status = status;
  a.token_stride = s->token_stride;
  a.head_stride = s->head_stride;
  a.inv_scale = 1.0f / q_scale;
  a.T = (int)T;
  a.k = s->k;
  a.H = s->H;
  a.rope_rows = s->rope_rows;
  a.interleaved = s->interleaved;
  a.tiles = (int)tiles;
  // Bands of one (head, tile) per job: as many CTAs as help. The busiest CTA's
  // bands decide; with equal ones fewer sets load Q fewer times.
  long long best = 0;
  a.sets = 1;
  for (int sets = 1; sets <= kBands; sets *= 2) {
    const long long bands = cdiv(tiles * s->H * sets, sms) * (kBands / sets);
    if (sets == 1 || bands < best) {
      best = bands;
      a.sets = sets;
    }
  }
  a.jobs = (int)(tiles * s->H * a.sets);
  a.wait_limit_ns = wait_limit_ns;
  a.withhold_first_copy = withhold;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.jobs < sms ? a.jobs : sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, absorb_kernel, a, tq, tw, to);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace

extern "C" int32_t mla_query_absorb(const mla_query_shape* s, const void* q, const void* w_uk,
                                    const float* rope, const int32_t* rope_starts, float q_scale,
                                    void* out, int32_t* status, mla_stream_t stream) {
  return absorb_impl(s, q, w_uk, rope, rope_starts, q_scale, out, status, stream, kWaitLimitNs, 0);
}

extern "C" int32_t mla_query_absorb_wait_test(const mla_query_shape* s, const void* q,
                                              const void* w_uk, const float* rope,
                                              const int32_t* rope_starts, float q_scale, void* out,
                                              int32_t* status, int32_t withhold,
                                              uint64_t wait_limit_ns, mla_stream_t stream) {
  if (!status) return MLA_ERR_NULL;
  if (wait_limit_ns < 1000000ull || wait_limit_ns > kWaitLimitNs || (withhold != 0 && withhold != 1))
    return MLA_ERR_SHAPE;
  return absorb_impl(s, q, w_uk, rope, rope_starts, q_scale, out, status, stream, wait_limit_ns,
                     withhold);
}
