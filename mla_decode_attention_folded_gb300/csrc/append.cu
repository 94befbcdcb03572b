// New tokens into the paged FP8 latent cache: the RMS norm of the 512 latent
// dims, the rotation of the 64 rope dims, E4M3 codes through the block table.
//
//   y[0:512]   = x[0:512] * rsqrt(mean(x[0:512]^2) + eps) * w     (w NULL: y = x)
//   y[512:576] = x[512:576], its 32 planes turned by the angles of the token's position
//   kv[block_table[r][j / 64]][j % 64] = e4m3(y / kv_scale),  j = starts[r] + i
//
// Bound by HBM for prompts (1152 B in, 576 B out and 256 B of angles, which
// neighbouring requests share in L2, per token) and by launch latency for
// decode steps. One warp per token: each lane holds 16 latent dims in
// registers between the sum of squares (five shuffles) and the stores, so a
// row is read once; lane p turns plane p. 24 ragged prompts, 101 k tokens: 31.1 - 31.8
// us, 5.6 TB/s (0.82 of the copy rate, 0.95 with the angles; issue slots 75 % busy);
// 128 x 7 tokens 2.1 - 2.3 us, 2 x 4 1.9 - 2.2 us. Warps that step over several tokens with the
// norm's weights in registers were slower (32.7 us: 55 registers). Every value is FP32
// from load to the one rounding to E4M3 (round to nearest even, saturating), the format
// the decode reads.
#include <cmath>

#include "checks.h"
#include "formats.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace mlafold {
namespace {

constexpr int kWarps = 4;

struct AppendArgs {
  const uint16_t* x;            // [tokens] rows of row_stride BF16
  const uint16_t* weight;       // [512] BF16, or null: no norm
  const float* rope;            // [rope_rows][32 cos, 32 sin]
  const int32_t* cu;            // [R + 1], or null: tokens / R each
  const int32_t* starts;        // [R]
  const int32_t* rope_starts;   // [R], or null: starts
  const int32_t* block_table;   // [R][max_pages]
  uint8_t* kv;                  // [num_pages][64][576]
  int32_t* status;              // may be null
  long long row_stride;
  float eps, inv_scale;
  int R, tokens, max_pages, num_pages, rope_rows;
};

// The request of row t in a ragged batch: the last r with cu[r] <= t, found by
// the warp 32 entries at a time. With cu out of order some r comes out; the
// caller checks cu[r] <= t < cu[r + 1] before it uses it.
__device__ __forceinline__ int ragged_request(const int32_t* cu, int R, int t, int lane) {
  int lo = 0, n = R;                        // entries cu[lo .. lo + n - 1] are candidates
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const bool le = lane * step < n && cu[lo + lane * step] <= t;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int hit = m ? 31 - __clz(m) : 0;
    const int end = lo + n;
    lo += hit * step;
    n = min(step, end - lo);
  }
  return lo;
}

// JOINS: the scale's reciprocal joins the norm's factor (16 products fewer).
template <bool INTERLEAVED, bool JOINS>
__global__ void __launch_bounds__(kWarps * 32) append_kernel(const AppendArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= a.tokens) return;
  const uint16_t* x = a.x + (long long)t * a.row_stride;
  const uint4 v0 = reinterpret_cast<const uint4*>(x)[lane];           // dims 8 lane ..
  const uint4 v1 = reinterpret_cast<const uint4*>(x + 256)[lane];     // dims 256 + 8 lane ..
  uint32_t p0, p1;                                                    // this lane's plane
  if (INTERLEAVED) {
    const uint32_t w = reinterpret_cast<const uint32_t*>(x + kDv)[lane];
    p0 = w << 16;
    p1 = w & 0xFFFF0000u;
  } else {
    p0 = (uint32_t)x[kDv + lane] << 16;
    p1 = (uint32_t)x[kDv + 32 + lane] << 16;
  }

  int r;
  long long i;                                        // offsets that are none may lie 2^31 below t
  if (a.cu) {
    r = ragged_request(a.cu, a.R, t, lane);
    const int first = a.cu[r];
    if (t < first || t >= a.cu[r + 1]) return;        // rows of no request
    i = (long long)t - first;
  } else {
    const int k = a.tokens / a.R;
    r = t / k;
    i = t - r * k;
  }
  const int start = a.starts[r];
  if (start < 0) return;                              // a padding request
  const long long j = start + i;                      // >= 0, as both are
  const long long pos = (a.rope_starts ? a.rope_starts[r] : start) + i;
  int page = -1;
  if (j < (long long)a.max_pages * kPage) page = a.block_table[(long long)r * a.max_pages + j / kPage];
  const bool page_ok = page >= 0 && page < a.num_pages, pos_ok = pos >= 0 && pos < a.rope_rows;
  if (!page_ok || !pos_ok) {
    if (a.status && lane == 0)
      atomicOr(a.status, (page_ok ? 0 : MLA_FAULT_PAGE_RANGE) | (pos_ok ? 0 : MLA_FAULT_ROPE_RANGE));
    return;
  }
  const float c = a.rope[pos * 64 + lane], s = a.rope[pos * 64 + 32 + lane];

  float f[16];
  bf16x8_to_f32(v0, f);
  bf16x8_to_f32(v1, f + 8);
  if (a.weight) {
    float ss = 0.f;
#pragma unroll
    for (int u = 0; u < 16; ++u) ss += f[u] * f[u];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float n = rsqrtf(ss * (1.f / kDv) + a.eps);
    float w[16];
    bf16x8_to_f32(reinterpret_cast<const uint4*>(a.weight)[lane], w);
    bf16x8_to_f32(reinterpret_cast<const uint4*>(a.weight + 256)[lane], w + 8);
    const float rs = JOINS ? n * a.inv_scale : n;
#pragma unroll
    for (int u = 0; u < 16; ++u) f[u] = f[u] * rs * w[u];
    if (!JOINS)
#pragma unroll
      for (int u = 0; u < 16; ++u) f[u] *= a.inv_scale;
  } else {
#pragma unroll
    for (int u = 0; u < 16; ++u) f[u] *= a.inv_scale;
  }
  uint8_t* dst = a.kv + ((size_t)page * kPage + (size_t)(j % kPage)) * kDqk;
  reinterpret_cast<uint2*>(dst)[lane] =
      make_uint2(f32x4_to_e4m3x4(f[0], f[1], f[2], f[3]), f32x4_to_e4m3x4(f[4], f[5], f[6], f[7]));
  reinterpret_cast<uint2*>(dst + 256)[lane] = make_uint2(
      f32x4_to_e4m3x4(f[8], f[9], f[10], f[11]), f32x4_to_e4m3x4(f[12], f[13], f[14], f[15]));
  const float x0 = __uint_as_float(p0), x1 = __uint_as_float(p1);
  const uint16_t e = f32x2_to_e4m3x2((x0 * c - x1 * s) * a.inv_scale,
                                     (x1 * c + x0 * s) * a.inv_scale);
  if (INTERLEAVED) {
    reinterpret_cast<uint16_t*>(dst + kDv)[lane] = e;
  } else {
    dst[kDv + lane] = (uint8_t)e;
    dst[kDv + 32 + lane] = (uint8_t)(e >> 8);
  }
}

}  // namespace
}  // namespace mlafold

using namespace mlafold;

extern "C" int32_t mla_kv_append(const mla_append_shape* s, const void* kv_new,
                                 const void* norm_weight, float norm_eps, const float* rope,
                                 const int32_t* cu_tokens, const int32_t* starts,
                                 const int32_t* rope_starts, const int32_t* block_table,
                                 float kv_scale, void* kv, int32_t* status, mla_stream_t stream) {
  if (!s) return MLA_ERR_NULL;
  if (s->page_size != kPage) return MLA_ERR_UNSUPPORTED;
  if (s->R < 1 || s->R > (1 << 20) || s->tokens < 0 || s->max_pages < 1 ||
      s->max_pages >= (1 << 25) || s->num_pages < 1 || s->num_pages >= (1 << 25) ||
      s->rope_rows < 1 || (s->interleaved != 0 && s->interleaved != 1) ||
      s->row_stride < kDqk || (!cu_tokens && s->tokens % s->R != 0))
    return MLA_ERR_SHAPE;
  if (!std::isfinite(kv_scale) || !(kv_scale > 0.f) || !std::isfinite(1.0f / kv_scale) ||
      !std::isfinite(norm_eps) || norm_eps < 0.f)
    return MLA_ERR_SHAPE;
  if (s->tokens == 0) return MLA_OK;
  if (!kv_new || !rope || !starts || !block_table || !kv) return MLA_ERR_NULL;
  if (!aligned(kv_new, 16) || s->row_stride % 8 != 0 || !aligned(norm_weight, 16) ||
      !aligned(kv, 16) || !aligned(rope, 4) || !aligned(cu_tokens, 4) || !aligned(starts, 4) ||
      !aligned(rope_starts, 4) || !aligned(block_table, 4) || !aligned(status, 4))
    return MLA_ERR_ALIGN;
  int st = check_device();
  if (st != MLA_OK) return st;
  AppendArgs a;
  a.x = static_cast<const uint16_t*>(kv_new);
  a.weight = static_cast<const uint16_t*>(norm_weight);
  a.rope = rope;
  a.cu = cu_tokens;
  a.starts = starts;
  a.rope_starts = rope_starts;
  a.block_table = block_table;
  a.kv = static_cast<uint8_t*>(kv);
  a.status = status;
  a.row_stride = s->row_stride;
  a.eps = norm_eps;
  a.inv_scale = 1.0f / kv_scale;
  a.R = s->R;
  a.tokens = s->tokens;
  a.max_pages = s->max_pages;
  a.num_pages = s->num_pages;
  a.rope_rows = s->rope_rows;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)cdiv(s->tokens, kWarps));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // With a scale near FP32's ends the norm's factor times its reciprocal could overflow, and
  // 0 times that be NaN: the products are then apart (24 prompts: 31.9 against 31.5 us).
  const bool joins = a.inv_scale > 0x1p-40f && a.inv_scale < 0x1p40f;
  auto* kernel = s->interleaved ? (joins ? append_kernel<true, true> : append_kernel<true, false>)
                                : (joins ? append_kernel<false, true> : append_kernel<false, false>);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
