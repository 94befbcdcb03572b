// Decode of a batch whose requests share a prefix: every row of the batch
// attends to the prefix's keys, which are read once for all requests, and to
// its own request's keys; one softmax over both.
//
//   s[n][j] = bmm1 * q[n] . kv[key j],  j over the prefix's keys, then the request's own
//   out[n]  = bmm2 * sum_j softmax_j(s[n]) kv[key j][0:512],  lse[n] = log2 sum_j 2^(s log2 e)
//
// The softmax splits over key sets by their LSEs: the prefix against all R*k*H
// rows (prefix_wide.cu), the requests' own keys by the planned decode, both into
// FP32 partials; the merge below joins all of a row's partials and rounds once
// to BF16.
//
// The merge is bound by memory: per row, the partials of its prefix pieces and
// of its own splits (2 KB each) in, 1 KB out. One warp per row; the lanes hold
// the partials' LSEs and share weights by shuffles, as the split reducer does.
#include "internal.h"
#include "prefix.h"
#include "ptx.cuh"

namespace mlafold {
namespace {

constexpr int kWarps = 8;                  // rows per CTA

struct MergeArgs {
  const int32_t* counts;                   // [R] splits of each request's own keys
  const int32_t* work;                     // their work list
  const int32_t* prefix_len;               // [1]
  const float* prefix_o;                   // [units + blocks - 1][128][512]
  const float* prefix_lse;                 // [units + blocks - 1][128]
  const float* own_o;                      // [slots][M][512]
  const float* own_lse;                    // [slots][M]
  uint16_t* out;                           // [N][512]
  float* lse;                              // [N], may be null
  float bmm2;
  int R, M, slots, prefix_pages, units, blocks;
};

__global__ void __launch_bounds__(kWarps * 32) prefix_merge_kernel(const MergeArgs a) {
  __shared__ int s_start;
  grid_dep_wait();
  grid_dep_launch();
  const int r = blockIdx.y, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) s_start = -1;
  __syncthreads();
  // The request's first partial slot: the list index of its split 0.
  for (int e = threadIdx.x; e < a.slots; e += blockDim.x) {
    const int w = a.work[e];
    if (w >= 0 && entry_request(w) == r && entry_split(w) == 0) s_start = e;
  }
  __syncthreads();
  const int start = s_start;
  int n_own = a.counts[r];
  if (start < 0 || n_own < 1 || start + n_own > a.slots) n_own = 0;   // not a plan of this shape
  const int tiles = (int)cdiv(wide_len(a.prefix_len, a.prefix_pages, nullptr, false), kWideKeys);
  const long long total = (long long)tiles * a.blocks;
  const long long used = total < a.units ? total : a.units;
  for (int m = blockIdx.x * kWarps + (threadIdx.x >> 5); m < a.M; m += gridDim.x * kWarps) {
    const size_t row = (size_t)r * a.M + m;
    // The prefix's pieces of this row's block, in consecutive slots.
    const long long block = row / kWideRows;
    int n_pre = 0;
    size_t pre = 0;
    if (tiles > 0) {
      const int u0 = wide_unit_of(block * tiles, total, used);
      n_pre = wide_unit_of((block + 1) * tiles - 1, total, used) - u0 + 1;
      pre = (size_t)(u0 + block) * kWideRows + row % kWideRows;
    }
    const int n = n_pre + n_own;
    // Partial s of this row: first the prefix's pieces, then the request's splits.
    auto lse_of = [&](int s) {
      return s < n_pre ? a.prefix_lse[pre + (size_t)s * kWideRows]
                       : a.own_lse[(size_t)(start + s - n_pre) * a.M + m];
    };
    auto row_of = [&](int s) {
      return reinterpret_cast<const float4*>(
          s < n_pre ? a.prefix_o + (pre + (size_t)s * kWideRows) * kDv
                    : a.own_o + ((size_t)(start + s - n_pre) * a.M + m) * kDv);
    };
    float mx = -INFINITY;
    for (int s = lane; s < n; s += 32) mx = fmaxf(mx, lse_of(s));
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    float4 acc[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
    float z = 0.f;
    for (int c0 = 0; c0 < n; c0 += 32) {
      const float lc = c0 + lane < n ? lse_of(c0 + lane) : -INFINITY;
      const float wc = (mx == -INFINITY || lc == -INFINITY) ? 0.f : ex2(lc - mx);
      z += wc;
      const int cn = min(32, n - c0);
#pragma unroll 2
      for (int s = 0; s < cn; ++s) {
        const float w = __shfl_sync(0xffffffffu, wc, s);
        const float4* src = row_of(c0 + s);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float4 o = src[v * 32 + lane];
          acc[v].x += w * o.x; acc[v].y += w * o.y; acc[v].z += w * o.z; acc[v].w += w * o.w;
        }
      }
    }
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    const float scale = z > 0.f ? a.bmm2 / z : 0.f;
    uint2* dst = reinterpret_cast<uint2*>(a.out + row * kDv);
#pragma unroll
    for (int v = 0; v < 4; ++v)
      dst[v * 32 + lane] =
          make_uint2((uint32_t)f32_to_bf16_bits(acc[v].x * scale) |
                         ((uint32_t)f32_to_bf16_bits(acc[v].y * scale) << 16),
                     (uint32_t)f32_to_bf16_bits(acc[v].z * scale) |
                         ((uint32_t)f32_to_bf16_bits(acc[v].w * scale) << 16));
    if (a.lse && lane == 0) a.lse[row] = z == 0.f ? -INFINITY : mx + __log2f(z);
  }
}

cudaError_t launch_merge(const MergeArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)cdiv(a.M, kWarps), (unsigned)a.R);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefix_merge_kernel, a);
}

// Row blocks of the batch and CTA pairs of the wide kernel.
int wide_blocks(const mla_shape& s) { return (int)cdiv((long long)s.R * s.k * s.H, kWideRows); }
int wide_units(const mla_shape& s) { return s.num_ctas / 2 > 0 ? s.num_ctas / 2 : 1; }

// Workspace offsets. Every split of a request's own keys has a partial, so
// that one-split rows too reach the merge unrounded.
struct Layout {
  size_t prefix_o, prefix_lse, own_o, own_lse, bytes;
};
Layout layout(const mla_shape& s) {
  const size_t ps = (size_t)(wide_units(s) + wide_blocks(s) - 1) * kWideRows;
  const size_t os = (size_t)plan_items(s) * s.k * s.H;
  Layout l;
  l.prefix_o = 0;
  l.prefix_lse = l.prefix_o + align256(ps * kDv * 4);
  l.own_o = l.prefix_lse + align256(ps * 4);
  l.own_lse = l.own_o + align256(os * kDv * 4);
  l.bytes = l.own_lse + align256(os * 4);
  return l;
}

int check_prefix_shape(const mla_shape* s, int prefix_pages) {
  const int st = check_shape(s);
  if (st != MLA_OK) return st;
  if (shape_groups(*s) != 1 || prefix_pages < 1 || prefix_pages > (1 << 24)) return MLA_ERR_SHAPE;
  return MLA_OK;
}

}  // namespace
}  // namespace mlafold

using namespace mlafold;

extern "C" int32_t mla_prefix_workspace_bytes(const mla_shape* shape, int32_t prefix_pages,
                                              size_t* bytes) {
  const int st = check_prefix_shape(shape, prefix_pages);
  if (st != MLA_OK) return st;
  if (!bytes) return MLA_ERR_NULL;
  *bytes = layout(*shape).bytes;
  return MLA_OK;
}

extern "C" int32_t mla_prefix_decode(const mla_shape* shape, int32_t prefix_pages, const void* q,
                                     const void* kv, const int32_t* prefix_table,
                                     const int32_t* prefix_len, const int32_t* block_table,
                                     const int32_t* seq_lens, float bmm1_scale, float bmm2_scale,
                                     const int32_t* counts, int32_t* work, int32_t list_len,
                                     void* workspace, size_t workspace_bytes_given, void* out,
                                     float* lse, int32_t* status, mla_stream_t stream) {
  int st = check_prefix_shape(shape, prefix_pages);
  if (st != MLA_OK) return st;
  if (!q || !kv || !prefix_table || !prefix_len || !block_table || !seq_lens || !counts || !work ||
      !workspace || !out)
    return MLA_ERR_NULL;
  if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(prefix_table, 4) || !aligned(prefix_len, 4) || !aligned(block_table, 4) ||
      !aligned(seq_lens, 4) || !aligned(counts, 4) || !aligned(work, 4) ||
      !aligned(workspace, 256) || !aligned(status, 4))
    return MLA_ERR_ALIGN;
  if (list_len < plan_list_len(*shape)) return MLA_ERR_LIST;
  const Layout l = layout(*shape);
  if (workspace_bytes_given < l.bytes) return MLA_ERR_WORKSPACE;
  if (!scales_ok(bmm1_scale, bmm2_scale)) return MLA_ERR_SHAPE;
  if ((st = check_device()) != MLA_OK) return st;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  WideArgs w;
  w.prefix_table = prefix_table;
  w.prefix_len = prefix_len;
  w.part_o = reinterpret_cast<float*>(ws + l.prefix_o);
  w.part_lse = reinterpret_cast<float*>(ws + l.prefix_lse);
  w.status = status;
  w.bmm1_log2 = (float)((double)bmm1_scale * 1.4426950408889634);
  w.N = (long long)shape->R * shape->k * shape->H;
  w.prefix_pages = prefix_pages;
  w.num_pages = shape->num_pages;
  w.units = wide_units(*shape);
  w.blocks = wide_blocks(*shape);
  if (launch_wide(w, static_cast<const uint8_t*>(q), static_cast<const uint8_t*>(kv), cs) !=
      cudaSuccess)
    return MLA_ERR_CUDA;
  DecodeArgs a = decode_args(*shape, q, kv, block_table, seq_lens, bmm1_scale, 1.f, counts, work, out, nullptr,
                  status);
  a.part_o = reinterpret_cast<float*>(ws + l.own_o);
  a.part_lse = reinterpret_cast<float*>(ws + l.own_lse);
  a.slots = plan_items(*shape);
  a.all_partial = 1;
  if (launch_decode(*shape, a, cs) != cudaSuccess) return MLA_ERR_CUDA;
  MergeArgs m;
  m.counts = counts;
  m.work = work;
  m.prefix_len = prefix_len;
  m.prefix_o = w.part_o;
  m.prefix_lse = w.part_lse;
  m.own_o = reinterpret_cast<const float*>(ws + l.own_o);
  m.own_lse = reinterpret_cast<const float*>(ws + l.own_lse);
  m.out = static_cast<uint16_t*>(out);
  m.lse = lse;
  m.bmm2 = bmm2_scale;
  m.R = shape->R;
  m.M = shape->k * shape->H;
  m.slots = plan_items(*shape);
  m.prefix_pages = prefix_pages;
  m.units = w.units;
  m.blocks = w.blocks;
  return launch_merge(m, cs) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
