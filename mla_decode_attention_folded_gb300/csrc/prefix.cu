// Decode of a batch whose requests share a prefix: every row of the batch
// attends to the prefix's keys, which are read once for all requests, and to
// its own request's keys; one softmax over both.
//
//   s[n][j] = bmm1 * q[n] . kv[key j],  j over the prefix's keys, then the request's own
//   out[n]  = bmm2 * sum_j softmax_j(s[n]) kv[key j][0:512],  lse[n] = log2 sum_j 2^(s log2 e)
//
// The softmax splits over key sets by their LSEs: prefix_wide.cu decodes blocks
// of rows against the prefix's keys and against the requests' own, in equal
// parts, into FP32 partials; the merge below joins all of a row's partials and
// rounds once to BF16. The plan is the line of work of prefix.h: one CTA, one
// thread per request, a scan. Where it does not serve the lengths at hand, wide_kernel
// and the merge lay them out themselves.
//
// The merge is bound by memory: per row, its partials (2 KB each) in, 1 KB out.
// One warp per row; the lanes hold the partials' LSEs and share weights by
// shuffles, as the split reducer does. 128 x 7 x 64 behind 16k: 57 us for 271 MB of
// partials and 59 MB out (5.8 TB/s); 64 x 7 x 8: 11 us from DRAM, where the loads'
// latency counts.
#include "checks.h"
#include "internal.h"
#include "prefix.h"
#include "ptx.cuh"

namespace mlafold {
namespace {

constexpr int kWarps = 8;                  // rows per CTA

__global__ void __launch_bounds__(kMaxR)
prefix_plan_kernel(const int32_t* __restrict__ seq_lens, int R, int max_pages, int own_blocks,
                   int32_t* __restrict__ plan) {
  __shared__ int s_warp[32];
  grid_dep_wait();
  grid_dep_launch();
  const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
  int sum = i < R ? wide_places(wide_len(seq_lens[i], max_pages), own_blocks) : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += t;
  }
  if (lane == 31) s_warp[warp] = sum;
  __syncthreads();
  for (int w = 0; w < warp; ++w) sum += s_warp[w];
  if (i < R) plan[i + 1] = sum;
  if (i == 0) plan[0] = 0;
}

struct MergeArgs {
  const int32_t* prefix_len;               // [1]
  const int32_t* plan;                     // [R + 1]
  const int32_t* seq_lens;                 // [R]
  const float* part_o;                     // [slots][128][512]
  const float* part_lse;                   // [slots][128]
  uint16_t* out;                           // [N][512]
  float* lse;                              // [N], may be null
  float bmm2;
  int R, M, prefix_pages, max_pages, units, blocks, own_blocks;
};

// EARLY: the first two partials are asked for before any LSE is there, at 99 registers.
template <bool EARLY>
__global__ void __launch_bounds__(kWarps * 32, EARLY ? 2 : 4)
prefix_merge_kernel(const MergeArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  __shared__ int s_before, s_all;
  const int r = blockIdx.y, lane = threadIdx.x & 31;
  const int m = blockIdx.x * kWarps + (threadIdx.x >> 5);
  // The places of the request, and of all: the plan's, unless wide_kernel made its own.
  int own = r > 0 ? a.plan[r] : 0, own_end = a.plan[r + 1], own_places = a.plan[a.R];
  if (a.plan[0] != 0) {
    if (threadIdx.x == 0) s_before = s_all = 0;
    __syncthreads();
    const auto places = [&](int i) {
      return wide_places(wide_len(a.seq_lens[i], a.max_pages), a.own_blocks);
    };
    int before = 0, all = 0;
    for (int i = threadIdx.x; i < a.R; i += kWarps * 32) {
      all += places(i);
      if (i < r) before += places(i);
    }
    atomicAdd(&s_before, before);
    atomicAdd(&s_all, all);
    __syncthreads();
    own = s_before;
    own_end = own + places(r);
    own_places = s_all;
  }
  if (m >= a.M) return;
  const size_t row = (size_t)r * a.M + m;
  const WideLine line(*a.prefix_len, own_places, a.prefix_pages, a.blocks, a.units);
  // The pieces of this row's two segments, in consecutive slots each.
  int n_pre = 0, n_own = 0;
  size_t pre = 0, mine = 0;
  auto pieces = [&](int first, int tiles, int segment, int in_block, size_t& at) {
    const int u0 = line.unit_of(first), u1 = line.unit_of(first + tiles - 1);
    at = (size_t)(u0 + segment) * kWideRows + in_block;
    return u1 - u0 + 1;
  };
  if (line.prefix_tiles > 0) {
    const int b = (int)(row / kWideRows);
    n_pre = pieces(b * (line.prefix_tiles + kWideCost), line.prefix_tiles, b,
                   (int)(row % kWideRows), pre);
  }
  const int span = (int)((unsigned)(own_end - own) / (unsigned)a.own_blocks);
  if (span > 0) {
    const int j = m / kWideRows;
    n_own = pieces(line.prefix_places + own + j * span, wide_own_tiles(span),
                   a.blocks + r * a.own_blocks + j, m % kWideRows, mine);
  }
  const int n = n_pre + n_own;
  auto at = [&](int s) {
    return s < n_pre ? pre + (size_t)s * kWideRows : mine + (size_t)(s - n_pre) * kWideRows;
  };
  float4 early[2][4] = {};
#pragma unroll
  for (int s = 0; s < 2; ++s)
    if (EARLY && s < n)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        early[s][v] = reinterpret_cast<const float4*>(a.part_o + at(s) * kDv)[v * 32 + lane];
  float mx = -INFINITY;
  for (int s = lane; s < n; s += 32) mx = fmaxf(mx, a.part_lse[at(s)]);
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  // fmaxf passes over a NaN LSE: where all others are empty too, mx is still -inf. The
  // weights then are 2^NaN, not 0: only empty partials weigh nothing.
  const float base = mx == -INFINITY ? 0.f : mx;
  float4 acc[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](int v, float w, const float4& o) {
    acc[v].x += w * o.x; acc[v].y += w * o.y; acc[v].z += w * o.z; acc[v].w += w * o.w;
  };
  float z = 0.f;
  for (int c0 = 0; c0 < n; c0 += 32) {
    const float lc = c0 + lane < n ? a.part_lse[at(c0 + lane)] : -INFINITY;
    const float wc = lc == -INFINITY ? 0.f : ex2(lc - base);
    z += wc;
    const int cn = min(32, n - c0);
    int s = 0;
    if (EARLY && c0 == 0) {
#pragma unroll
      for (; s < 2; ++s) {
        const float w = __shfl_sync(0xffffffffu, wc, s);       // 0 past the last partial
#pragma unroll
        for (int v = 0; v < 4; ++v) add(v, w, early[s][v]);
      }
    }
#pragma unroll 2
    for (; s < cn; ++s) {
      const float w = __shfl_sync(0xffffffffu, wc, s);
      const float4* src = reinterpret_cast<const float4*>(a.part_o + at(c0 + s) * kDv);
#pragma unroll
      for (int v = 0; v < 4; ++v) add(v, w, src[v * 32 + lane]);
    }
  }
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  const float scale = z > 0.f ? a.bmm2 / z : z;          // NaN stays
  uint2* dst = reinterpret_cast<uint2*>(a.out + row * kDv);
#pragma unroll
  for (int v = 0; v < 4; ++v)
    dst[v * 32 + lane] =
        make_uint2((uint32_t)f32_to_bf16_bits(acc[v].x * scale) |
                       ((uint32_t)f32_to_bf16_bits(acc[v].y * scale) << 16),
                   (uint32_t)f32_to_bf16_bits(acc[v].z * scale) |
                       ((uint32_t)f32_to_bf16_bits(acc[v].w * scale) << 16));
  if (a.lse && lane == 0) a.lse[row] = z == 0.f ? -INFINITY : base + __log2f(z);
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Row blocks of the batch and of a request, and pairs of CTAs.
int wide_blocks(const mla_shape& s) { return (int)cdiv((long long)s.R * s.k * s.H, kWideRows); }
int wide_own_blocks(const mla_shape& s) { return (int)cdiv(s.k * s.H, kWideRows); }
int wide_units(const mla_shape& s) { return s.num_ctas / 2 > 0 ? s.num_ctas / 2 : 1; }

// Workspace: FP32 partials [slots][128][512], then their LSEs [slots][128].
size_t wide_rows(const mla_shape& s) {
  return ((size_t)wide_units(s) + wide_blocks(s) + (size_t)s.R * wide_own_blocks(s) - 1) * kWideRows;
}
size_t wide_out_bytes(const mla_shape& s) { return align256(wide_rows(s) * kDv * 4); }
size_t wide_bytes(const mla_shape& s) { return wide_out_bytes(s) + align256(wide_rows(s) * 4); }

// Places on the line of work: 31 bits hold them.
bool places_fit(const mla_shape& s, int prefix_pages) {
  const long long prefix =
      wide_blocks(s) * (cdiv((long long)prefix_pages * kPage, kWideKeys) + kWideCost);
  return prefix + wide_own_most(s.R, wide_own_blocks(s), s.max_pages) < (1LL << 31) &&
         wide_rows(s) < (1ull << 31);
}

int check_prefix_shape(const mla_shape* s) {
  const int st = check_shape(s);
  if (st != MLA_OK) return st;
  return shape_groups(*s) == 1 && places_fit(*s, 1) ? MLA_OK : MLA_ERR_SHAPE;
}

}  // namespace
}  // namespace mlafold

using namespace mlafold;

extern "C" int32_t mla_prefix_workspace_bytes(const mla_shape* shape, size_t* bytes) {
  const int st = check_prefix_shape(shape);
  if (st != MLA_OK) return st;
  if (!bytes) return MLA_ERR_NULL;
  *bytes = wide_bytes(*shape);
  return MLA_OK;
}

extern "C" int32_t mla_prefix_plan(const mla_shape* shape, const int32_t* seq_lens, int32_t* plan,
                                   int32_t plan_len, mla_stream_t stream) {
  int st = check_prefix_shape(shape);
  if (st != MLA_OK) return st;
  if (!seq_lens || !plan) return MLA_ERR_NULL;
  if (!aligned(seq_lens, 4) || !aligned(plan, 4)) return MLA_ERR_ALIGN;
  if (plan_len < shape->R + 1) return MLA_ERR_LIST;
  if ((st = check_device()) != MLA_OK) return st;
  const cudaError_t e =
      launch(prefix_plan_kernel, dim3(1), (shape->R + 31) / 32 * 32,
             reinterpret_cast<cudaStream_t>(stream), seq_lens, shape->R, shape->max_pages,
             wide_own_blocks(*shape), plan);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

namespace {

// test_limit_ns: 0, or the failure-detection test's (WideArgs::wait_limit_ns).
int32_t decode_impl(const mla_shape* shape, int32_t prefix_pages, const void* q, const void* kv,
                    const int32_t* prefix_table, const int32_t* prefix_len,
                    const int32_t* block_table, const int32_t* seq_lens, float bmm1_scale,
                    float bmm2_scale, int32_t* plan, int32_t plan_len, void* workspace,
                    size_t workspace_bytes_given, void* out, float* lse, int32_t* status,
                    mla_stream_t stream, unsigned long long test_limit_ns) {
  int st = check_prefix_shape(shape);
  if (st != MLA_OK) return st;
  if (prefix_pages < 1 || prefix_pages > (1 << 24) || !places_fit(*shape, prefix_pages))
    return MLA_ERR_SHAPE;
  if (!q || !kv || !prefix_table || !prefix_len || !block_table || !seq_lens || !plan ||
      !workspace || !out)
    return MLA_ERR_NULL;
  if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
      !aligned(prefix_table, 4) || !aligned(prefix_len, 4) || !aligned(block_table, 4) ||
      !aligned(seq_lens, 4) || !aligned(plan, 4) || !aligned(workspace, 256) || !aligned(status, 4))
    return MLA_ERR_ALIGN;
  if (plan_len < shape->R + 1) return MLA_ERR_LIST;
  if (workspace_bytes_given < wide_bytes(*shape)) return MLA_ERR_WORKSPACE;
  if (!scales_ok(bmm1_scale, bmm2_scale)) return MLA_ERR_SHAPE;
  if ((st = check_device()) != MLA_OK) return st;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  WideArgs w;
  w.prefix_table = prefix_table;
  w.prefix_len = prefix_len;
  w.block_table = block_table;
  w.seq_lens = seq_lens;
  w.plan = plan;
  w.part_o = static_cast<float*>(workspace);
  w.part_lse = reinterpret_cast<float*>(static_cast<char*>(workspace) + wide_out_bytes(*shape));
  w.status = status;
  w.bmm1_log2 = (float)((double)bmm1_scale * 1.4426950408889634);
  w.N = (long long)shape->R * shape->k * shape->H;
  w.R = shape->R;
  w.M = shape->k * shape->H;
  w.prefix_pages = prefix_pages;
  w.max_pages = shape->max_pages;
  w.num_pages = shape->num_pages;
  w.units = wide_units(*shape);
  w.blocks = wide_blocks(*shape);
  w.own_blocks = wide_own_blocks(*shape);
  w.own_tiles = (int)cdiv((long long)w.max_pages * kPage, kWideKeys);
  w.own_most = (int)wide_own_most(w.R, w.own_blocks, w.max_pages);
  w.wait_limit_ns = test_limit_ns;
  if (launch_wide(w, static_cast<const uint8_t*>(q), static_cast<const uint8_t*>(kv), cs) !=
      cudaSuccess)
    return MLA_ERR_CUDA;
  MergeArgs m;
  m.prefix_len = prefix_len;
  m.plan = w.plan;
  m.seq_lens = seq_lens;
  m.part_o = w.part_o;
  m.part_lse = w.part_lse;
  m.out = static_cast<uint16_t*>(out);
  m.lse = lse;
  m.bmm2 = bmm2_scale;
  m.R = w.R;
  m.M = w.M;
  m.prefix_pages = prefix_pages;
  m.max_pages = w.max_pages;
  m.units = w.units;
  m.blocks = w.blocks;
  m.own_blocks = w.own_blocks;
  // While all rows are resident at once, a row's chain of loads is what the merge takes:
  // the early one (2 x 4 x 8 behind 300 17.8 against 20.0 us with plan and decode, 32 x 4 x 8
  // behind 4k 27.4 against 30.7, 24 x 1 x 64 behind 64k 113 against 118). With more rows,
  // warps in flight count (128 x 7 x 64 behind 16k 1205 against 1186).
  const dim3 grid((unsigned)cdiv(w.M, kWarps), (unsigned)w.R);
  const bool early = (long long)grid.x * grid.y <= 2LL * shape->num_ctas;
  return launch(early ? prefix_merge_kernel<true> : prefix_merge_kernel<false>, grid, kWarps * 32,
                cs, m) == cudaSuccess
             ? MLA_OK
             : MLA_ERR_CUDA;
}

}  // namespace

extern "C" int32_t mla_prefix_decode(const mla_shape* shape, int32_t prefix_pages, const void* q,
                                     const void* kv, const int32_t* prefix_table,
                                     const int32_t* prefix_len, const int32_t* block_table,
                                     const int32_t* seq_lens, float bmm1_scale, float bmm2_scale,
                                     int32_t* plan, int32_t plan_len, void* workspace,
                                     size_t workspace_bytes_given, void* out, float* lse,
                                     int32_t* status, mla_stream_t stream) {
  return decode_impl(shape, prefix_pages, q, kv, prefix_table, prefix_len, block_table, seq_lens,
                     bmm1_scale, bmm2_scale, plan, plan_len, workspace, workspace_bytes_given, out,
                     lse, status, stream, 0);
}

extern "C" int32_t mla_prefix_decode_wait_test(
    const mla_shape* shape, int32_t prefix_pages, const void* q, const void* kv,
    const int32_t* prefix_table, const int32_t* prefix_len, const int32_t* block_table,
    const int32_t* seq_lens, float bmm1_scale, float bmm2_scale, int32_t* plan, int32_t plan_len,
    void* workspace, size_t workspace_bytes_given, void* out, float* lse, int32_t* status,
    uint64_t wait_limit_ns, mla_stream_t stream) {
  if (!status) return MLA_ERR_NULL;
  if (wait_limit_ns < 1000000ull || wait_limit_ns > 2000000000ull) return MLA_ERR_SHAPE;
  return decode_impl(shape, prefix_pages, q, kv, prefix_table, prefix_len, block_table, seq_lens,
                     bmm1_scale, bmm2_scale, plan, plan_len, workspace, workspace_bytes_given, out,
                     lse, status, stream, wait_limit_ns);
}
