// moe.cu -- the mixture-of-experts layer for a few tokens (gptq_moe): the router's kernel, the
// workspace and the launches of the expert products (moe.cuh).
//
// The router's kernel: a CTA takes one expert and four tokens, its warps a share of hidden each, and
// writes their logits, summed in fp32 (a warp alone for all of hidden took 13 us at one token); further
// CTAs rewrite the activations as the expert products read them (store_run) and zero the arrival
// counters of the expert products.
#include "gptq_device.cuh"
#include "gptq_internal.h"
#include "moe.cuh"
#include "serving_internal.h"

namespace gptq {

cudaError_t launch_moe_b2(const moe::Args&, const int32_t*, const moe::Args&, const int32_t*, int, int*, cudaStream_t);
cudaError_t launch_moe_b3(const moe::Args&, const int32_t*, const moe::Args&, const int32_t*, int, int*, cudaStream_t);
cudaError_t launch_moe_b4(const moe::Args&, const int32_t*, const moe::Args&, const int32_t*, int, int*, cudaStream_t);
cudaError_t launch_moe_b8(const moe::Args&, const int32_t*, const moe::Args&, const int32_t*, int, int*, cudaStream_t);

namespace moe {
namespace {

constexpr int kRouteWarps = 8, kRouteTokens = 4;
constexpr size_t kCounterBytes = 4096;   // UP's runs
static_assert(kMaxRuns * 4 <= kCounterBytes, "counters");

struct Space {
  size_t slots, logits, act, act_scale, h, h_scale, partials, total;
};
Space space(int tokens, int hidden, int inter, int experts, int topk) {
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  const size_t rows = static_cast<size_t>(tokens) * topk;
  Space s;
  s.slots = kCounterBytes;
  s.logits = s.slots + 256;
  s.act = s.logits + up(static_cast<size_t>(tokens) * experts * 4);
  s.act_scale = s.act + up(static_cast<size_t>(tokens) * hidden * 2);
  s.h = s.act_scale + up(static_cast<size_t>(tokens) * ((hidden + kRun - 1) / kRun) * 4);
  s.h_scale = s.h + up(rows * 2 * inter * 2);              // two parts at most
  s.partials = s.h_scale + up(rows * ((inter + kRun - 1) / kRun) * 4);
  s.total = s.partials + static_cast<size_t>(kMaxRuns) * 2 * tokens * kCols * 4;
  return s;
}

struct RouteArgs {
  const void* x;
  const void* router;
  int tokens, hidden, experts;
  float* logits;
  __half* act;
  float* act_scale;
  unsigned* counters;
};

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = F16Traits<T>::to_f32(F16Traits<T>::from_bits(lo16((&w.x)[i])));
    v[2 * i + 1] = F16Traits<T>::to_f32(F16Traits<T>::from_bits(hi16((&w.x)[i])));
  }
}

template <typename T, int BITS>
__global__ void __launch_bounds__(kRouteWarps * 32) k_route(const RouteArgs a) {
  __shared__ float sm[kRouteWarps][kRouteTokens];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  decode::pdl_wait();
  decode::pdl_launch_dependents();
  const int tblocks = (a.tokens + kRouteTokens - 1) / kRouteTokens, units = a.experts * tblocks;
  if (static_cast<int>(blockIdx.x) < units) {
    const int e = blockIdx.x / tblocks, t0 = blockIdx.x % tblocks * kRouteTokens;
    const T* r = static_cast<const T*>(a.router) + static_cast<long long>(e) * a.hidden;
    float s[kRouteTokens] = {};
    for (int k = threadIdx.x * 8; k < a.hidden; k += kRouteWarps * 256) {
      float rv[8], xv[8];
      unpack8<T>(__ldg(reinterpret_cast<const uint4*>(r + k)), rv);
      uint4 x[kRouteTokens];
#pragma unroll
      for (int j = 0; j < kRouteTokens; ++j) {
        const int t = t0 + j < a.tokens ? t0 + j : a.tokens - 1;
        x[j] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) + static_cast<long long>(t) * a.hidden + k));
      }
#pragma unroll
      for (int j = 0; j < kRouteTokens; ++j) {
        unpack8<T>(x[j], xv);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[j] = fmaf(xv[i], rv[i], s[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < kRouteTokens; ++j) {
#pragma unroll
      for (int o = 16; o; o >>= 1) s[j] += __shfl_xor_sync(0xFFFFFFFFu, s[j], o);
      if (lane == 0) sm[warp][j] = s[j];
    }
    __syncthreads();
    if (threadIdx.x < kRouteTokens && t0 + static_cast<int>(threadIdx.x) < a.tokens) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kRouteWarps; ++w) v += sm[w][threadIdx.x];
      a.logits[(t0 + threadIdx.x) * a.experts + e] = v;
    }
    return;
  }
  const int runs = (a.hidden + kRun - 1) / kRun, item = (static_cast<int>(blockIdx.x) - units) * kRouteWarps + warp;
  for (int i = (static_cast<int>(blockIdx.x) - units) * kRouteWarps * 32 + threadIdx.x; i < kMaxRuns; i += (gridDim.x - units) * kRouteWarps * 32)
    a.counters[i] = 0u;
  if (item >= a.tokens * runs) return;
  const int t = item / runs, j0 = item % runs * kRun, j = j0 + 4 * lane;
  float v[4] = {};
  if (j < a.hidden) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const T*>(a.x) + static_cast<long long>(t) * a.hidden + j));
    v[0] = F16Traits<T>::to_f32(F16Traits<T>::from_bits(lo16(w.x)));
    v[1] = F16Traits<T>::to_f32(F16Traits<T>::from_bits(hi16(w.x)));
    v[2] = F16Traits<T>::to_f32(F16Traits<T>::from_bits(lo16(w.y)));
    v[3] = F16Traits<T>::to_f32(F16Traits<T>::from_bits(hi16(w.y)));
  }
  store_run<BITS>(v, j0, a.hidden, 1, a.act + static_cast<long long>(t) * a.hidden, a.act_scale + static_cast<long long>(t) * runs + j0 / kRun);
}

template <typename T>
cudaError_t launch_route(const RouteArgs& a, int bits, int grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kRouteWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  switch (bits) {
    case 2: return cudaLaunchKernelEx(&cfg, k_route<T, 2>, a);
    case 3: return cudaLaunchKernelEx(&cfg, k_route<T, 3>, a);
    case 4: return cudaLaunchKernelEx(&cfg, k_route<T, 4>, a);
    default: return cudaLaunchKernelEx(&cfg, k_route<T, 8>, a);
  }
}

}  // namespace
}  // namespace moe

size_t moe_workspace_bytes(int tokens, int hidden, int inter, int experts, int topk) {
  return moe::space(tokens, hidden, inter, experts, topk).total;
}

cudaError_t launch_moe(const MoeProblem& p, cudaStream_t stream) {
  using moe::kRun;
  const moe::Space s = moe::space(p.tokens, p.hidden, p.inter, p.experts, p.topk);
  char* ws = static_cast<char*>(p.workspace);
  unsigned* counters = static_cast<unsigned*>(p.workspace);

  moe::RouteArgs ra;
  ra.x = p.x; ra.router = p.router;
  ra.tokens = p.tokens; ra.hidden = p.hidden; ra.experts = p.experts;
  ra.logits = reinterpret_cast<float*>(ws + s.logits);
  ra.act = reinterpret_cast<__half*>(ws + s.act);
  ra.act_scale = reinterpret_cast<float*>(ws + s.act_scale);
  ra.counters = counters;
  const int tblocks = (p.tokens + moe::kRouteTokens - 1) / moe::kRouteTokens;
  const int runs = (p.hidden + kRun - 1) / kRun;
  const int grid = p.experts * tblocks + (p.tokens * runs + moe::kRouteWarps - 1) / moe::kRouteWarps;
  cudaError_t e = p.dtype == 0 ? moe::launch_route<__half>(ra, p.bits, grid, stream)
                               : moe::launch_route<__nv_bfloat16>(ra, p.bits, grid, stream);
  if (e != cudaSuccess) return e;

  moe::Args up = {};
  up.K = p.hidden; up.N = 2 * p.inter; up.group = p.group_up; up.G = p.hidden / p.group_up; up.zero_offset = p.zero_offset;
  up.qzeros = p.up.qzeros;
  up.scales = static_cast<const __half*>(p.up.scales);
  up.tokens = p.tokens;
  up.parts = 1;
  up.h_parts = p.dtype == 0 ? 2 : 1;
  up.experts = p.experts; up.topk = p.topk; up.renormalize = p.renormalize;
  up.logits = ra.logits;
  up.ids = p.ids; up.weights = p.weights;
  up.act = ra.act; up.act_scale = ra.act_scale; up.act_runs = runs;
  up.jblocks = (p.inter + moe::kCols / 2 - 1) / (moe::kCols / 2);
  up.inter = p.inter;
  up.h = reinterpret_cast<__half*>(ws + s.h);
  up.h_scale = reinterpret_cast<float*>(ws + s.h_scale);
  up.h_runs = (p.inter + kRun - 1) / kRun;
  up.counters = counters;
  up.partials = reinterpret_cast<float*>(ws + s.partials);
  up.status = p.status;
  moe::Args down = up;
  down.parts = up.h_parts;
  down.K = p.inter; down.N = p.hidden; down.group = p.group_down; down.G = p.inter / p.group_down;
  down.qzeros = p.down.qzeros;
  down.scales = static_cast<const __half*>(p.down.scales);
  down.act = up.h; down.act_scale = up.h_scale; down.act_runs = up.h_runs;
  down.jblocks = (p.hidden + moe::kCols - 1) / moe::kCols;
  down.out = p.out;
  down.dtype = p.dtype;
  down.slots = reinterpret_cast<int*>(ws + s.slots);
  int down_grid = 0;
  switch (p.bits) {
    case 2: e = launch_moe_b2(up, p.up.qweight, down, p.down.qweight, p.experts, &down_grid, stream); break;
    case 3: e = launch_moe_b3(up, p.up.qweight, down, p.down.qweight, p.experts, &down_grid, stream); break;
    case 4: e = launch_moe_b4(up, p.up.qweight, down, p.down.qweight, p.experts, &down_grid, stream); break;
    default: e = launch_moe_b8(up, p.up.qweight, down, p.down.qweight, p.experts, &down_grid, stream);
  }
  if (e != cudaSuccess) return e;
  const int chunk = p.bits == 2 ? moe::Chunk<2>::kK : p.bits == 3 ? moe::Chunk<3>::kK : p.bits == 4 ? moe::Chunk<4>::kK : moe::Chunk<8>::kK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(down.jblocks, p.tokens);
  cfg.blockDim = dim3(moe::kCols);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int nk = (p.inter + chunk - 1) / chunk;
  const float* parts = down.partials;
  const int* slots = down.slots;
  if (p.dtype == 0)
    return cudaLaunchKernelEx(&cfg, moe::k_sum_parts<__half>, parts, slots, nk, down.jblocks, down_grid, p.tokens, p.hidden,
                              static_cast<__half*>(p.out));
  return cudaLaunchKernelEx(&cfg, moe::k_sum_parts<__nv_bfloat16>, parts, slots, nk, down.jblocks, down_grid, p.tokens, p.hidden,
                            static_cast<__nv_bfloat16*>(p.out));
}

}  // namespace gptq
