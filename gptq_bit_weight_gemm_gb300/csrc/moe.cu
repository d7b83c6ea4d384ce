// moe.cu -- the mixture-of-experts layer for a few tokens on packed expert weights.
#include <math_constants.h>

#include "gptq_device.cuh"
#include "gptq_internal.h"
#include "serving_internal.h"

namespace gptq {
namespace {

struct Layout {
  size_t ids, weights, logits, h, total;
};
Layout layout(int tokens, int inter, int experts, int topk) {
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  Layout l;
  l.ids = 4096;
  l.weights = l.ids + up(static_cast<size_t>(tokens) * topk * 4);
  l.logits = l.weights + up(static_cast<size_t>(tokens) * topk * 4);
  l.h = l.logits + up(static_cast<size_t>(tokens) * experts * 4);
  l.total = l.h + static_cast<size_t>(tokens) * topk * inter * 4;
  return l;
}

template <typename T>
__device__ __forceinline__ float act(const void* p, long long i) {
  return F16Traits<T>::to_f32(static_cast<const T*>(p)[i]);
}

template <typename T>
__global__ void __launch_bounds__(1024) k_route(const MoeProblem p, float* logits, int* ids, float* weights) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  for (int i = warp; i < p.tokens * p.experts; i += nw) {
    const int t = i / p.experts, e = i % p.experts;
    float s = 0.f;
    for (int k = lane; k < p.hidden; k += 32)
      s = fmaf(act<T>(p.x, static_cast<long long>(t) * p.hidden + k), act<T>(p.router, static_cast<long long>(e) * p.hidden + k), s);
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (lane == 0) logits[i] = s;
  }
  __syncthreads();
  for (int t = warp; t < p.tokens; t += nw) {
    const float* row = logits + t * p.experts;
    float m = -CUDART_INF_F, sum = 0.f, kept = 0.f;
    for (int e = lane; e < p.experts; e += 32) m = fmaxf(m, row[e]);
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    for (int e = lane; e < p.experts; e += 32) sum += expf(row[e] - m);
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    float last_v = CUDART_INF_F;
    int last_e = -1;
    for (int j = 0; j < p.topk; ++j) {            // the best expert after the last one in (value, index) order
      float bv = -CUDART_INF_F;
      int be = 0x7FFFFFFF;
      for (int e = lane; e < p.experts; e += 32) {
        const float v = isnan(row[e]) ? -CUDART_INF_F : row[e];
        const bool after = v < last_v || (v == last_v && e > last_e);
        if (after && (be == 0x7FFFFFFF || v > bv)) { bv = v; be = e; }
      }
      for (int o = 16; o; o >>= 1) {
        const float ov = __shfl_xor_sync(0xFFFFFFFFu, bv, o);
        const int oe = __shfl_xor_sync(0xFFFFFFFFu, be, o);
        if (oe != 0x7FFFFFFF && (be == 0x7FFFFFFF || ov > bv || (ov == bv && oe < be))) { bv = ov; be = oe; }
      }
      const float pr = expf(bv - m) / sum;
      kept += pr;
      if (lane == 0) {
        ids[t * p.topk + j] = be;
        weights[t * p.topk + j] = pr;
      }
      last_v = bv;
      last_e = be;
    }
    __syncwarp();
    if (p.renormalize)
      for (int j = lane; j < p.topk; j += 32) weights[t * p.topk + j] /= kept;
    __syncwarp();
    for (int j = lane; j < p.topk; j += 32) {
      if (p.ids) p.ids[t * p.topk + j] = ids[t * p.topk + j];
      if (p.weights) p.weights[t * p.topk + j] = weights[t * p.topk + j];
    }
  }
}

// fp32 weight (k, n) of expert e
__device__ __forceinline__ float weight_at(const PackedExperts& w, int e, int k, int n, int K, int N, int bits, int group,
                                           int zero_offset) {
  const int G = K / group;
  auto field = [&](uint32_t lo, uint32_t hi, int sh) { return __funnelshift_r(lo, hi, sh) & ((1u << bits) - 1u); };
  const int rows = K / 32 * bits, bit = k * bits, words = N / 32 * bits, zbit = n * bits;
  const int32_t* qw = w.qweight + (static_cast<long long>(e) * rows + (bit >> 5)) * N + n;
  const uint32_t lo = qw[0], hi = (bit & 31) + bits > 32 ? qw[N] : 0;
  const long long gz = static_cast<long long>(e) * G + k / group;
  const int32_t* qz = w.qzeros + gz * words + (zbit >> 5);
  const uint32_t zlo = qz[0], zhi = (zbit & 31) + bits > 32 ? qz[1] : 0;
  const int q = static_cast<int>(field(lo, hi, bit & 31)), z = static_cast<int>(field(zlo, zhi, zbit & 31)) + zero_offset;
  return static_cast<float>(q - z) * __half2float(static_cast<const __half*>(w.scales)[gz * N + n]);
}

template <typename T>
__global__ void k_up(const MoeProblem p, const int* ids, float* h) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x, pair = blockIdx.y, t = pair / p.topk, e = ids[pair];
  if (i >= p.inter) return;
  float g = 0.f, u = 0.f;
  for (int k = 0; k < p.hidden; ++k) {
    const float x = act<T>(p.x, static_cast<long long>(t) * p.hidden + k);
    g = fmaf(x, weight_at(p.up, e, k, i, p.hidden, 2 * p.inter, p.bits, p.group_up, p.zero_offset), g);
    u = fmaf(x, weight_at(p.up, e, k, p.inter + i, p.hidden, 2 * p.inter, p.bits, p.group_up, p.zero_offset), u);
  }
  h[static_cast<long long>(pair) * p.inter + i] = g / (1.f + expf(-g)) * u;
}

template <typename T>
__global__ void k_down(const MoeProblem p, const int* ids, const float* weights, const float* h) {
  const int n = blockIdx.x * blockDim.x + threadIdx.x, t = blockIdx.y;
  if (n >= p.hidden) return;
  float out = 0.f;
  for (int j = 0; j < p.topk; ++j) {
    const int pair = t * p.topk + j;
    float y = 0.f;
    for (int k = 0; k < p.inter; ++k)
      y = fmaf(h[static_cast<long long>(pair) * p.inter + k],
               weight_at(p.down, ids[pair], k, n, p.inter, p.hidden, p.bits, p.group_down, p.zero_offset), y);
    out = fmaf(weights[pair], y, out);
  }
  static_cast<T*>(p.out)[static_cast<long long>(t) * p.hidden + n] = F16Traits<T>::from_f32(out);
}

template <typename T>
void launch(const MoeProblem& p, const Layout& l, cudaStream_t s) {
  char* ws = static_cast<char*>(p.workspace);
  int* ids = reinterpret_cast<int*>(ws + l.ids);
  float* weights = reinterpret_cast<float*>(ws + l.weights);
  float* h = reinterpret_cast<float*>(ws + l.h);
  k_route<T><<<1, 1024, 0, s>>>(p, reinterpret_cast<float*>(ws + l.logits), ids, weights);
  k_up<T><<<dim3((p.inter + 127) / 128, p.tokens * p.topk), 128, 0, s>>>(p, ids, h);
  k_down<T><<<dim3((p.hidden + 127) / 128, p.tokens), 128, 0, s>>>(p, ids, weights, h);
}

}  // namespace

size_t moe_workspace_bytes(int tokens, int, int inter, int experts, int topk) {
  return layout(tokens, inter, experts, topk).total;
}

cudaError_t launch_moe(const MoeProblem& p, cudaStream_t stream) {
  const Layout l = layout(p.tokens, p.inter, p.experts, p.topk);
  if (p.dtype == 0) launch<__half>(p, l, stream);
  else launch<__nv_bfloat16>(p, l, stream);
  return cudaGetLastError();
}

}  // namespace gptq
