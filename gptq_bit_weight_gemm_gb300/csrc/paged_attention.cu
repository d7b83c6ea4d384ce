// paged_attention.cu -- attention of one new token of each sequence over a paged key-value cache.
#include <math_constants.h>

#include "gptq_device.cuh"
#include "gptq_internal.h"
#include "serving_internal.h"

namespace gptq {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxDim = 256;

// The keys of sequence b that its new token attends to: [lo, n).
__device__ __forceinline__ void live_keys(const AttentionProblem& p, int b, int& lo, int& n) {
  n = p.lens[b];
  const int most = p.table_width * p.page_size;
  if (n < 0 || n > most) {
    atomicOr(p.status, kStatusSeqLen);
    n = n < 0 ? 0 : most;
  }
  lo = p.window > 0 && n > p.window ? n - p.window : 0;
}

template <typename T>
__global__ void k_append(const AttentionProblem p) {
  const int b = blockIdx.x;
  int lo, n;
  live_keys(p, b, lo, n);
  if (n == 0) return;
  const int page = p.table[static_cast<long long>(b) * p.table_width + (n - 1) / p.page_size];
  const int slot = (n - 1) % p.page_size;
  if (page < 0 || page >= p.pages) {
    if (threadIdx.x == 0) atomicOr(p.status, kStatusPageRange);
    return;
  }
  for (int i = threadIdx.x; i < p.kv_heads * p.head_dim; i += blockDim.x) {
    const int h = i / p.head_dim, d = i % p.head_dim;
    static_cast<T*>(p.k_cache)[page * p.k_page + slot * p.k_slot + h * p.k_head + d] =
        static_cast<const T*>(p.k_new)[b * p.kn_batch + i];
    static_cast<T*>(p.v_cache)[page * p.v_page + slot * p.v_slot + h * p.v_head + d] =
        static_cast<const T*>(p.v_new)[b * p.vn_batch + i];
  }
}

// One CTA per (head, sequence); every warp takes every kWarps-th key with its own running maximum,
// sum and accumulator, joined at the end in warp order.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) k_attention(const AttentionProblem p) {
  using Tr = F16Traits<T>;
  const int h = blockIdx.x, b = blockIdx.y, hk = h / (p.heads / p.kv_heads);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ float sm_m[kWarps], sm_l[kWarps], sm_o[kWarps][kMaxDim];
  int lo, n;
  live_keys(p, b, lo, n);
  const T* q = static_cast<const T*>(p.q) + b * p.q_batch + h * p.head_dim;
  float m = -CUDART_INF_F, l = 0.f, o[kMaxDim / 32] = {};
  for (int j = lo + warp; j < n; j += kWarps) {
    const int page = p.table[static_cast<long long>(b) * p.table_width + j / p.page_size];
    if (page < 0 || page >= p.pages) {
      if (lane == 0) atomicOr(p.status, kStatusPageRange);
      continue;
    }
    const T* k = static_cast<const T*>(p.k_cache) + page * p.k_page + (j % p.page_size) * p.k_slot + hk * p.k_head;
    const T* v = static_cast<const T*>(p.v_cache) + page * p.v_page + (j % p.page_size) * p.v_slot + hk * p.v_head;
    float s = 0.f;
    for (int d = lane; d < p.head_dim; d += 32) s = fmaf(Tr::to_f32(q[d]), Tr::to_f32(k[d]), s);
#pragma unroll
    for (int i = 16; i; i >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, i);
    s *= p.scale;
    const float mn = fmaxf(m, s);
    const float base = mn == -CUDART_INF_F ? 0.f : mn;
    const float keep = expf(m - base), e = expf(s - base);
    l = l * keep + e;
#pragma unroll
    for (int i = 0; i < kMaxDim / 32; ++i)
      if (lane + 32 * i < p.head_dim) o[i] = o[i] * keep + e * Tr::to_f32(v[lane + 32 * i]);
    m = mn;
  }
  if (lane == 0) {
    sm_m[warp] = m;
    sm_l[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < kMaxDim / 32; ++i) sm_o[warp][lane + 32 * i] = o[i];
  __syncthreads();
  float M = -CUDART_INF_F;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w]);
  const float base = M == -CUDART_INF_F ? 0.f : M;
  float L = 0.f, f[kWarps];
  for (int w = 0; w < kWarps; ++w) {
    f[w] = expf(sm_m[w] - base);
    L += sm_l[w] * f[w];
  }
  T* out = static_cast<T*>(p.out) + (static_cast<long long>(b) * p.heads + h) * p.head_dim;
  for (int d = threadIdx.x; d < p.head_dim; d += kWarps * 32) {
    float v = 0.f;
    for (int w = 0; w < kWarps; ++w) v += sm_o[w][d] * f[w];
    out[d] = Tr::from_f32(L > 0.f || isnan(L) ? v / L : 0.f);
  }
  if (p.lse && threadIdx.x == 0) p.lse[static_cast<long long>(b) * p.heads + h] = M + logf(L);
}

}  // namespace

size_t attention_workspace_bytes(int, int, int) { return 256; }

cudaError_t launch_paged_attention(const AttentionProblem& p, cudaStream_t stream) {
  const dim3 grid(p.heads, p.batch);
  if (p.dtype == 0) {
    if (p.k_new) k_append<__half><<<p.batch, 128, 0, stream>>>(p);
    k_attention<__half><<<grid, kWarps * 32, 0, stream>>>(p);
  } else {
    if (p.k_new) k_append<__nv_bfloat16><<<p.batch, 128, 0, stream>>>(p);
    k_attention<__nv_bfloat16><<<grid, kWarps * 32, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace gptq
