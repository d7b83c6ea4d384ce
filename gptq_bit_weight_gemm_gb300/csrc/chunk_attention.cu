// chunk_attention.cu -- causal attention of each sequence's new tokens over its paged keys and values:
//   out = sum_j p_j v_j,  p = softmax_j(scale q . k_j),  over the keys j in [max(0, t - window + 1), t] of the
// row at position t.
//
// With the maximum m, the sum l and the accumulator o of the keys so far, a new score s moves them to
//   m' = max(m, s),  l' = l e^(m - m') + e^(s - m'),  o' = o e^(m - m') + e^(s - m') v.
//
// A warp takes a row and head, a lane DP / 32 dimensions.
#include <math_constants.h>

#include "decode.cuh"
#include "gptq_device.cuh"
#include "gptq_internal.h"
#include "prompt_internal.h"

namespace gptq {
namespace chunk {

constexpr int kWarps = 8, kThreads = kWarps * 32;

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) k_chunk(const ChunkProblem p) {
  using Tr = F16Traits<T>;
  constexpr int kDims = DP / 32;
  decode::pdl_launch_dependents();
  decode::pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long item = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int row = static_cast<int>(item / p.heads), h = static_cast<int>(item % p.heads);
  const int kvh = h / (p.heads / p.kv_heads);
  if (blockIdx.x == 0)
    for (int s = threadIdx.x; s < p.batch; s += kThreads)
      if (p.cu[s] < 0 || p.cu[s + 1] < p.cu[s] || p.cu[s + 1] > p.tokens) atomicOr(p.status, kStatusTokenRows);
  if (row >= p.tokens) return;
  // the row's sequence
  int b = -1, first = 0, end = 0;
  for (int s = 0; s < p.batch; ++s) {
    const int c0 = p.cu[s], c1 = p.cu[s + 1];
    first = min(max(c0, 0), p.tokens);
    end = max(first, min(c1, p.tokens));
    if (row >= first && row < end) {
      b = s;
      break;
    }
  }
  if (b < 0) return;
  const int most = p.table_width * p.page_size, raw = p.lens[b], n = min(max(raw, 0), most);
  if (raw != n && lane == 0) atomicOr(p.status, kStatusSeqLen);
  const int at = n - (end - first) + row - first;
  const int lo = p.window > 0 ? max(0, at - p.window + 1) : 0;
  float q[kDims], o[kDims] = {}, m = -CUDART_INF_F, l = 0.f;
  const T* qp = static_cast<const T*>(p.q) + row * p.q_token + static_cast<long long>(h) * p.head_dim;
#pragma unroll
  for (int i = 0; i < kDims; ++i) {
    const int d = lane + 32 * i;
    q[i] = d < p.head_dim ? Tr::to_f32(qp[d]) : 0.f;
  }
  for (int j = lo; j <= at; ++j) {
    const int page = p.table[static_cast<long long>(b) * p.table_width + j / p.page_size], slot = j % p.page_size;
    if (page < 0 || page >= p.pages) {
      if (lane == 0) atomicOr(p.status, kStatusPageRange);
      continue;
    }
    const T* k = static_cast<const T*>(p.k_cache) + page * p.k_page + slot * p.k_slot + kvh * p.k_head;
    const T* v = static_cast<const T*>(p.v_cache) + page * p.v_page + slot * p.v_slot + kvh * p.v_head;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kDims; ++i) {
      const int d = lane + 32 * i;
      if (d < p.head_dim) s += q[i] * Tr::to_f32(k[d]);
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, x);
    s *= p.scale;
    const float mn = fmaxf(m, s), base = mn == -CUDART_INF_F ? 0.f : mn;
    const float keep = expf(m - base), e = expf(s - base);
    m = mn;
    l = l * keep + e;
#pragma unroll
    for (int i = 0; i < kDims; ++i) {
      const int d = lane + 32 * i;
      if (d < p.head_dim) o[i] = o[i] * keep + e * Tr::to_f32(v[d]);
    }
  }
  const long long to = static_cast<long long>(row) * p.heads + h;
  const float inv = l > 0.f || isnan(l) ? 1.f / l : 0.f;
#pragma unroll
  for (int i = 0; i < kDims; ++i) {
    const int d = lane + 32 * i;
    if (d < p.head_dim) static_cast<T*>(p.out)[to * p.head_dim + d] = Tr::from_f32(o[i] * inv);
  }
  if (p.lse && lane == 0) p.lse[to] = m + logf(l);
}

template <typename T>
cudaError_t launch(const ChunkProblem& p, cudaStream_t stream) {
  const long long items = static_cast<long long>(p.tokens) * p.heads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((items + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (p.head_dim <= 64) return cudaLaunchKernelEx(&cfg, k_chunk<T, 64>, p);
  if (p.head_dim <= 128) return cudaLaunchKernelEx(&cfg, k_chunk<T, 128>, p);
  return cudaLaunchKernelEx(&cfg, k_chunk<T, 256>, p);
}

}  // namespace chunk

size_t chunk_attention_workspace_bytes(int, int, int) { return 4096; }

cudaError_t launch_chunk_attention(const ChunkProblem& p, cudaStream_t stream) {
  return p.dtype == 0 ? chunk::launch<__half>(p, stream) : chunk::launch<__nv_bfloat16>(p, stream);
}

}  // namespace gptq
