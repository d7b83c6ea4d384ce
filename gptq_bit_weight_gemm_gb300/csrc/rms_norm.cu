// rms_norm.cu -- root-mean-square norm of rows with the residual's addition:
//   s = residual + x,  residual_out = s,  out = s * weight / sqrt(mean(s^2) + eps).
//
// Bound: x and the residual are read once, the residual and the result written once, a few flops an
// element: HBM for many rows, the chain launch - load - sum - store for few.
#include "decode.cuh"
#include "gptq_device.cuh"
#include "gptq_internal.h"
#include "prompt_internal.h"

namespace gptq {
namespace norm {

constexpr int kThreads = 256;

__device__ __forceinline__ float load(const void* p, int dtype, long long i) {
  if (dtype == 0) return __half2float(static_cast<const __half*>(p)[i]);
  if (dtype == 1) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void store(void* p, int dtype, long long i, float v) {
  if (dtype == 0) static_cast<__half*>(p)[i] = __float2half_rn(v);
  else if (dtype == 1) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<float*>(p)[i] = v;
}

__global__ void __launch_bounds__(kThreads) k_norm(const NormProblem p) {
  __shared__ float part[kThreads / 32];
  decode::pdl_launch_dependents();
  decode::pdl_wait();
  const long long row = blockIdx.x;
  auto value = [&](int i) {
    float s = load(p.x, p.dtype, row * p.x_stride + i);
    if (p.residual) s += load(p.residual, p.residual_dtype, row * p.residual_stride + i);
    return s;
  };
  float sum = 0.f;
  for (int i = threadIdx.x; i < p.hidden; i += kThreads) {
    const float s = value(i);
    sum += s * s;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
  __syncthreads();
  sum = 0.f;
  for (int w = 0; w < kThreads / 32; ++w) sum += part[w];
  const float inv = 1.f / sqrtf(sum / static_cast<float>(p.hidden) + p.eps);
  // what is written may be where it was read from: each place by the thread that reads it
  for (int i = threadIdx.x; i < p.hidden; i += kThreads) {
    const float s = value(i);
    const float w = p.weight ? load(p.weight, p.weight_dtype, i) : 1.f;
    if (p.residual) store(p.residual_out, p.residual_dtype, row * p.residual_out_stride + i, s);
    store(p.out, p.out_dtype, row * p.out_stride + i, s * inv * w);
  }
}

}  // namespace norm

cudaError_t launch_rms_norm(const NormProblem& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.rows);
  cfg.blockDim = dim3(norm::kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm::k_norm, p);
}

}  // namespace gptq
