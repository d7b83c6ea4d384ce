// rms_norm.cu -- root-mean-square norm of rows with the residual's addition:
//   s = residual + x,  residual_out = s,  out = s * weight / sqrt(mean(s^2) + eps).
//
// Bound: x and the residual are read once, the residual and the result written once, a few flops an
// element: HBM for many rows, the chain launch - load - sum - store for few.
//
// A row stays in registers between the sum and the result: as many threads as it has runs of 8 elements, up
// to 1024, and up to 4 runs a thread (longer rows are read a second time).  Runs begin at the
// 8-element boundaries of memory, not of the row, so that rows of any length are read 16 bytes at a
// time as long as all tensors' rows begin at the same place within such a run (of 16-byte pieces, for fp32); the
// ends of a row, and rows of tensors that do not, go element by element (4096 rows of 4096, bf16 on an fp32 residual: 40 us in runs, 121 by element).
#include "decode.cuh"
#include "gptq_device.cuh"
#include "gptq_internal.h"
#include "prompt_internal.h"

namespace gptq {
namespace norm {

constexpr int kF16 = 0, kBF16 = 1, kF32 = 2, kNone = 3;

__device__ __forceinline__ float load1(const void* p, int dtype, long long i) {
  if (dtype == kF16) return __half2float(static_cast<const __half*>(p)[i]);
  if (dtype == kBF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void store1(void* p, int dtype, long long i, float v) {
  if (dtype == kF16) static_cast<__half*>(p)[i] = __float2half_rn(v);
  else if (dtype == kBF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<float*>(p)[i] = v;
}
// 8 elements from a place that is a multiple of 8 of them (fp32: of 4)
__device__ __forceinline__ void load8(const void* p, int dtype, long long i, float (&v)[8]) {
  if (dtype == kF32) {
    const float4* from = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = from[0], b = from[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    return;
  }
  const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t x = (&w.x)[j];
    v[2 * j] = dtype == kF16 ? __half2float(__ushort_as_half(lo16(x))) : __uint_as_float(x << 16);
    v[2 * j + 1] = dtype == kF16 ? __half2float(__ushort_as_half(hi16(x))) : __uint_as_float(x & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void store8(void* p, int dtype, long long i, const float (&v)[8]) {
  if (dtype == kF32) {
    float4* to = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    to[0] = make_float4(v[0], v[1], v[2], v[3]);
    to[1] = make_float4(v[4], v[5], v[6], v[7]);
    return;
  }
  uint4 w;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    (&w.x)[j] = dtype == kF16 ? pack2(v[2 * j], v[2 * j + 1], __half()) : pack2(v[2 * j], v[2 * j + 1], __nv_bfloat16());
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = w;
}

struct Args {
  NormProblem p;
  int base;            // the first row's place within a run of 8 elements
  int step;            // by how much a row's place is behind the row before's
  int even;            // all tensors' rows begin at the same place of a run: 16 bytes at a time
  int weight_even;     // the weight's runs, from its first element, begin on 16 bytes
};

// X, R: types of x and the residual.  TPR threads a row; NV runs a thread (0: the row is read again).
template <int X, int R, int TPR, int NV>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) k_norm(const __grid_constant__ Args a) {
  constexpr int kRows = TPR < 128 ? 128 / TPR : 1, kWarps = TPR / 32;
  const NormProblem& p = a.p;
  __shared__ float part[TPR < 128 ? 1 : kWarps];
  decode::pdl_launch_dependents();
  decode::pdl_wait();
  const long long row = static_cast<long long>(blockIdx.x) * kRows + threadIdx.x / TPR;
  if (row >= p.rows) return;               // (whole warps: only rows of one warp share a CTA)
  const int t = threadIdx.x % TPR;
  const int place = a.even ? static_cast<int>((a.base + row * a.step) & 7) : 0;   // of the row's first element
  const int runs = (place + p.hidden + 7) / 8;
  const long long x0 = row * p.x_stride, r0 = row * p.residual_stride, ro0 = row * p.residual_out_stride, o0 = row * p.out_stride;
  auto inside = [&](int run) { return a.even && run * 8 >= place && run * 8 + 8 <= place + p.hidden; };
  auto value = [&](int run, float (&s)[8]) {
    const int i = run * 8 - place;
    if (inside(run)) {
      load8(p.x, X, x0 + i, s);
      if (R != kNone) {
        float r[8];
        load8(p.residual, R, r0 + i, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] += r[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s[j] = 0.f;
        if (i + j >= 0 && i + j < p.hidden) {
          s[j] = load1(p.x, X, x0 + i + j);
          if (R != kNone) s[j] += load1(p.residual, R, r0 + i + j);
        }
      }
    }
  };
  auto square = [](const float (&s)[8]) {
    return ((s[0] * s[0] + s[1] * s[1]) + (s[2] * s[2] + s[3] * s[3])) + ((s[4] * s[4] + s[5] * s[5]) + (s[6] * s[6] + s[7] * s[7]));
  };
  float s[NV > 0 ? NV : 1][8], sum = 0.f;
  if constexpr (NV > 0) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (t + v * TPR < runs) value(t + v * TPR, s[v]);
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (t + v * TPR < runs) sum += square(s[v]);
  } else {
    for (int run = t; run < runs; run += TPR) {
      value(run, s[0]);
      sum += square(s[0]);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if constexpr (kWarps > 1) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
    __syncthreads();
    // every warp joins the parts in the same order
    const int lane = threadIdx.x & 31;
    sum = lane < kWarps ? part[lane] : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  }
  const float inv = 1.f / sqrtf(sum / static_cast<float>(p.hidden) + p.eps);
  auto finish = [&](int run, float (&v)[8]) {
    const int i = run * 8 - place;
    float w[8];
    const bool in = inside(run);
    if (in && R != kNone) store8(p.residual_out, R, ro0 + i, v);
    if (p.weight == nullptr) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = 1.f;
    } else if (in && place == 0 && a.weight_even) {
      load8(p.weight, p.weight_dtype, i, w);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = i + j >= 0 && i + j < p.hidden ? load1(p.weight, p.weight_dtype, i + j) : 0.f;
    }
    if (in) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = v[j] * inv * w[j];
      store8(p.out, p.out_dtype, o0 + i, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (i + j < 0 || i + j >= p.hidden) continue;
        if (R != kNone) store1(p.residual_out, R, ro0 + i + j, v[j]);
        store1(p.out, p.out_dtype, o0 + i + j, v[j] * inv * w[j]);
      }
    }
  };
  // what is written may be where it was read from: the row has been read whole, or its places by the same thread
  if constexpr (NV > 0) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (t + v * TPR < runs) finish(t + v * TPR, s[v]);
  } else {
    for (int run = t; run < runs; run += TPR) {
      value(run, s[0]);
      finish(run, s[0]);
    }
  }
}

template <int X, int R>
cudaError_t launch(const Args& a, cudaStream_t stream) {
  const int runs = (a.p.hidden + 7) / 8 + (a.even && (a.base || a.step) ? 1 : 0);   // (a shifted row touches one more)
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto go = [&](auto kern, int tpr) {
    const int rows = tpr < 128 ? 128 / tpr : 1;
    cfg.gridDim = dim3((a.p.rows + rows - 1) / rows);
    cfg.blockDim = dim3(tpr < 128 ? 128 : tpr);
    return cudaLaunchKernelEx(&cfg, kern, a);
  };
  if (runs <= 32) return go(k_norm<X, R, 32, 1>, 32);
  if (runs <= 64) return go(k_norm<X, R, 32, 2>, 32);
  if (runs <= 128) return go(k_norm<X, R, 128, 1>, 128);
  if (runs <= 256) return go(k_norm<X, R, 256, 1>, 256);
  if (runs <= 512) return go(k_norm<X, R, 256, 2>, 256);
  if (runs <= 1024) return go(k_norm<X, R, 512, 2>, 512);
  if (runs <= 2048) return go(k_norm<X, R, 512, 4>, 512);
  if (runs <= 4096) return go(k_norm<X, R, 1024, 4>, 1024);
  return go(k_norm<X, R, 1024, 0>, 1024);
}

template <int X>
cudaError_t launch_x(const Args& a, cudaStream_t stream) {
  if (!a.p.residual) return launch<X, kNone>(a, stream);
  if (a.p.residual_dtype == kF16) return launch<X, kF16>(a, stream);
  if (a.p.residual_dtype == kBF16) return launch<X, kBF16>(a, stream);
  return launch<X, kF32>(a, stream);
}

}  // namespace norm

cudaError_t launch_rms_norm(const NormProblem& p, cudaStream_t stream) {
  norm::Args a;
  a.p = p;
  // A tensor's place: which element of a run of 8 its first one is.  The runs are those of a 16-bit tensor, where there
  // is one: 16 bytes of it.  Of fp32 a run is two times 16 bytes, so that a place 4 elements off does as well.
  auto place = [](const void* t, int dtype) {
    const uintptr_t size = dtype == norm::kF32 ? 4 : 2, at = reinterpret_cast<uintptr_t>(t);
    return static_cast<int>(at / size % 8);
  };
  const struct { const void* t; int dtype; long long stride; } all[4] = {
      {p.x, p.dtype, p.x_stride}, {p.out, p.out_dtype, p.out_stride},
      {p.residual, p.residual_dtype, p.residual_stride}, {p.residual_out, p.residual_dtype, p.residual_out_stride}};
  const int tensors = p.residual ? 4 : 2;
  int first = 0;
  while (first < tensors && all[first].dtype == norm::kF32) ++first;
  if (first == tensors) first = 0;
  a.base = place(all[first].t, all[first].dtype);
  a.step = static_cast<int>(all[first].stride % 8);
  a.even = 1;
  for (int i = 0; i < tensors; ++i) {
    const int piece = all[i].dtype == norm::kF32 ? 4 : 8;
    if ((place(all[i].t, all[i].dtype) - a.base) % piece || (all[i].stride - a.step) % piece) a.even = 0;
  }
  a.weight_even = p.weight && place(p.weight, p.weight_dtype) % (p.weight_dtype == norm::kF32 ? 4 : 8) == 0;
  if (p.dtype == norm::kF16) return norm::launch_x<norm::kF16>(a, stream);
  if (p.dtype == norm::kBF16) return norm::launch_x<norm::kBF16>(a, stream);
  return norm::launch_x<norm::kF32>(a, stream);
}

}  // namespace gptq
