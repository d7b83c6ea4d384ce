// rotary.cu -- rotary embedding of a step's queries and keys, and the append of its keys and values to
// the paged cache.
//
// The angle of pair i at position p is p f_i.  In fp32 its product is off by up to p f_i 2^-24 rad: 0.008 at
// position 131072.  Here f_i / (2 pi) is a whole number of 2^-64 turns, so that p times it, modulo 2^64, is
// the angle modulo a turn, exactly: one integer multiplication.  Its upper 32 bits, as a signed number, are the
// argument of sincospi in units of 2^-31 (rounding it to fp32 moves the angle by pi 2^-25 at most).
//
// Bound: q, k and v are read once and written once.
#include "decode.cuh"
#include "gptq_device.cuh"
#include "gptq_internal.h"
#include "prompt_internal.h"

namespace gptq {
namespace rotary {

constexpr int kThreads = 256;

__device__ __forceinline__ float2 turn(unsigned long long turns, int position, float amplitude) {
  const unsigned long long at = turns * static_cast<unsigned long long>(static_cast<long long>(position));
  float s, c;
  sincospif(static_cast<float>(static_cast<int>(at >> 32)) * 4.656612873077393e-10f, &s, &c);   // 2^-31
  return make_float2(c * amplitude, s * amplitude);
}

// A CTA a token: the turns of its pairs, then its heads.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_rotary(const RotaryProblem p) {
  using Tr = F16Traits<T>;
  __shared__ float2 cs[128];
  __shared__ long long k_row, v_row;
  decode::pdl_launch_dependents();
  decode::pdl_wait();
  const int t = blockIdx.x, half = p.rot_dim / 2, D = p.head_dim;
  for (int i = threadIdx.x; i < half; i += kThreads) cs[i] = turn(p.turns[i], p.positions[t], p.amplitude);
  if (threadIdx.x == 0) {
    k_row = v_row = -1;
    if (p.slots) {
      const long long slot = p.slots[t];
      if (slot >= static_cast<long long>(p.pages) * p.page_size) {
        atomicOr(p.status, kStatusSlotRange);
      } else if (slot >= 0) {
        k_row = slot / p.page_size * p.k_page + slot % p.page_size * p.k_slot;
        v_row = slot / p.page_size * p.v_page + slot % p.page_size * p.v_slot;
      }
    }
  }
  __syncthreads();
  // one item: a pair of a head, or two dimensions that are not turned
  const int pairs = D / 2, rows = p.heads + p.kv_heads * (v_row >= 0 ? 2 : 1);
  for (int item = threadIdx.x; item < rows * pairs; item += kThreads) {
    const int row = item / pairs, i = item % pairs;
    const int kind = row < p.heads ? 0 : (row < p.heads + p.kv_heads ? 1 : 2);
    const int h = row - (kind == 0 ? 0 : kind == 1 ? p.heads : p.heads + p.kv_heads);
    const bool turned = i < half && kind < 2;
    const int a = i >= half || p.interleaved ? 2 * i : i, b = i >= half || p.interleaved ? 2 * i + 1 : i + half;
    const T* from = (kind == 0 ? static_cast<const T*>(p.q) + t * p.q_token
                               : kind == 1 ? static_cast<const T*>(p.k) + t * p.k_token
                                           : static_cast<const T*>(p.v) + t * p.v_token) + static_cast<long long>(h) * D;
    T x = from[a], y = from[b];
    if (turned) {
      const float fx = Tr::to_f32(x), fy = Tr::to_f32(y);
      x = Tr::from_f32(fx * cs[i].x - fy * cs[i].y);
      y = Tr::from_f32(fx * cs[i].y + fy * cs[i].x);
    }
    auto put = [&](T* to) { to[a] = x, to[b] = y; };
    if (kind == 0) put(static_cast<T*>(p.q_out) + t * p.qo_token + static_cast<long long>(h) * D);
    if (kind == 1 && p.k_out) put(static_cast<T*>(p.k_out) + t * p.ko_token + static_cast<long long>(h) * D);
    if (kind == 1 && k_row >= 0) put(static_cast<T*>(p.k_cache) + k_row + h * p.k_head);
    if (kind == 2) put(static_cast<T*>(p.v_cache) + v_row + h * p.v_head);
  }
}

}  // namespace rotary

cudaError_t launch_rotary(const RotaryProblem& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.tokens);
  cfg.blockDim = dim3(rotary::kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.dtype == 0 ? cudaLaunchKernelEx(&cfg, rotary::k_rotary<__half>, p)
                      : cudaLaunchKernelEx(&cfg, rotary::k_rotary<__nv_bfloat16>, p);
}

}  // namespace gptq
