// sample.cu -- one token for each row of logits, from a given uniform number.
#include <math_constants.h>

#include "gptq_device.cuh"
#include "gptq_internal.h"
#include "serving_internal.h"

namespace gptq {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
typedef unsigned long long u64;

// Order-preserving bits of a logit: NaN lowest, -0 as 0.
__device__ __forceinline__ uint32_t key_of(float l) {
  if (isnan(l)) return 0u;
  const uint32_t b = __float_as_uint(l + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

template <int DT>
__device__ __forceinline__ float load_logit(const void* p, long long i) {
  if constexpr (DT == 0) return __half2float(static_cast<const __half*>(p)[i]);
  if constexpr (DT == 1) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return static_cast<const float*>(p)[i];
}

__device__ __forceinline__ float weight_of(float l, float top, float temp) {
  if (top == CUDART_INF_F) return l == CUDART_INF_F ? 1.f : 0.f;
  return expf((l - top) / temp);
}
__device__ __forceinline__ u64 mass_of(float w) { return static_cast<u64>(__float2ull_rn(w * 4294967296.f)); }

__device__ u64 block_sum(u64 v, u64* sm) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
  for (int w = 0; w < kWarps; ++w) v += sm[w];
  return v;
}

// One CTA per row.  The kept set is "keys above thr, and the first `ties` tokens of key thr", found
// by bisection over the 32 key bits, with exact integer counts and masses.
template <int DT>
__global__ void __launch_bounds__(kThreads) k_sample(const SampleProblem p) {
  __shared__ u64 sm[kWarps];
  __shared__ u64 seg_mass[kWarps];
  __shared__ int seg_ties[kWarps];
  const int b = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = b * p.row_stride;
  auto key_at = [&](int i) { return key_of(load_logit<DT>(p.logits, row + i)); };
  uint32_t best = 0;
  for (int i = threadIdx.x; i < p.vocab; i += kThreads) best = max(best, key_at(i));
  for (int o = 16; o; o >>= 1) best = max(best, __shfl_xor_sync(0xFFFFFFFFu, best, o));
  if (lane == 0) sm[warp] = best;
  __syncthreads();
  for (int w = 0; w < kWarps; ++w) best = max(best, static_cast<uint32_t>(sm[w]));
  const float top = best ? logit_of(best) : -CUDART_INF_F;
  if (top == -CUDART_INF_F) {
    if (threadIdx.x == 0) {
      p.token[b] = -1;
      if (p.logprob) p.logprob[b] = CUDART_NAN_F;
      atomicOr(p.status, kStatusNoToken);
    }
    return;
  }
  float temp = p.temperature ? p.temperature[b] : 1.f;
  const float top_p = p.top_p ? p.top_p[b] : 1.f, min_p = p.min_p ? p.min_p[b] : 0.f;
  int k = p.top_k && p.top_k[b] > 0 ? p.top_k[b] : p.vocab;
  if (!(temp > 0.f)) { temp = 1.f; k = 1; }
  if (!(top_p > 0.f) || !(min_p <= 1.f)) k = 1;
  auto mass_at = [&](uint32_t key) { return key ? mass_of(weight_of(logit_of(key), top, temp)) : 0ull; };

  // (thr, ties) after top-k
  uint32_t thr = 0;
  int ties = p.vocab;
  if (k < p.vocab) {
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t cand = thr | (1u << bit);
      u64 c = 0;
      for (int i = threadIdx.x; i < p.vocab; i += kThreads) c += key_at(i) >= cand;
      if (block_sum(c, sm) >= static_cast<u64>(k)) thr = cand;
    }
    u64 c = 0;
    for (int i = threadIdx.x; i < p.vocab; i += kThreads) c += key_at(i) > thr;
    ties = k - static_cast<int>(block_sum(c, sm));
  }
  if (top_p < 1.f) {
    // mass of the keys above v, and the top-k total
    auto above = [&](uint32_t v) {
      u64 m = 0;
      for (int i = threadIdx.x; i < p.vocab; i += kThreads) {
        const uint32_t key = key_at(i);
        if (key > v) m += mass_at(key);
      }
      return block_sum(m, sm);
    };
    u64 n_thr = 0;
    for (int i = threadIdx.x; i < p.vocab; i += kThreads) n_thr += key_at(i) == thr;
    n_thr = block_sum(n_thr, sm);
    const u64 at_thr = n_thr < static_cast<u64>(ties) ? n_thr : ties;
    const double limit = static_cast<double>(top_p) * static_cast<double>(above(thr) + at_thr * mass_at(thr));
    // the smallest v >= thr with mass above v < limit
    uint32_t lo = thr, hi = best;
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo) / 2;
      if (static_cast<double>(above(mid)) < limit) hi = mid;
      else lo = mid + 1;
    }
    const u64 a = above(lo), m = mass_at(lo);
    int r = lo == thr ? ties : p.vocab;
    if (m > 0) {
      // ties i = 0, 1, ... stay while a + i m < limit
      u64 q = static_cast<u64>(ceil((limit - static_cast<double>(a)) / static_cast<double>(m)));
      if (q < 1) q = 1;
      if (q < static_cast<u64>(r)) r = static_cast<int>(q);
    }
    thr = lo;
    ties = r;
  }
  auto kept_mass = [&](uint32_t key) {
    if (key == 0) return 0ull;
    const float w = weight_of(logit_of(key), top, temp);
    return w >= min_p || key == best ? mass_of(w) : 0ull;
  };
  // each warp sums one run of the row; ties count from the row's start
  const int run = (p.vocab + kWarps - 1) / kWarps, i0 = min(warp * run, p.vocab), i1 = min(i0 + run, p.vocab);
  int nt = 0;
  for (int i = i0 + lane; i < i1; i += 32) nt += key_at(i) == thr;
  nt = __reduce_add_sync(0xFFFFFFFFu, nt);
  if (lane == 0) seg_ties[warp] = nt;
  __syncthreads();
  int tie0 = 0;
  for (int w = 0; w < warp; ++w) tie0 += seg_ties[w];
  auto each = [&](auto f) {          // f(index, kept mass) of the run, 32 at a time, in index order
    int seen = tie0;
    for (int i = i0; i < i1; i += 32) {
      const uint32_t key = i + lane < i1 ? key_at(i + lane) : 0u;
      const bool tie = i + lane < i1 && key == thr;
      const unsigned mask = __ballot_sync(0xFFFFFFFFu, tie);
      const bool in = key > thr || (tie && seen + __popc(mask & ((1u << lane) - 1)) < ties);
      if (!f(i + lane, in ? kept_mass(key) : 0ull, key)) break;
      seen += __popc(mask);
    }
  };
  u64 mine = 0;
  each([&](int, u64 m, uint32_t) { mine += m; return true; });
  for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, o);
  if (lane == 0) seg_mass[warp] = mine;
  __syncthreads();
  u64 total = 0, before = 0;
  int last = -1;                     // the last run with mass
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += seg_mass[w];
    total += seg_mass[w];
    if (seg_mass[w]) last = w;
  }
  float u = p.uniform[b];
  u = u > 0.f ? u : 0.f;
  const double target = static_cast<double>(u) * static_cast<double>(total);
  const bool over = !(target < static_cast<double>(total));       // u >= 1: the last kept token
  const bool here = over ? warp == last
                         : static_cast<double>(before) <= target && target < static_cast<double>(before + mine);
  if (!here) return;
  u64 cum = before;
  int found = -1;
  uint32_t found_key = 0;
  each([&](int i, u64 m, uint32_t key) {
    u64 c = m;
    for (int o = 1; o < 32; o <<= 1) {
      const u64 v = __shfl_up_sync(0xFFFFFFFFu, c, o);
      if (lane >= o) c += v;
    }
    c += cum;
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, m > 0 && (over || static_cast<double>(c) > target));
    if (hit) {
      const int src = over ? 31 - __clz(hit) : __ffs(hit) - 1;
      found = __shfl_sync(0xFFFFFFFFu, i, src);
      found_key = __shfl_sync(0xFFFFFFFFu, key, src);
    }
    cum = __shfl_sync(0xFFFFFFFFu, c, 31);
    return over || !hit;
  });
  if (lane == 0) {
    p.token[b] = found;
    if (p.logprob) {
      const float x = top == CUDART_INF_F ? 0.f : (logit_of(found_key) - top) / temp;
      p.logprob[b] = static_cast<float>(static_cast<double>(x) - log(static_cast<double>(total) / 4294967296.0));
    }
  }
}

}  // namespace

cudaError_t launch_sample(const SampleProblem& p, cudaStream_t stream) {
  if (p.dtype == 0) k_sample<0><<<p.batch, kThreads, 0, stream>>>(p);
  else if (p.dtype == 1) k_sample<1><<<p.batch, kThreads, 0, stream>>>(p);
  else k_sample<2><<<p.batch, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace gptq
