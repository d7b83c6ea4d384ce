// sample.cu -- one token for each row of logits, from a given uniform number (gptq_sample).
//
// With x = (l - max l) / T, w = e^x and the tokens ordered by l (equal ones by index), every setting
// keeps a prefix of that order: the first top_k, then those before which less than top_p of the mass
// lies, then those with w >= min_p.  So the kept set is "logits above a threshold, and the first few of
// those equal to it", and the token is found by cumulating the kept masses in index order.  Nothing is
// sorted but the few tokens around a threshold.  Masses are integers of 2^-39 of the best token's, whose
// sums do not depend on their order: atomics and splits do not change a result.  Rounding them loses at
// most 2^-40 a token, 2^-18 of the total at 2^22 tokens; units of 2^-31 lost a tail of 131072 tokens 22.3
// below the best altogether, 2.7e-5 of the total.
//
// Bound: the logits are read once from HBM (a cluster of CTAs holds a row in its shared memory); what
// costs time is the passes over the row on chip and, more, the cluster's barriers between them, at which the
// others wait while CTA 0 joins the histograms, finds the bin, sorts its tokens and cuts them.
//   1. load, largest and smallest logit;
//   2. a histogram of max - l: counts, and masses where the mass decides (no top_k, or a long one);
//   3. with a short top_k, everything down to the bin that holds the k-th goes to one CTA, which sorts
//      and finishes; otherwise the tokens of the bin that the threshold falls into are sorted there;
//   4. the kept masses summed and searched in index order.
// Rows whose threshold bin holds more tokens than the list (equal or nearly equal logits by the
// thousand) bisect the threshold over the 32 bits of the logit, a pass each.
//
// Measured (GB300): 64 rows of 131072 bf16 logits 15 us without a threshold, 23 us with top_k, 39.5 us with
// top_p alone (one 64-bit shared atomic a token instead of the histogram's two: 59 us); one row of 32000
// 11.5 us.
#include <cooperative_groups.h>
#include <math_constants.h>

#include <atomic>
#include <type_traits>

#include "gptq_device.cuh"
#include "gptq_internal.h"
#include "serving_internal.h"

namespace gptq {
namespace sampling {

namespace cg = cooperative_groups;
typedef unsigned long long u64;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2048, kOver = kBins - 1;     // the last bin: logits too low to have a mass
constexpr int kList = 2048;                        // tokens that are sorted, at most
constexpr int kShortK = 1024;
constexpr int kSubs = 128;                         // sub-runs of a CTA's tokens, 8 a warp
constexpr int kMaxCluster = 8;
constexpr int kMaxSlice = 65535;                   // tokens of a CTA whose 16-bit half masses fit 32-bit sums
constexpr float kReach = 28.f;                     // e^-28 2^39 rounds to no mass
constexpr float kOne = 549755813888.f;             // 2^39, the best token's mass
constexpr float kNearDepth = 5.1986039f;           // 7.5 ln 2: a weight of 2^-7.5 lies so far below the best, times T

// Order-preserving bits of a logit: NaN lowest (0), -0 as 0.
__device__ __forceinline__ uint32_t key_of(float l) {
  if (isnan(l)) return 0u;
  const uint32_t b = __float_as_uint(l + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}
template <int DT>
__device__ __forceinline__ float load_logit(const void* p, int i) {
  if constexpr (DT == 0) return __half2float(static_cast<const __half*>(p)[i]);
  else if constexpr (DT == 1) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}
template <int DT>
__device__ __forceinline__ void unpack(const uint4& x, float (&l)[DT == 2 ? 4 : 8]) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint32_t u = (&x.x)[w];
    if constexpr (DT == 2) {
      l[w] = __uint_as_float(u);
    } else if constexpr (DT == 1) {
      l[2 * w] = __uint_as_float(u << 16);
      l[2 * w + 1] = __uint_as_float(u & 0xFFFF0000u);
    } else {
      l[2 * w] = __half2float(__ushort_as_half(lo16(u)));
      l[2 * w + 1] = __half2float(__ushort_as_half(hi16(u)));
    }
  }
}
// w (at most 1.5) to the nearest whole number of 2^-(U + V), as hi 2^-U + lo 2^-(U + V), added to hi and (signed)
// lo: adding 2^(23 - U) leaves the multiple of 2^-U in the low bits, and what is left of w is exact.
template <int U, int V>
__device__ __forceinline__ void add_parts(float w, uint32_t& hi, uint32_t& lo) {
  constexpr uint32_t kBase = static_cast<uint32_t>(127 + 23 - U) << 23, kRest = static_cast<uint32_t>(127 + 23 - U - V) << 23 | 0x400000u;
  const float t = w + __uint_as_float(kBase);
  hi += __float_as_uint(t) - kBase;
  lo += __float_as_uint((w - (t - __uint_as_float(kBase))) + __uint_as_float(kRest)) - kRest;
}
__device__ __forceinline__ u64 joined(uint32_t hi, uint32_t lo, int v) {
  return (static_cast<u64>(hi) << v) + static_cast<u64>(static_cast<long long>(static_cast<int>(lo)));
}
__device__ __forceinline__ u64 mass_of(float w) {
  uint32_t hi = 0, lo = 0;
  add_parts<20, 19>(w, hi, lo);
  return joined(hi, lo, 19);
}

// Comparisons of whole masses with a fraction of a total, as whole numbers (fp64 is slow here):
// m < fraction * total is m < below_part, and cum > fraction * total is cum >= beyond_part.
__device__ __forceinline__ u64 below_part(float fraction, u64 total) {
  return static_cast<u64>(ceil(static_cast<double>(fraction) * static_cast<double>(total)));
}
__device__ __forceinline__ u64 beyond_part(float fraction, u64 total) {
  return static_cast<u64>(floor(static_cast<double>(fraction) * static_cast<double>(total))) + 1;
}

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
__device__ __forceinline__ u64 warp_scan(u64 v) {          // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 u = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

struct Shared {
  // the histogram; in CTA 0 afterwards its running sums: cum_m[b], cum_c[b] through bin b
  union {
    struct { uint32_t count[kBins], hi[kBins], lo[kBins]; };
    struct { uint32_t cum_c[kBins]; u64 cum_m[kBins]; };
  };
  alignas(16) u64 list[kList];
  u64 slots[2][kMaxCluster];       // cluster sums, every CTA's part in every CTA
  float2 range[kMaxCluster];       // largest logit of each CTA, and the smallest of a sample of its tokens
  u64 part_m[kMaxCluster];         // kept mass above the threshold, and ties, of each CTA
  int part_t[kMaxCluster];
  u64 warp_m[kWarps];
  int warp_t[kWarps];
  u64 sub_m[kSubs];                // the same of each sub-run of this CTA's tokens
  int sub_t[kSubs];
  u64 scan_m[kWarps];
  uint32_t scan_c[kWarps];
  int listed;                      // CTA 0: entries of the list
  int bin_lo, bin_hi, verdict;     // from CTA 0: the bins to list; what happens next
  uint32_t thr;                    // from CTA 0: keys above thr are kept, and the first `ties` of key thr
  int ties;
};

// What a CTA may hold of its row so that two share an SM, or that one has all of it: an SM has 228 KB, of
// which each CTA's launch takes 1 KB
constexpr size_t kSmSmem = 228 * 1024, kCtaSmem = sizeof(Shared) + 1024;
constexpr size_t kHeldOfTwo = (kSmSmem / 2 - kCtaSmem) & ~static_cast<size_t>(15), kHeldOfOne = 160 * 1024;
static_assert(2 * (kHeldOfTwo + kCtaSmem) <= kSmSmem && kHeldOfTwo > 64 * 1024, "two CTAs an SM");
static_assert(kHeldOfOne + kCtaSmem <= kSmSmem, "one CTA an SM");

enum Verdict { kGather = 1, kBisect = 2, kReady = 3 };

// The list's first n entries in descending order (padded with zeros to a power of two).
__device__ void sort_list(u64* list, int n) {
  // a few entries go straight to their places, each the number of larger ones (they differ all): 256
  // take 0.7 us so, and 3 us in the 36 steps below
  if (n <= kThreads) {
    const int i = threadIdx.x;
    u64 e = 0;
    int at = 0;
    __syncthreads();
    if (i < 16 && n + i < kList) list[n + i] = 0ull;
    __syncthreads();
    if ((i & ~31) < n) {
      e = i < n ? list[i] : 0ull;
      for (int j = 0; j < n; j += 16)
#pragma unroll
        for (int o = 0; o < 16; o += 2) {
          const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(list + j + o);
          at += (x.x > e) + (x.y > e);
        }
    }
    __syncthreads();
    if (i < n) list[at] = e;
    __syncthreads();
    return;
  }
  int size = 1;
  while (size < n) size <<= 1;
  for (int i = n + static_cast<int>(threadIdx.x); i < size; i += kThreads) list[i] = 0ull;
  __syncthreads();
  for (int k = 2; k <= size; k <<= 1)
    for (int j = k >> 1; j; j >>= 1) {
      for (int i = threadIdx.x; i < size / 2; i += kThreads) {
        const int a = 2 * i - (i & (j - 1)), b = a + j;    // a: i with a zero bit inserted at j
        const u64 x = list[a], y = list[b];
        if ((x < y) == ((a & k) == 0)) {
          list[a] = y;
          list[b] = x;
        }
      }
      __syncthreads();
    }
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 2) k_sample(const SampleProblem p, int held) {
  __shared__ Shared sh;
  extern __shared__ __align__(16) unsigned char dyn[];
  cg::cluster_group cluster = cg::this_cluster();
  const int cs = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int row = blockIdx.x / cs;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kSize = DT == 2 ? 4 : 2, kVec = 16 / kSize;
  // a CTA's shared memory may be written by the others once it has started
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // this CTA's run of the row, [0, n) of `data`, tokens start + i
  const int start = static_cast<int>(static_cast<long long>(p.vocab) * rank / cs);
  const int n = static_cast<int>(static_cast<long long>(p.vocab) * (rank + 1) / cs) - start;
  const char* src = static_cast<const char*>(p.logits) + (row * p.row_stride + start) * kSize;
  // vectors of 16 bytes from the address below src that is a multiple of 16: token i is element i + skew.
  // What lies before token 0 and after token n - 1 reads as NaN, which no rule keeps.
  const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15) / kSize;
  const int vecs = (n + skew + kVec - 1) / kVec;
  const char* base = src - skew * kSize;
  auto edge_vec = [&](int v, float (&l)[kVec]) {           // from global memory, token by token
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int i = v * kVec + j - skew;
      l[j] = i >= 0 && i < n ? load_logit<DT>(src, i) : CUDART_NAN_F;
    }
  };
  float top = -CUDART_INF_F, low = CUDART_INF_F;           // fmaxf and fminf pass over NaN
  {
    uint4* to = reinterpret_cast<uint4*>(dyn);
    const int inner0 = skew ? 1 : 0, inner1 = (n + skew) / kVec;   // whole vectors
#pragma unroll 4
    for (int v = inner0 + static_cast<int>(threadIdx.x); v < inner1; v += kThreads) {
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(base) + v);
      if (held) to[v] = x;
      float l[kVec];
      unpack<DT>(x, l);
#pragma unroll
      for (int j = 0; j < kVec; ++j) top = fmaxf(top, l[j]);
      low = fminf(low, l[0] > -CUDART_INF_F ? l[0] : low);
    }
    if (threadIdx.x < 2) {                                 // the first and the last, where they are not whole
      const int v = threadIdx.x == 0 ? 0 : vecs - 1;
      if (v < inner0 || v >= inner1) {
        float l[kVec];
        edge_vec(v, l);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          top = fmaxf(top, l[j]);
          low = fminf(low, l[j] > -CUDART_INF_F ? l[j] : low);
          const int i = v * kVec + j - skew;
          if (held) {
            if constexpr (DT == 2) reinterpret_cast<float*>(dyn)[i + skew] = l[j];
            else reinterpret_cast<uint16_t*>(dyn)[i + skew] = i >= 0 && i < n ? reinterpret_cast<const uint16_t*>(src)[i] : uint16_t(0x7FFF);
          }
        }
      }
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    low = fminf(low, __shfl_xor_sync(0xFFFFFFFFu, low, o));
  }
  if (lane == 0) {
    sh.scan_c[warp] = __float_as_uint(top);
    sh.warp_t[warp] = __float_as_int(low);
  }
  for (int i = threadIdx.x; i < kBins; i += kThreads) sh.count[i] = sh.hi[i] = sh.lo[i] = 0u;
  if (threadIdx.x == 0) sh.listed = 0;
  __syncthreads();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (static_cast<int>(threadIdx.x) < cs) {
    for (int w = 0; w < kWarps; ++w) {
      top = fmaxf(top, __uint_as_float(sh.scan_c[w]));
      low = fminf(low, __int_as_float(sh.warp_t[w]));
    }
    cluster.map_shared_rank(&sh, threadIdx.x)->range[rank] = make_float2(top, low);
  }
  cluster.sync();
  for (int r = 0; r < cs; ++r) {
    top = fmaxf(top, sh.range[r].x);
    low = fminf(low, sh.range[r].y);
  }
  // +inf logits share the mass: they count as 0 and the others as -inf
  const bool has_inf = top == CUDART_INF_F;
  if (top == -CUDART_INF_F) {                              // nothing above -inf
    if (rank == 0 && threadIdx.x == 0) {
      p.token[row] = -1;
      if (p.logprob) p.logprob[row] = CUDART_NAN_F;
      atomicOr(p.status, kStatusNoToken);
    }
    return;
  }
  if (has_inf) top = low = 0.f;
  top += 0.f;                                              // -0 as 0
  const uint32_t best = key_of(top);
  float temp = p.temperature ? p.temperature[row] : 1.f;
  const float top_p = p.top_p ? p.top_p[row] : 1.f, min_p = p.min_p ? p.min_p[row] : 0.f;
  float u = p.uniform[row];
  u = u > 0.f ? u : 0.f;
  int k = p.top_k && p.top_k[row] > 0 ? min(p.top_k[row], p.vocab) : p.vocab;
  if (!(temp > 0.f)) {
    temp = 1.f;
    k = 1;
  }
  if (!(top_p > 0.f) || !(min_p <= 1.f)) k = 1;
  auto load_vec = [&](int v, float (&l)[kVec]) {
    if (held) {
      unpack<DT>(reinterpret_cast<const uint4*>(dyn)[v], l);
    } else if (v * kVec >= skew && (v + 1) * kVec <= n + skew) {
      unpack<DT>(__ldg(reinterpret_cast<const uint4*>(base) + v), l);
    } else {
      edge_vec(v, l);
    }
    if (has_inf)
#pragma unroll
      for (int j = 0; j < kVec; ++j) l[j] = l[j] == CUDART_INF_F ? 0.f : -CUDART_INF_F;
  };
  auto each = [&](auto f) {                                // f(logit, token), in any order
#pragma unroll 1
    for (int v = threadIdx.x; v < vecs; v += kThreads) {
      float l[kVec];
      load_vec(v, l);
#pragma unroll
      for (int j = 0; j < kVec; ++j) f(l[j], start + v * kVec + j - skew);
    }
  };
  // w = e^((l - top) / T) as a power of two: the exponent is rounded once more than in the definition,
  // by 2^-24 of itself
  const float rate = fminf(1.44269504088896341f / temp, 3e38f);
  auto weight_of = [&](float l) {
    float w;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"((l - top) * rate));   // 2 units in the last place
    return w;
  };
  auto weight_at = [&](uint32_t key) { return weight_of(logit_of(key)); };
  // the mass with min_p's part of the rule (the best token, of weight 1, always has it); NaN has none
  const float least = min_p > 0.f ? fminf(min_p, 1.f) : 0.f;
  auto kept_mass = [&](float l) {
    const float w = weight_of(l);
    return mass_of(w >= least ? w : 0.f);
  };
  Shared* const boss = cluster.map_shared_rank(&sh, 0);
  int parity = 0;
  auto cluster_sum = [&](u64 v) {                          // of every thread's v
    v = warp_sum(v);
    if (lane == 0) sh.warp_m[warp] = v;
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < cs) {
      u64 all = 0;
      for (int w = 0; w < kWarps; ++w) all += sh.warp_m[w];
      cluster.map_shared_rank(&sh, threadIdx.x)->slots[parity][rank] = all;
    }
    cluster.sync();
    u64 all = 0;
    for (int r = 0; r < cs; ++r) all += sh.slots[parity][r];
    parity ^= 1;
    return all;
  };
  auto write = [&](int token, uint32_t key, u64 total) {
    p.token[row] = token;
    if (p.logprob)
      p.logprob[row] = (logit_of(key) - top) / temp - logf(static_cast<float>(total) * (1.f / kOne));
  };

  uint32_t thr = 0u;
  int ties = p.vocab;
  if (k == 1) {
    thr = best;
    ties = 1;
  } else if (k < p.vocab || top_p < 1.f) {
    const bool short_k = k <= kShortK;
    // ---- the histogram of top - l over the reach of the masses
    const float reach = fminf(kReach * temp, 3.402823466e38f), span = low <= top ? fminf(top - low, reach) : reach;
    // bins a unit of the logits: the span's, but none finer than weights can tell (1e-9 T)
    const float scale = fminf(fminf((kOver - 0.5f) / span, 1e9f / temp), 3e38f);
    // NaN, -inf and what has no mass: the last bin; what is lower than the sampled lowest: the two before.
    // Bins below `edge`, a whole number of them or all but those of tokens past it, hold masses in units of
    // 2^-31, which weights of 2^-8 and more are multiples of, the others, below 2^-7, 2^8 times finer ones
    // (edge lies at weights of 2^-7.5, and a bin is far narrower than that).  So the sums over 65535 tokens of
    // the two halves of either take 32 bits each
    const float at_near = kNearDepth * (temp * scale);
    const float edge = at_near < kOver - 2 ? fmaxf(floorf(at_near), 1.f) : fmaxf(at_near, kOver - 1.f);
    auto place_of = [&](float l, bool& near) {             // (not called past the reach)
      const float x = (top - l) * scale;
      near = x < edge;
      return static_cast<int>(fminf(x, near ? kOver - 2.f : kOver - 1.f));
    };
    auto bin_of = [&](float l) {
      bool near;
      return top - l <= reach ? place_of(l, near) : kOver;
    };
    const bool by_mass = top_p < 1.f && !short_k;
    const bool fits = n <= kMaxSlice;
    if (by_mass && fits)
      each([&](float l, int) {
        if (top - l <= reach) {
          bool near;
          const int b = place_of(l, near);
          const float w = weight_of(l);
          uint32_t hi = 0, lo = 0;
          add_parts<15, 16>(near ? w : 256.f * w, hi, lo);
          if (k < p.vocab) atomicAdd(&sh.count[b], 1u);    // else the list's own count will do
          atomicAdd(&sh.hi[b], hi);
          atomicAdd(&sh.lo[b], lo);
        }
      });
    else if (short_k && p.vocab / kVec >= 4 * k)
      // the largest of each vector only: k vectors reach as far down as their k-th largest, so at least k
      // tokens do, and what lies above is little more than k tokens
      for (int v = threadIdx.x; v < vecs; v += kThreads) {
        float l[kVec], most = -CUDART_INF_F;
        load_vec(v, l);
#pragma unroll
        for (int j = 0; j < kVec; ++j) most = fmaxf(most, l[j]);
        const int b = bin_of(most);
        if (b < kOver) atomicAdd(&sh.count[b], 1u);
      }
    else
      each([&](float l, int) {
        const int b = bin_of(l);
        if (b < kOver) atomicAdd(&sh.count[b], 1u);
      });
    cluster.sync();
    // ---- CTA 0: running sums over the cluster's bins, 4 bins a thread
    u64 mass_total = 0;
    if (rank == 0) {
      constexpr int kPer = kBins / kThreads;
      static_assert(kPer == 4, "a uint4 of bins per thread");
      u64 m[4] = {};
      uint32_t c[4] = {};
#pragma unroll 4
      for (int r = 0; r < cs; ++r) {
        const Shared* s = cluster.map_shared_rank(&sh, r);
        const uint4 x = reinterpret_cast<const uint4*>(s->count)[threadIdx.x];
        c[0] += x.x; c[1] += x.y; c[2] += x.z; c[3] += x.w;
        if (by_mass) {
          const uint4 h = reinterpret_cast<const uint4*>(s->hi)[threadIdx.x], l = reinterpret_cast<const uint4*>(s->lo)[threadIdx.x];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const u64 sum = joined((&h.x)[j], (&l.x)[j], 16);
            m[j] += static_cast<float>(4 * threadIdx.x + j) < fminf(edge, kOver - 1.f) ? sum << 8 : sum;
          }
        }
      }
#pragma unroll
      for (int j = 1; j < 4; ++j) {
        c[j] += c[j - 1];
        m[j] += m[j - 1];
      }
      const u64 wm = warp_scan(m[3]), wc = warp_scan(c[3]);
      if (lane == 31) {
        sh.scan_m[warp] = wm;
        sh.scan_c[warp] = static_cast<uint32_t>(wc);
      }
      __syncthreads();                                     // and every thread has read this CTA's bins
      u64 m0 = wm - m[3], c0 = wc - c[3];
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) {
          m0 += sh.scan_m[w];
          c0 += sh.scan_c[w];
        }
        mass_total += sh.scan_m[w];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sh.cum_c[4 * threadIdx.x + j] = c[j] + static_cast<uint32_t>(c0);
        sh.cum_m[4 * threadIdx.x + j] = m[j] + m0;
      }
      __syncthreads();
    }
    // CTA 0: the first bin through which a running sum reaches a goal (kOver: none does)
    auto first_bin = [&](auto reaches) {
      int b = kOver;
      for (int i = threadIdx.x; i < kOver; i += kThreads)
        if (reaches(i)) {
          b = i;
          break;
        }
      b = __reduce_min_sync(0xFFFFFFFFu, b);
      __syncthreads();
      if (lane == 0) sh.warp_t[warp] = b;
      __syncthreads();
      for (int w = 0; w < kWarps; ++w) b = min(b, sh.warp_t[w]);
      return b;
    };
    auto tell = [&](int verdict, int lo, int hi) {         // CTA 0 to all
      if (static_cast<int>(threadIdx.x) < cs) {
        Shared* s = cluster.map_shared_rank(&sh, threadIdx.x);
        s->verdict = verdict;
        s->bin_lo = lo;
        s->bin_hi = hi;
        s->thr = thr;
        s->ties = ties;
      }
    };
    auto below = [&](int b) { return b > 0 ? sh.cum_c[b - 1] : 0u; };
    auto below_m = [&](int b) { return b > 0 ? sh.cum_m[b - 1] : 0ull; };
    // all CTAs: the tokens of bins bin_lo .. bin_hi into CTA 0's list, from a list of this CTA's own (an
    // atomic on another CTA's memory takes most of a microsecond, one after the other in a warp).  Of one
    // bin (`few`) a warp seldom has a token, and looks for it by its bit (64 rows of 131072 with top_p: 37.4
    // us, 39.2 token by token); all bins down to the k-th token's hold some of nearly every warp's, and a
    // loop over the bits of its busiest lane takes longer (256 rows of 50257 with top_k: 31 us, 50 so)
    auto gather = [&](auto few) {
      const int lo = sh.bin_lo, hi = sh.bin_hi;
      // most tokens are below or above: two comparisons, with half a bin to spare for their rounding
      const float floor = hi < kOver - 2 ? top - (hi + 1.5f) / scale * (1.f + 1e-5f) : -CUDART_INF_F;
      const float roof = top - (lo - 0.5f) / scale * (1.f - 1e-5f);
#pragma unroll 2
      for (int v = threadIdx.x; v < vecs; v += kThreads) {
        float l[kVec];
        load_vec(v, l);
        auto put = [&](float one, int i) {
          const int b = bin_of(one);
          if (b >= lo && b <= hi) {
            const int at = atomicAdd(&sh.listed, 1);
            if (at < kList) sh.list[at] = static_cast<u64>(key_of(one)) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(start + i));
          }
        };
        if constexpr (few.value) {
          uint32_t hits = 0;
#pragma unroll
          for (int j = 0; j < kVec; ++j) hits |= l[j] >= floor && l[j] <= roof ? 1u << j : 0u;
          while (hits) {
            const int at_j = __ffs(hits) - 1;
            hits &= hits - 1;
            float one = l[0];
#pragma unroll
            for (int j = 1; j < kVec; ++j) one = at_j == j ? l[j] : one;
            put(one, v * kVec + at_j - skew);
          }
        } else {
          bool any = false;
#pragma unroll
          for (int j = 0; j < kVec; ++j) any |= l[j] >= floor && l[j] <= roof;
          if (!any) continue;
#pragma unroll
          for (int j = 0; j < kVec; ++j) put(l[j], v * kVec + j - skew);
        }
      }
      if (rank != 0) {
        __syncthreads();
        const int count = sh.listed;
        if (threadIdx.x == 0) sh.bin_lo = count > 0 ? atomicAdd(&boss->listed, count) : 0;
        __syncthreads();
        const int at = sh.bin_lo;
        for (int i = threadIdx.x; i < count && at + i < kList && i < kList; i += kThreads) boss->list[at + i] = sh.list[i];
        if (threadIdx.x == 0) sh.listed = 0;
      }
    };
    auto key_in = [&](int i) { return static_cast<uint32_t>(sh.list[i] >> 32); };
    // CTA 0: the place of the threshold after the first r of the sorted list: its key, and how many of
    // that key are kept
    auto cut_after = [&](int r) {
      const uint32_t key = key_in(r - 1);
      int same = 0;
      for (int i = threadIdx.x; i < r; i += kThreads) same += key_in(i) == key;
      same = __reduce_add_sync(0xFFFFFFFFu, same);
      __syncthreads();
      if (lane == 0) sh.warp_t[warp] = same;
      __syncthreads();
      same = 0;
      for (int w = 0; w < kWarps; ++w) same += sh.warp_t[w];
      thr = key;
      ties = same;
    };
    // CTA 0: masses of the sorted list's first r in order, this thread's 4 before / sum
    auto scan_list = [&](int r, auto mass, u64 (&before)[4], u64 (&m)[4]) {
      u64 sum = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = 4 * threadIdx.x + j;
        m[j] = i < r ? mass(i) : 0ull;
        before[j] = sum;
        sum += m[j];
      }
      const u64 incl = warp_scan(sum);
      __syncthreads();
      if (lane == 31) sh.scan_m[warp] = incl;
      __syncthreads();
      u64 base = incl - sum, total = 0;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) base += sh.scan_m[w];
        total += sh.scan_m[w];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) before[j] += base;
      return total;
    };
    auto count_true = [&](int v) {
      v = __reduce_add_sync(0xFFFFFFFFu, v);
      __syncthreads();
      if (lane == 0) sh.warp_t[warp] = v;
      __syncthreads();
      v = 0;
      for (int w = 0; w < kWarps; ++w) v += sh.warp_t[w];
      return v;
    };
    static_assert(kList == 4 * kThreads, "4 entries of the list per thread");

    if (short_k) {
      if (rank == 0) {
        const int b = first_bin([&](int i) { return sh.cum_c[i] >= static_cast<uint32_t>(k); });
        const int last = b < kOver ? b : kOver - 1;        // fewer than k tokens with a mass: all of them
        tell(sh.cum_c[last] <= kList ? kGather : kBisect, 0, last);
      }
      cluster.sync();
      bool listed = false;
      if (sh.verdict == kGather) {
        gather(std::false_type());
        cluster.sync();
        listed = boss->listed <= kList;                    // (the bins counted vectors, not tokens)
        cluster.sync();
      }
      if (listed) {
        if (rank != 0) return;                             // CTA 0 has everything that can be kept
        int r = sh.listed;
        sort_list(sh.list, r);
        r = min(r, k);
        u64 before[4], m[4];
        const u64 all = scan_list(r, [&](int i) { return mass_of(weight_at(key_in(i))); }, before, m);
        const u64 limit = top_p < 1.f ? below_part(top_p, all) : ~0ull;
        int keep = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = 4 * threadIdx.x + j;
          keep += i < r && (i == 0 || (before[j] < limit && weight_at(key_in(i)) >= min_p));
        }
        r = count_true(keep);                              // the kept ones are a prefix
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (4 * static_cast<int>(threadIdx.x) + j == r - 1) sh.slots[0][0] = before[j] + m[j];   // their mass
        // in index order: by adding up, of a few, those of lower index
        if (r <= kThreads) {
          u64* const mass = sh.cum_m;
          const int i = threadIdx.x;
          const u64 e = i < r ? sh.list[i] : 0ull;
          const u64 mine = i < r ? mass_of(weight_at(static_cast<uint32_t>(e >> 32))) : 0ull;
          mass[i] = mine;
          __syncthreads();
          if ((i & ~31) < r) {
            const u64 total = sh.slots[0][0];
            u64 lower = 0;
#pragma unroll 2
            for (int j0 = 0; j0 < r; j0 += 4) {            // (past r the masses are 0)
              const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(mass + j0), b = *reinterpret_cast<const ulonglong2*>(mass + j0 + 2);
              const u64 four[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (static_cast<uint32_t>(sh.list[j0 + j]) > static_cast<uint32_t>(e)) lower += four[j];   // ~index
            }
            // the token whose masses reach past the target (u >= 1: the last one)
            const u64 goal = min(beyond_part(u, total), total), end = lower + mine;
            if (i < r && lower < goal && goal <= end) write(static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(e)), static_cast<uint32_t>(e >> 32), total);
          }
          return;
        }
        // or sorted: (index, key) ascending is (~index, key) descending
        for (int i = threadIdx.x; i < r; i += kThreads) {
          const u64 e = sh.list[i];
          sh.list[i] = e << 32 | e >> 32;
        }
        __syncthreads();
        sort_list(sh.list, r);
        auto low_key = [&](int i) { return static_cast<uint32_t>(sh.list[i]); };
        const u64 total = scan_list(r, [&](int i) { return mass_of(weight_at(low_key(i))); }, before, m);
        const u64 goal = min(beyond_part(u, total), total);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = 4 * threadIdx.x + j;
          if (i < r && before[j] < goal && goal <= before[j] + m[j]) write(static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(sh.list[i] >> 32)), low_key(i), total);
        }
        return;
      }
    } else {
      // a long top_k or none: the bin of the k-th token, then the bin where top_p of the mass is reached
      if (rank == 0) {
        const int b = k < p.vocab ? first_bin([&](int i) { return sh.cum_c[i] >= static_cast<uint32_t>(k); }) : kOver;
        if (b < kOver) {
          const uint32_t in = sh.cum_c[b] - below(b);
          tell(in <= kList && (!by_mass || p.vocab <= kMaxSlice * cs) ? kGather : kBisect, b, b);
        } else if (by_mass) {
          // top_k cuts nothing that has a mass
          const u64 limit = below_part(top_p, mass_total);
          const int pb = first_bin([&](int i) { return sh.cum_m[i] >= limit; });
          const uint32_t in = pb < kOver ? sh.cum_c[pb] - below(pb) : 0u;
          tell(p.vocab > kMaxSlice * cs || in > kList ? kBisect : (pb < kOver ? kGather : kReady), pb, pb);
        } else {
          tell(kReady, 0, 0);
        }
      }
      cluster.sync();
      const bool k_first = k < p.vocab;
      if (sh.verdict == kGather) {
        gather(std::true_type());
        cluster.sync();
        if (rank == 0 && sh.listed > kList) {
          __syncthreads();                                 // (every thread has read it)
          tell(kBisect, 0, 0);
        } else if (rank == 0) {
          int bin = sh.bin_lo, r = sh.listed;
          sort_list(sh.list, r);
          bool again = false;
          u64 before[4], m[4];
          u64 goal_mass = mass_total;
          int within = r;                                  // of the sorted list, what top_k leaves
          const bool cut_k = k_first && sh.cum_c[bin] >= static_cast<uint32_t>(k) && below(bin) < static_cast<uint32_t>(k);
          if (cut_k) {
            within = k - static_cast<int>(below(bin));
            cut_after(within);
            if (by_mass) {
              goal_mass = below_m(bin) + scan_list(within, [&](int i) { return mass_of(weight_at(key_in(i))); }, before, m);
              const u64 limit = below_part(top_p, goal_mass);
              const int pb = first_bin([&](int i) { return i >= bin || sh.cum_m[i] >= limit; });
              if (pb < bin) {                              // top_p ends in an earlier bin: list that one
                const uint32_t in = sh.cum_c[pb] - below(pb);
                again = true;
                if (threadIdx.x == 0) {
                  sh.listed = 0;
                  sh.slots[0][0] = goal_mass;              // (no cluster sum runs meanwhile)
                }
                tell(in <= kList ? kGather : kBisect, pb, pb);
              }
            }
          }
          if (!again) {
            if (by_mass) {
              const u64 limit = below_part(top_p, goal_mass);
              scan_list(within, [&](int i) { return mass_of(weight_at(key_in(i))); }, before, m);
              int keep = 0;
#pragma unroll
              for (int j = 0; j < 4; ++j)
                keep += 4 * static_cast<int>(threadIdx.x) + j < within && before[j] + below_m(bin) < limit;
              keep = count_true(keep);
              cut_after(keep > 0 ? keep : 1);
            }
            tell(kReady, 0, 0);
          }
        }
        cluster.sync();
        if (sh.verdict == kGather) {                       // the earlier bin
          gather(std::true_type());
          cluster.sync();
          if (rank == 0) {
            const int bin = sh.bin_lo, r = sh.listed;
            const u64 limit = below_part(top_p, sh.slots[0][0]);
            sort_list(sh.list, r);
            u64 before[4], m[4];
            scan_list(r, [&](int i) { return mass_of(weight_at(key_in(i))); }, before, m);
            int keep = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              keep += 4 * static_cast<int>(threadIdx.x) + j < r && before[j] + below_m(bin) < limit;
            keep = count_true(keep);
            cut_after(keep > 0 ? keep : 1);
            tell(kReady, 0, 0);
          }
          cluster.sync();
        }
      }
      if (sh.verdict == kReady) {
        thr = sh.thr;
        ties = sh.ties;
      }
    }
    if (short_k || sh.verdict == kBisect) {                // (a short top_k that could be listed has returned)
      thr = 0u;
      ties = p.vocab;
      auto mass_at = [&](uint32_t key) { return key ? mass_of(weight_at(key)) : 0ull; };
      if (k < p.vocab) {
        for (int bit = 31; bit >= 0; --bit) {
          const uint32_t cand = thr | (1u << bit);
          u64 c = 0;
          each([&](float l, int) { c += key_of(l) >= cand; });
          if (cluster_sum(c) >= static_cast<u64>(k)) thr = cand;
        }
        u64 c = 0;
        each([&](float l, int) { c += key_of(l) > thr; });
        ties = k - static_cast<int>(cluster_sum(c));
      }
      if (top_p < 1.f) {
        auto above = [&](uint32_t v) {                     // mass of the keys above v
          u64 m = 0;
          each([&](float l, int) {
            const uint32_t key = key_of(l);
            if (key > v) m += mass_at(key);
          });
          return cluster_sum(m);
        };
        u64 at_thr = 0;
        each([&](float l, int) { at_thr += key_of(l) == thr; });
        at_thr = cluster_sum(at_thr);
        if (at_thr > static_cast<u64>(ties)) at_thr = ties;
        const u64 limit = below_part(top_p, above(thr) + at_thr * mass_at(thr));
        // the smallest key v >= thr with less than the limit above it
        uint32_t lo = thr, hi = best;
        while (lo < hi) {
          const uint32_t mid = lo + (hi - lo) / 2;
          if (above(mid) < limit) hi = mid;
          else lo = mid + 1;
        }
        const u64 a = above(lo), m = mass_at(lo);
        int r = lo == thr ? ties : p.vocab;
        if (m > 0) {                                       // ties i = 0, 1, ... stay while a + i m < limit
          const u64 q = limit > a ? (limit - a + m - 1) / m : 1;
          if (q < static_cast<u64>(r)) r = static_cast<int>(q);
        }
        thr = lo;
        ties = r;
      }
    }
  }

  // ---- the kept masses in index order: sub-runs of this CTA's tokens, then the CTAs.  Ties have one
  // mass each, so a sub-run needs only the mass above the threshold and its number of ties.
  const float cut = thr ? logit_of(thr) : -CUDART_INF_F;   // (nothing is cut: ties of -inf have no mass)
  const u64 tie_mass = thr ? kept_mass(cut) : 0ull;
  const int chunks = (vecs + 31) / 32;                     // a sub-run is whole chunks of 32 vectors
  auto sub_begin = [&](int q) { return static_cast<int>(static_cast<long long>(chunks) * q / kSubs); };
  auto chunk_at = [&](int c, float (&l)[kVec]) {
    if (c * 32 + lane < vecs) {
      load_vec(c * 32 + lane, l);
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j) l[j] = CUDART_NAN_F;
    }
  };
#pragma unroll 2
  for (int q = warp * (kSubs / kWarps); q < (warp + 1) * (kSubs / kWarps); ++q) {
    uint32_t hi = 0, lo = 0;
    int t = 0;
    const int c1 = sub_begin(q + 1);
#pragma unroll 1
    for (int c = sub_begin(q); c < c1; ++c) {
      float l[kVec];
      chunk_at(c, l);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        const float w = weight_of(l[j]);                   // (without a branch around it)
        add_parts<20, 19>(l[j] > cut && w >= least ? w : 0.f, hi, lo);
        t += l[j] == cut;
      }
    }
    // a sub-run holds less than 2^13 tokens, a lane of it less than 2^9: hi stays below 2^29, lo below 2^28
    u64 mine = joined(hi, lo, 19);
    const u64 part = __reduce_add_sync(0xFFFFFFFFu, static_cast<uint32_t>(mine) & 0x7FFFFFFu);
    mine = (static_cast<u64>(__reduce_add_sync(0xFFFFFFFFu, static_cast<uint32_t>(mine >> 27))) << 27) + part;
    t = __reduce_add_sync(0xFFFFFFFFu, t);
    if (lane == 0) {
      sh.sub_m[q] = mine;
      sh.sub_t[q] = t;
    }
  }
  __syncthreads();
  // warp 0 goes on alone: 4 sub-runs a lane, summed for the cluster
  if (warp == 0) {
    u64 all = 0;
    int ties_here = 0;
#pragma unroll
    for (int j = 0; j < kSubs / 32; ++j) {
      all += sh.sub_m[lane * (kSubs / 32) + j];
      ties_here += sh.sub_t[lane * (kSubs / 32) + j];
    }
    all = warp_sum(all);
    ties_here = __reduce_add_sync(0xFFFFFFFFu, ties_here);
    if (lane < cs) {
      Shared* s = cluster.map_shared_rank(&sh, lane);
      s->part_m[rank] = all;
      s->part_t[rank] = ties_here;
    }
  }
  cluster.sync();                                          // the last access to another CTA's memory
  if (warp != 0) return;
  u64 before = 0, total = 0;                               // kept mass before this CTA's tokens, in all
  int tied = 0, seen = 0;                                  // ties before them
  auto kept_ties = [&](int from, int count) { return max(0, min(count, ties - from)); };
  for (int r = 0; r < cs; ++r) {
    const u64 m = sh.part_m[r] + static_cast<u64>(kept_ties(seen, sh.part_t[r])) * tie_mass;
    if (r == rank) {
      before = total;
      tied = seen;
    }
    total += m;
    seen += sh.part_t[r];
  }
  // the sub-run in which the kept masses reach past the target (u >= 1: the one where they end)
  const u64 goal = min(beyond_part(u, total), total);
  int q = -1;
  {
    constexpr int kEach = kSubs / 32;
    int t[kEach], lane_t = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) lane_t += t[j] = sh.sub_t[lane * kEach + j];
    int from = lane_t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, from, o);
      if (lane >= o) from += v;
    }
    from += tied - lane_t;
    u64 m[kEach], lane_m = 0;
    int f = from;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      m[j] = sh.sub_m[lane * kEach + j] + static_cast<u64>(kept_ties(f, t[j])) * tie_mass;
      f += t[j];
      lane_m += m[j];
    }
    u64 at = before + warp_scan(lane_m) - lane_m;
    f = from;
    int mine = -1;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      if (at < goal && goal <= at + m[j]) {
        mine = lane * kEach + j;
        before = at;
        tied = f;
      }
      at += m[j];
      f += t[j];
    }
    const unsigned who = __ballot_sync(0xFFFFFFFFu, mine >= 0);
    if (who == 0) return;                                  // in another CTA's tokens
    const int owner = __ffs(who) - 1;
    q = __shfl_sync(0xFFFFFFFFu, mine, owner);
    before = __shfl_sync(0xFFFFFFFFu, before, owner);
    tied = __shfl_sync(0xFFFFFFFFu, tied, owner);
  }
  const int c1 = sub_begin(q + 1);
  for (int c = sub_begin(q); c < c1; ++c) {
    float l[kVec];
    chunk_at(c, l);
    int t = 0;
#pragma unroll
    for (int j = 0; j < kVec; ++j) t += l[j] == cut;
    int tscan = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, tscan, o);
      if (lane >= o) tscan += v;
    }
    int at = tied + tscan - t;
    u64 m[kVec], sum = 0;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      m[j] = l[j] > cut ? kept_mass(l[j]) : 0ull;
      if (l[j] == cut && at++ < ties) m[j] = tie_mass;
      sum += m[j];
    }
    const u64 incl = warp_scan(sum);
    u64 run = before + incl - sum;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const u64 e = run + m[j];
      if (run < goal && goal <= e) write(start + (c * 32 + lane) * kVec + j - skew, key_of(l[j]), total);
      run = e;
    }
    before += __shfl_sync(0xFFFFFFFFu, incl, 31);
    tied += __shfl_sync(0xFFFFFFFFu, tscan, 31);
    if (before >= goal) break;
  }
}

template <int DT>
cudaError_t launch(const SampleProblem& p, cudaStream_t stream) {
  constexpr int kSize = DT == 2 ? 4 : 2;
  const DeviceInfo& dev = device_info();
  // CTAs per row: as many as run at once, two on an SM, and more where the row's masses need them for
  // exact sums of 32 bits; at most 2 * kThreads tokens a CTA are too few to split
  int cs = 1;
  while (cs < kMaxCluster && p.vocab / cs > 2 * kThreads &&
         (static_cast<long long>(p.batch) * 2 * cs <= 2 * dev.sm_count || p.vocab > kMaxSlice * cs))
    cs *= 2;
  // the row stays in shared memory where that leaves room for as many CTAs; else it is read again from L2
  // (256 rows of 36000 / 36500 fp16 logits, mixed settings: 36 us held and 39 read again; held all the same,
  // with one CTA an SM, 36500 took 43)
  size_t smem = ((static_cast<size_t>(p.vocab) / cs + 1) * kSize + 31) & ~static_cast<size_t>(15);
  const bool one_each = static_cast<long long>(p.batch) * cs <= dev.sm_count;
  const bool held = smem <= (one_each ? kHeldOfOne : kHeldOfTwo);
  if (!held) smem = 0;
  auto kern = k_sample<DT>;
  static std::atomic<unsigned long long> opted_in{0};       // per device
  if (dev.device >= 64 || !(opted_in.load(std::memory_order_relaxed) & (1ull << dev.device))) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kHeldOfOne));
    if (e != cudaSuccess) return e;
    if (dev.device < 64) opted_in.fetch_or(1ull << dev.device, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.batch) * cs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, p, static_cast<int>(held));
}

}  // namespace sampling

cudaError_t launch_sample(const SampleProblem& p, cudaStream_t stream) {
  if (p.dtype == 0) return sampling::launch<0>(p, stream);
  if (p.dtype == 1) return sampling::launch<1>(p, stream);
  return sampling::launch<2>(p, stream);
}

}  // namespace gptq
