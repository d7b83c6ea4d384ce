// sample.cu -- one token for each row of logits, from a given uniform number (gptq_sample).
//
// With x = (l - max l) / T, w = e^x and the tokens ordered by l (equal ones by index), every setting
// keeps a prefix of that order: the first top_k, then those before which less than top_p of the mass
// lies, then those with w >= min_p.  So the kept set is "logits above a threshold, and the first few of
// those equal to it", and the token is found by cumulating the kept masses in index order.  Nothing is
// sorted but the few tokens around a threshold.  Masses are integers of 2^-32 of the best token's, whose
// sums do not depend on their order: atomics and splits do not change a result.
//
// Bound: the logits are read once from HBM (a cluster of CTAs holds a row in its shared memory); what
// costs time is the passes over the row on chip and the cluster's barriers between them.
//   1. load, largest and smallest logit;
//   2. a histogram of max - l: counts, and masses where the mass decides (no top_k, or a long one);
//   3. with a short top_k, everything down to the bin that holds the k-th goes to one CTA, which sorts
//      and finishes; otherwise the tokens of the bin that the threshold falls into are sorted there;
//   4. the kept masses summed and searched in index order.
// Rows whose threshold bin holds more tokens than the list (equal or nearly equal logits by the
// thousand) bisect the threshold over the 32 bits of the logit, a pass each.
#include <cooperative_groups.h>
#include <math_constants.h>

#include <atomic>

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
constexpr int kMaxCluster = 8;
constexpr int kMaxSlice = 65535;                   // tokens of a CTA whose 16-bit half masses fit 32-bit sums
constexpr float kReach = 24.f;                     // e^-24 2^32 rounds to no mass

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
__device__ __forceinline__ u64 mass_of(float w) { return __float2ull_rn(w * 4294967296.f); }

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
  u64 list[kList];
  u64 slots[2][kMaxCluster];       // cluster sums, every CTA's part in every CTA
  uint2 range[kMaxCluster];        // largest and smallest key of each CTA
  u64 part_m[kMaxCluster];         // kept mass above the threshold, and ties, of each CTA
  int part_t[kMaxCluster];
  u64 warp_m[kWarps];
  int warp_t[kWarps];
  u64 scan_m[kWarps];
  uint32_t scan_c[kWarps];
  int listed;                      // CTA 0: entries of the list
  int bin_lo, bin_hi, verdict;     // from CTA 0: the bins to list; what happens next
  uint32_t thr;                    // from CTA 0: keys above thr are kept, and the first `ties` of key thr
  int ties;
  int found;
  uint32_t found_key;
};

enum Verdict { kGather = 1, kBisect = 2, kReady = 3 };

// The list's first n entries in descending order (padded with zeros to a power of two).
__device__ void sort_list(u64* list, int n) {
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
__global__ void __launch_bounds__(kThreads) k_sample(const SampleProblem p, int held) {
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
  const void* data = src;
  uint32_t best = 0u, least = 0xFFFFFFFFu;
  auto see = [&](float l) {
    const uint32_t k = key_of(l);
    best = max(best, k);
    if (k > 0x007FFFFFu) least = min(least, k);            // not NaN, not -inf
  };
  {
    // 16 bytes at a time between the ends, kept at the same place modulo 16 in shared memory
    const int head = min(n, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(src) & 15)) & 15) / kSize);
    const int vecs = (n - head) / kVec;
    unsigned char* to = dyn + (reinterpret_cast<uintptr_t>(src) & 15);
    auto one = [&](int i) {
      const float l = load_logit<DT>(src, i);
      see(l);
      if (held) {
        if constexpr (DT == 2) reinterpret_cast<float*>(to)[i] = l;
        else reinterpret_cast<uint16_t*>(to)[i] = reinterpret_cast<const uint16_t*>(src)[i];
      }
    };
    if (static_cast<int>(threadIdx.x) < head) one(threadIdx.x);
    const int tail = head + vecs * kVec + static_cast<int>(threadIdx.x);
    if (tail < n) one(tail);
    const uint4* from = reinterpret_cast<const uint4*>(src + head * kSize);
    uint4* into = reinterpret_cast<uint4*>(to + head * kSize);
#pragma unroll 4
    for (int v = threadIdx.x; v < vecs; v += kThreads) {
      const uint4 x = __ldg(from + v);
      if (held) into[v] = x;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t u = (&x.x)[w];
        if constexpr (DT == 2) {
          see(__uint_as_float(u));
        } else if constexpr (DT == 1) {
          see(__uint_as_float(u << 16));
          see(__uint_as_float(u & 0xFFFF0000u));
        } else {
          see(__half2float(__ushort_as_half(lo16(u))));
          see(__half2float(__ushort_as_half(hi16(u))));
        }
      }
    }
    if (held) data = to;
  }
  best = __reduce_max_sync(0xFFFFFFFFu, best);
  least = __reduce_min_sync(0xFFFFFFFFu, least);
  if (lane == 0) {
    sh.scan_c[warp] = best;
    sh.warp_t[warp] = static_cast<int>(least);
  }
  for (int i = threadIdx.x; i < kBins; i += kThreads) sh.count[i] = sh.hi[i] = sh.lo[i] = 0u;
  if (threadIdx.x == 0) {
    sh.listed = 0;
    sh.found = -1;
  }
  __syncthreads();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (static_cast<int>(threadIdx.x) < cs) {
    for (int w = 0; w < kWarps; ++w) {
      best = max(best, sh.scan_c[w]);
      least = min(least, static_cast<uint32_t>(sh.warp_t[w]));
    }
    cluster.map_shared_rank(&sh, threadIdx.x)->range[rank] = make_uint2(best, least);
  }
  cluster.sync();
  for (int r = 0; r < cs; ++r) {
    best = max(best, sh.range[r].x);
    least = min(least, sh.range[r].y);
  }
  // +inf logits share the mass: they count as 0 and the others as -inf
  const bool has_inf = best == key_of(CUDART_INF_F);
  if (best <= key_of(-CUDART_INF_F)) {                     // nothing above -inf
    if (rank == 0 && threadIdx.x == 0) {
      p.token[row] = -1;
      if (p.logprob) p.logprob[row] = CUDART_NAN_F;
      atomicOr(p.status, kStatusNoToken);
    }
    return;
  }
  const float top = has_inf ? 0.f : logit_of(best);
  best = key_of(top);
  const float low = has_inf ? 0.f : logit_of(least);
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
  auto value_at = [&](int i) {
    const float l = load_logit<DT>(data, i);
    return has_inf ? (l == CUDART_INF_F ? 0.f : -CUDART_INF_F) : l;
  };
  auto weight_at = [&](uint32_t key) { return expf((logit_of(key) - top) / temp); };
  auto kept_mass = [&](uint32_t key) {                     // min_p's part of the rule included
    const float w = weight_at(key);
    return w >= min_p || key == best ? mass_of(w) : 0ull;
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
      p.logprob[row] = static_cast<float>(static_cast<double>((logit_of(key) - top) / temp) -
                                          log(static_cast<double>(total) / 4294967296.0));
  };

  uint32_t thr = 0u;
  int ties = p.vocab;
  if (k == 1) {
    thr = best;
    ties = 1;
  } else if (k < p.vocab || top_p < 1.f) {
    const bool short_k = k <= kShortK;
    // ---- the histogram of top - l over the reach of the masses
    const float span = fminf(top - low, kReach * temp);
    const float scale = span > 0.f ? fminf((kOver - 0.5f) / span, 3e38f) : 0.f;
    auto bin_of = [&](float l) {                           // NaN and -inf: the last
      const float d = (top - l) * scale;
      return d < static_cast<float>(kOver) ? static_cast<int>(d) : kOver;
    };
    const bool by_mass = top_p < 1.f && !short_k;
    const bool fits = n <= kMaxSlice;
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const float l = value_at(i);
      const int b = bin_of(l);
      if (b < kOver) {
        atomicAdd(&sh.count[b], 1u);
        if (by_mass && fits) {
          const u64 m = mass_of(expf((l - top) / temp));
          atomicAdd(&sh.hi[b], static_cast<uint32_t>(m >> 16));
          atomicAdd(&sh.lo[b], static_cast<uint32_t>(m & 0xFFFFu));
        }
      }
    }
    cluster.sync();
    // ---- CTA 0: running sums over the cluster's bins, 4 bins a thread
    u64 mass_total = 0;
    if (rank == 0) {
      constexpr int kPer = kBins / kThreads;
      static_assert(kPer == 4, "a uint4 of bins per thread");
      u64 m[4] = {};
      uint32_t c[4] = {};
      for (int r = 0; r < cs; ++r) {
        const Shared* s = cluster.map_shared_rank(&sh, r);
        const uint4 x = reinterpret_cast<const uint4*>(s->count)[threadIdx.x];
        c[0] += x.x; c[1] += x.y; c[2] += x.z; c[3] += x.w;
        if (by_mass) {
          const uint4 h = reinterpret_cast<const uint4*>(s->hi)[threadIdx.x], l = reinterpret_cast<const uint4*>(s->lo)[threadIdx.x];
#pragma unroll
          for (int j = 0; j < 4; ++j) m[j] += (static_cast<u64>((&h.x)[j]) << 16) + (&l.x)[j];
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
    // all CTAs: the tokens of bins bin_lo .. bin_hi into CTA 0's list
    auto gather = [&]() {
      const int lo = sh.bin_lo, hi = sh.bin_hi;
      for (int i = threadIdx.x; i < n; i += kThreads) {
        const float l = value_at(i);
        const int b = bin_of(l);
        if (b >= lo && b <= hi) {
          const int at = atomicAdd(&boss->listed, 1);
          if (at < kList) boss->list[at] = static_cast<u64>(key_of(l)) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(start + i));
        }
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
      if (sh.verdict == kGather) {
        gather();
        cluster.sync();
        if (rank != 0) return;                             // CTA 0 has everything that can be kept
        int r = min(sh.listed, kList);
        sort_list(sh.list, r);
        r = min(r, k);
        u64 before[4], m[4];
        const u64 all = scan_list(r, [&](int i) { return mass_of(weight_at(key_in(i))); }, before, m);
        const double limit = top_p < 1.f ? static_cast<double>(top_p) * static_cast<double>(all) : 2.0 * static_cast<double>(all);
        int keep = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = 4 * threadIdx.x + j;
          keep += i < r && (i == 0 || (static_cast<double>(before[j]) < limit && weight_at(key_in(i)) >= min_p));
        }
        r = count_true(keep);                              // the kept ones are a prefix
        // in index order: (index, key) ascending is (~index, key) descending
        for (int i = threadIdx.x; i < r; i += kThreads) {
          const u64 e = sh.list[i];
          sh.list[i] = e << 32 | e >> 32;
        }
        __syncthreads();
        sort_list(sh.list, r);
        auto low_key = [&](int i) { return static_cast<uint32_t>(sh.list[i]); };
        const u64 total = scan_list(r, [&](int i) { return mass_of(weight_at(low_key(i))); }, before, m);
        const double target = static_cast<double>(u) * static_cast<double>(total);
        const bool over = !(target < static_cast<double>(total));   // u >= 1: the last kept token
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = 4 * threadIdx.x + j;
          const u64 end = before[j] + m[j];
          const bool hit = over ? end == total : static_cast<double>(before[j]) <= target && target < static_cast<double>(end);
          if (i < r && m[j] > 0 && hit) write(static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(sh.list[i] >> 32)), low_key(i), total);
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
          const double limit = static_cast<double>(top_p) * static_cast<double>(mass_total);
          const int pb = first_bin([&](int i) { return static_cast<double>(sh.cum_m[i]) >= limit; });
          const uint32_t in = pb < kOver ? sh.cum_c[pb] - below(pb) : 0u;
          tell(p.vocab > kMaxSlice * cs || in > kList ? kBisect : (pb < kOver ? kGather : kReady), pb, pb);
        } else {
          tell(kReady, 0, 0);
        }
      }
      cluster.sync();
      const bool k_first = k < p.vocab;
      if (sh.verdict == kGather) {
        gather();
        cluster.sync();
        if (rank == 0) {
          int bin = sh.bin_lo, r = min(sh.listed, kList);
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
              const double limit = static_cast<double>(top_p) * static_cast<double>(goal_mass);
              const int pb = first_bin([&](int i) { return i >= bin || static_cast<double>(sh.cum_m[i]) >= limit; });
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
              const double limit = static_cast<double>(top_p) * static_cast<double>(goal_mass);
              scan_list(within, [&](int i) { return mass_of(weight_at(key_in(i))); }, before, m);
              int keep = 0;
#pragma unroll
              for (int j = 0; j < 4; ++j)
                keep += 4 * static_cast<int>(threadIdx.x) + j < within && static_cast<double>(before[j] + below_m(bin)) < limit;
              keep = count_true(keep);
              cut_after(keep > 0 ? keep : 1);
            }
            tell(kReady, 0, 0);
          }
        }
        cluster.sync();
        if (sh.verdict == kGather) {                       // the earlier bin
          gather();
          cluster.sync();
          if (rank == 0) {
            const int bin = sh.bin_lo, r = min(sh.listed, kList);
            const double limit = static_cast<double>(top_p) * static_cast<double>(sh.slots[0][0]);
            sort_list(sh.list, r);
            u64 before[4], m[4];
            scan_list(r, [&](int i) { return mass_of(weight_at(key_in(i))); }, before, m);
            int keep = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              keep += 4 * static_cast<int>(threadIdx.x) + j < r && static_cast<double>(before[j] + below_m(bin)) < limit;
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
    if (sh.verdict == kBisect) {
      thr = 0u;
      ties = p.vocab;
      auto key_at = [&](int i) { return key_of(value_at(i)); };
      auto mass_at = [&](uint32_t key) { return key ? mass_of(weight_at(key)) : 0ull; };
      if (k < p.vocab) {
        for (int bit = 31; bit >= 0; --bit) {
          const uint32_t cand = thr | (1u << bit);
          u64 c = 0;
          for (int i = threadIdx.x; i < n; i += kThreads) c += key_at(i) >= cand;
          if (cluster_sum(c) >= static_cast<u64>(k)) thr = cand;
        }
        u64 c = 0;
        for (int i = threadIdx.x; i < n; i += kThreads) c += key_at(i) > thr;
        ties = k - static_cast<int>(cluster_sum(c));
      }
      if (top_p < 1.f) {
        auto above = [&](uint32_t v) {                     // mass of the keys above v
          u64 m = 0;
          for (int i = threadIdx.x; i < n; i += kThreads) {
            const uint32_t key = key_at(i);
            if (key > v) m += mass_at(key);
          }
          return cluster_sum(m);
        };
        u64 at_thr = 0;
        for (int i = threadIdx.x; i < n; i += kThreads) at_thr += key_at(i) == thr;
        at_thr = cluster_sum(at_thr);
        if (at_thr > static_cast<u64>(ties)) at_thr = ties;
        const double limit = static_cast<double>(top_p) * static_cast<double>(above(thr) + at_thr * mass_at(thr));
        // the smallest key v >= thr with less than the limit above it
        uint32_t lo = thr, hi = best;
        while (lo < hi) {
          const uint32_t mid = lo + (hi - lo) / 2;
          if (static_cast<double>(above(mid)) < limit) hi = mid;
          else lo = mid + 1;
        }
        const u64 a = above(lo), m = mass_at(lo);
        int r = lo == thr ? ties : p.vocab;
        if (m > 0) {                                       // ties i = 0, 1, ... stay while a + i m < limit
          u64 q = static_cast<u64>(ceil((limit - static_cast<double>(a)) / static_cast<double>(m)));
          if (q < 1) q = 1;
          if (q < static_cast<u64>(r)) r = static_cast<int>(q);
        }
        thr = lo;
        ties = r;
      }
    }
  }

  // ---- the kept masses in index order: each warp's run of this CTA's tokens, then the CTAs.  Ties have
  // one mass each, so a run needs only the mass above the threshold and its number of ties.
  const int chunks = (n + 127) / 128;                      // a warp's run is whole chunks of 128 tokens
  const int c0 = chunks * warp / kWarps, c1 = chunks * (warp + 1) / kWarps;
  const u64 tie_mass = thr ? kept_mass(thr) : 0ull;
  auto chunk_at = [&](int c, u64 (&m)[4], bool (&tie)[4]) {   // this lane's 4 tokens of chunk c
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = c * 128 + 4 * lane + j;
      const uint32_t key = i < n ? key_of(value_at(i)) : 0u;
      tie[j] = i < n && key == thr;
      m[j] = key > thr ? kept_mass(key) : 0ull;
    }
  };
  {
    u64 mine = 0;
    int t = 0;
    for (int c = c0; c < c1; ++c) {
      u64 m[4];
      bool tie[4];
      chunk_at(c, m, tie);
      mine += (m[0] + m[1]) + (m[2] + m[3]);
      t += tie[0] + tie[1] + tie[2] + tie[3];
    }
    mine = warp_sum(mine);
    t = __reduce_add_sync(0xFFFFFFFFu, t);
    __syncthreads();
    if (lane == 0) {
      sh.warp_m[warp] = mine;
      sh.warp_t[warp] = t;
    }
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < cs) {
      u64 all = 0;
      int ties_here = 0;
      for (int w = 0; w < kWarps; ++w) {
        all += sh.warp_m[w];
        ties_here += sh.warp_t[w];
      }
      Shared* s = cluster.map_shared_rank(&sh, threadIdx.x);
      s->part_m[rank] = all;
      s->part_t[rank] = ties_here;
    }
  }
  cluster.sync();                                          // the last access to another CTA's memory
  u64 before = 0, total = 0;                               // kept mass before this warp's run, in all
  int tied = 0;                                            // ties before this warp's run
  int seen = 0;
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
  for (int w = 0; w < warp; ++w) {
    before += sh.warp_m[w] + static_cast<u64>(kept_ties(tied, sh.warp_t[w])) * tie_mass;
    tied += sh.warp_t[w];
  }
  const u64 end = before + sh.warp_m[warp] + static_cast<u64>(kept_ties(tied, sh.warp_t[warp])) * tie_mass;
  const double target = static_cast<double>(u) * static_cast<double>(total);
  const bool over = !(target < static_cast<double>(total));   // u >= 1: the last kept token
  // the run that holds the target (over: the run whose end is the total, with a mass of its own)
  if (!(over ? end == total && end > before : static_cast<double>(before) <= target && target < static_cast<double>(end))) return;
  for (int c = c0; c < c1; ++c) {
    u64 m[4];
    bool tie[4];
    chunk_at(c, m, tie);
    const int t = tie[0] + tie[1] + tie[2] + tie[3];
    int tscan = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, tscan, o);
      if (lane >= o) tscan += v;
    }
    int at = tied + tscan - t;
    u64 sum = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (tie[j] && at++ < ties) m[j] = tie_mass;
      sum += m[j];
    }
    const u64 incl = warp_scan(sum);
    u64 run = before + incl - sum;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const u64 e = run + m[j];
      const bool hit = over ? e == total : static_cast<double>(run) <= target && target < static_cast<double>(e);
      if (m[j] > 0 && hit) {
        const int i = c * 128 + 4 * lane + j;
        write(start + i, key_of(value_at(i)), total);
      }
      run = e;
    }
    before += __shfl_sync(0xFFFFFFFFu, incl, 31);
    tied += __shfl_sync(0xFFFFFFFFu, tscan, 31);
    if (over ? before == total : target < static_cast<double>(before)) break;
  }
}

template <int DT>
cudaError_t launch(const SampleProblem& p, cudaStream_t stream) {
  constexpr int kSize = DT == 2 ? 4 : 2;
  const DeviceInfo& dev = device_info();
  // CTAs per row: enough to fill the GPU and to hold the row in shared memory with exact histograms
  int cs = 1;
  auto bytes = [&](int c) { return (static_cast<size_t>(p.vocab) / c + 1) * kSize + 16; };
  while (cs < kMaxCluster && (static_cast<long long>(p.batch) * cs < 2 * dev.sm_count || p.vocab > kMaxSlice * cs || bytes(cs) > 96 * 1024) &&
         p.vocab / cs > 2 * kThreads)
    cs *= 2;
  size_t smem = bytes(cs);
  const bool held = smem <= 160 * 1024;
  if (!held) smem = 0;
  auto kern = k_sample<DT>;
  static std::atomic<unsigned long long> opted_in{0};       // per device
  if (dev.device >= 64 || !(opted_in.load(std::memory_order_relaxed) & (1ull << dev.device))) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
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
