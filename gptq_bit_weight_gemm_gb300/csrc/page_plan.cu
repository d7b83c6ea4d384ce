// page_plan.cu -- lengths, rows, positions and slots of a step, and the pages it takes and gives back.
//
// Three sums over the sequences say where everything goes: new tokens (rows), pages given back (places at the
// end of the free list), pages taken (places from its end).  They are whole numbers below 2^31, and
// saturate there: sums of numbers cut to a limit do not depend on the order either.
//
// Bound: latency.  The data are a few bytes a token; the chain is launch - lengths - sums - free list - table.
//
// One cluster of CTAs: each makes the same sums for itself and takes a share of the pages and rows, found back by
// bisection in the sums.  One cluster barrier orders the steps: pages given back before pages taken (the same
// places of the list), and all reading of the inputs before what may be written over them.
#include <limits.h>

#include <atomic>

#include "decode.cuh"
#include "gptq_internal.h"
#include "prompt_internal.h"

namespace gptq {
namespace plan {

constexpr int kThreads = 512, kWarps = kThreads / 32, kCtas = 8, kAll = kThreads * kCtas;

__device__ __forceinline__ unsigned add_sat(unsigned a, unsigned b) { return min(a + b, static_cast<unsigned>(INT_MAX)); }
__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// with release and acquire: global memory written before it is seen after it
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// What becomes of a sequence: tokens before and after (after = -1: it would be longer than the table), new rows.
struct Change {
  int before, after, rows;
};

__device__ __forceinline__ Change change_of(int cached, int added, int most, bool* cut) {
  Change c;
  c.before = cached < 0 ? 0 : min(cached, most);
  *cut = c.before != cached;
  const long long n = static_cast<long long>(c.before) + added;
  c.after = n < 0 ? 0 : (n > most ? -1 : static_cast<int>(n));
  *cut |= n < 0 || n > most;
  c.rows = max(added, 0);
  return c;
}

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads) k_plan(const PlanProblem p) {
  extern __shared__ int sm[];
  int* const before = sm;                       // per sequence: Change, then rows, pages given and taken before it
  int* const after = before + p.batch;
  int* const row0 = after + p.batch;
  int* const give0 = row0 + p.batch;
  int* const take0 = give0 + p.batch;
  __shared__ unsigned warp_sum[3][kWarps];
  __shared__ int granted;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = cluster_rank(), all = rank * kThreads + tid;   // this thread among the cluster's
  decode::pdl_launch_dependents();
  decode::pdl_wait();
  const int most = p.table_width * p.page_size;
  auto pages_of = [&](int n) { return static_cast<int>((static_cast<unsigned>(n) + p.page_size - 1) / p.page_size); };

  // ---- the sums
  const int count_in = *p.free_count, count = min(max(count_in, 0), p.free_capacity);
  unsigned total[3] = {0, 0, 0};
  if (tid == 0) granted = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
    const int b = b0 + tid;
    unsigned own[3] = {0, 0, 0}, sum[3];
    if (b < p.batch) {
      bool cut;
      const Change c = change_of(p.cached[b], p.added[b], most, &cut);
      if (cut && rank == 0) atomicOr(p.status, kStatusSeqLen);
      before[b] = c.before;
      after[b] = c.after;
      const int have = pages_of(c.before), need = c.after < 0 ? have : pages_of(c.after);
      own[0] = c.rows;
      own[1] = max(have - need, 0);
      own[2] = max(need - have, 0);
    }
#pragma unroll
    for (int x = 0; x < 3; ++x) {
      sum[x] = own[x];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned v = __shfl_up_sync(0xFFFFFFFFu, sum[x], o);
        if (lane >= o) sum[x] = add_sat(sum[x], v);
      }
      if (lane == 31) warp_sum[x][warp] = sum[x];
      // the sum before this thread, within its warp
      sum[x] = __shfl_up_sync(0xFFFFFFFFu, sum[x], 1);
      if (lane == 0) sum[x] = 0;
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < 3; ++x) {
      unsigned v = lane < kWarps ? warp_sum[x][lane] : 0;
#pragma unroll
      for (int o = 1; o < kWarps; o <<= 1) {
        const unsigned u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v = add_sat(v, u);
      }
      const unsigned base = __shfl_sync(0xFFFFFFFFu, v, max(warp - 1, 0));
      sum[x] = add_sat(sum[x], add_sat(total[x], warp ? base : 0));
      total[x] = add_sat(total[x], __shfl_sync(0xFFFFFFFFu, v, kWarps - 1));
    }
    if (b < p.batch) {
      row0[b] = sum[0];
      give0[b] = sum[1];
      take0[b] = sum[2];
    }
    __syncthreads();
  }
  const int rows = min(static_cast<int>(total[0]), p.max_tokens);
  const int given = min(static_cast<int>(total[1]), p.free_capacity - count), avail = count + given;
  if (all == 0) {
    if (static_cast<int>(total[0]) > p.max_tokens) atomicOr(p.status, kStatusTokenRows);
    if (count != count_in || given != static_cast<int>(total[1])) atomicOr(p.status, kStatusNoPage);
  }
  // ---- which sequences get their pages: all of them or none, while the list lasts
  for (int b = tid; b < p.batch; b += kThreads) {
    const int take = after[b] < 0 ? 0 : max(pages_of(after[b]) - pages_of(before[b]), 0);
    if (take > 0) {
      if (take > avail - take0[b]) {
        if (rank == 0) atomicOr(p.status, kStatusNoPage);
        after[b] = -1;
      } else {
        atomicMax(&granted, take0[b] + take);
      }
    }
  }
  __syncthreads();
  // the last sequence whose items begin at or before x
  auto owner = [&](const int* first, int x) {
    int lo = 0, hi = p.batch - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= x) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  };
  auto entry = [&](int b, int e) { return p.table + static_cast<long long>(b) * p.table_width + e; };
  // ---- pages back to the list
  for (int g = all; g < given; g += kAll) {
    const int b = owner(give0, g);
    p.free_pages[count + g] = *entry(b, pages_of(after[b]) + g - give0[b]);
  }
  // every CTA has read the inputs, and the pages are on the list
  cluster_barrier();
  // ---- pages from it
  for (int x = all; x < granted; x += kAll) {
    const int b = owner(take0, x);
    *entry(b, pages_of(before[b]) + x - take0[b]) = p.free_pages[avail - 1 - x];
  }
  for (int b = all; b < p.batch; b += kAll) {
    p.seq_lens[b] = after[b] < 0 ? before[b] : after[b];
    p.cu_tokens[b] = min(row0[b], rows);
  }
  if (all == 0) {
    p.cu_tokens[p.batch] = rows;
    *p.free_count_out = avail - granted;
  }
  // ---- rows: a page that this step takes is read from the list, not from the table
  for (int t = all; t < p.max_tokens; t += kAll) {
    int at = 0;
    long long slot = -1;
    if (t < rows) {
      const int b = owner(row0, t);
      at = before[b] + t - row0[b];
      if (after[b] >= 0) {
        const int e = at / p.page_size, have = pages_of(before[b]);
        const int page = e < have ? *entry(b, e) : p.free_pages[avail - 1 - take0[b] - (e - have)];
        slot = static_cast<long long>(page) * p.page_size + (at - e * p.page_size);
      }
    }
    p.positions[t] = at;
    p.slots[t] = slot;
  }
}

}  // namespace plan

cudaError_t launch_page_plan(const PlanProblem& p, cudaStream_t stream) {
  const int smem = p.batch * 5 * 4;
  static std::atomic<unsigned long long> opted_in{0};       // per device
  const int device = device_info().device;
  if (device >= 64 || !(opted_in.load(std::memory_order_relaxed) & (1ull << device))) {
    const cudaError_t e = cudaFuncSetAttribute(plan::k_plan, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxPlanBatch * 5 * 4);
    if (e != cudaSuccess) return e;
    if (device < 64) opted_in.fetch_or(1ull << device, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(plan::kCtas);
  cfg.blockDim = dim3(plan::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, plan::k_plan, p);
}

}  // namespace gptq
