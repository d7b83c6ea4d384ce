// chunk_attention.cuh -- causal attention of each sequence's new tokens over its paged keys and values:
//   out = sum_j p_j v_j,  p = softmax_j(scale q . k_j),  over the keys j in [max(0, t - window + 1), t] of the
// row at position t.
//
// One pass over the keys: with the maximum m, the sum l and the accumulator o of the keys so far, a block of scores
// s moves them to  m' = max(m, max s),  l' = l e^(m - m') + sum e^(s - m'),  o' = o e^(m - m') + e^(s - m') v,
// and two partial results of disjoint keys join the same way.
//
// Bound: 4 flops per visible key, query head and dimension on the tensor cores, for chunks of some hundred rows and
// more; the cache's bytes for fewer.
//
// Rows: the query heads that share a key head read the same keys, so the rows of an item are the pairs (token,
// head of the group), 256 of them (128 for head_dim above 128) for one sequence and kv head: two
// accumulators of 128 rows that share every tile of keys and values.
//
// Split: items cost what their visible key tiles cost, from 1 to thousands.  All of them, one after the
// other, are a line of key tiles that is cut into as many equal runs as there are SMs, on the device, from the
// lengths; an item cut by a run's end leaves partial results (m, l, o) in the workspace, two a run at most, and a
// second kernel joins them, all SMs at work on the rows.  Where there are many items and the last ones are small they
// are dealt out whole instead.
//
// A CTA: softmax warps 0-3 and 4-7 (one accumulator each, a thread a row), loader warps 8-11, and in the last
// four one that issues the MMAs, one that walks the line and two that look over values.  S = q k^T goes to
// tensor memory; a softmax thread reads its row, writes the probabilities back over it as 16-bit values, and
// these are the A operand of p v straight from tensor memory, in two halves of the keys so that the product
// of the first begins while the second is made.  While one accumulator's softmax runs, the tensor cores work
// for the other.  The accumulator o is rescaled by the softmax threads themselves, only where a row's
// maximum has grown by more than 2^8 since the last time: until then probabilities are simply larger than
// 1 (the scores' MMA completes after the p v before it, so o is at rest then).
//
// Rounding: a probability enters the product as one value of the cache's type (11 significant bits in fp16, 8 in bf16),
// once; together with the rounding of the result the error against 64 bits is 1.4 times that of the rounding alone
// (bf16 2.3e-3 against 1.7e-3, fp16 2.6e-4 against 2.0e-4; the attention of single tokens carries them in two values, whose
// products it has to spare).  As a sum of two values it would be the rounding alone, for
// half as many MMAs again and more softmax instructions: 4096 tokens on 32768 keys took 2.8 ms so, against 1.34.
// fp16 probabilities are taken 2^7 times as large, so that a long flat tail behind one large score is not lost
// in fp16's range.
//
// Keys, values and queries come as TMA boxes of 64 dimensions by the keys that divide a page (8 to 32).  Pages that 8
// does not divide, and caches whose strides a tensor map does not take, are copied by cp.async, 16 bytes a lane.  cp.async
// alone reached 870 TFLOP/s on the case above, at 64 KB a tile its issue and the lanes' waiting for it was the bound.
//
// Values that some row of the item must not see (later tokens', outside the window) could reach it as 0 x NaN:
// in the tiles that not every row sees, infinite and NaN values are replaced by 0 (and those of keys that no row sees,
// which may never have been written), and the rows that do see them get them added at the end.  In the tiles that
// every row sees they go through the MMAs, where a probability too small for 16 bits makes 0 x inf of them: a row whose
// result is not finite looks these values up again, and takes their own sum.  The join keeps its factors above 0.
// (The look at each result costs 1 % at most: four prompts 227 -> 229 us, a mixed batch 108 -> 110.)
//
// What the steps brought, us for 4096 tokens on 32768 keys (32 query and 8 kv heads of 128, bf16) / four prompts of 1300 to
// 4096 tokens (32 kv heads, fp16) / a mixed batch of 16: a warp a row 619708 / 59324 / 21621; tcgen05 3019 / 465 / 179;
// no spills 2334 / 394 / 148; copies handed on as they land, P in halves, 128-byte blocks 2000 / 396 / 152; MMAs issued by
// a converged warp (a lone thread's descriptors go through vector registers: 125 cycles an MMA, against 64 of the
// tensor cores) 1648 / 335 / 135; TMA boxes, tiles at the diagonal looked over by two warps 1391 / 330 / 117; results in
// 64-byte pieces 1330 / 331 / 111; items dealt out whole 1330 / 228 / 112; joins two parts at a time, the table past the
// first-level cache 1345 / 227 / 109; the scores' MMAs unrolled for more head_dims 1315 / 225 / 106; infinite values looked up again
// 1340 / 229 / 109; the MMA sequence chosen before the loop over the tiles 1285 / 224 / 104 (1430 to 1480 us for the first where
// calls follow one another for long: 1.37 kW, and clocks that go by it).
#pragma once

#include <cuda.h>
#include <limits.h>
#include <math_constants.h>

#include <atomic>
#include <type_traits>

#include "chunk_ptx.cuh"
#include "decode.cuh"
#include "gptq_device.cuh"
#include "gptq_internal.h"
#include "prompt_internal.h"

namespace gptq {
namespace chunk {

constexpr int kMaxRuns = 160;            // CTAs, at most: one on each of the 152 SMs
constexpr size_t kRecordBytes = kMaxRuns * 32;
constexpr uint64_t kDrainLimitNs = 2000000000ull;   // for what is in flight when a wait has given up
constexpr float kGrow = 8.f;             // log2 of what a row's maximum may grow by before o is rescaled
// An item counts as its tiles and kItemUnits more: opening and closing it.
constexpr int kItemUnits = 3;
constexpr int kMinShare = 2;             // units of a run, at least

template <typename T>
__host__ __device__ constexpr float lift() { return std::is_same<T, __half>::value ? 7.f : 0.f; }

// Dimensions padded to DP (64, 128, 256).
template <int DP>
struct Shape {
  static constexpr int kNQ = DP == 256 ? 1 : 2;            // accumulators of 128 rows
  static constexpr int kRows = kNQ * 128;
  static constexpr int kKeys = DP == 256 ? 64 : 128;       // of a tile
  static constexpr int kStages = DP == 64 ? 8 : 5;         // tiles of keys or values in flight
  static constexpr int kAhead = kStages - 2;               // loads left open behind the last one issued (6 at most)
  static constexpr int kThreads = (kNQ + 2) * 128;
  static constexpr int kLoadWarp0 = kNQ * 4, kMmaWarp = kLoadWarp0 + 4, kWalkWarp = kMmaWarp + 1, kLookWarp0 = kMmaWarp + 2;
  static constexpr uint32_t kQBytes = 128 * DP * 2;        // queries of one accumulator
  static constexpr uint32_t kTileBytes = kKeys * DP * 2;
  static constexpr uint32_t kOffKV = kNQ * kQBytes;
  static constexpr uint32_t kOffControl = kOffKV + kStages * kTileBytes;
};

// One item's part in a run.
struct Item {
  int kv_head;
  int first;               // row of the sequence's first new token
  int row0, rows;          // first packed row (token * group + head), live rows from there
  int position0;           // position of the sequence's first new token
  int b, key_lo, key_hi;   // keys any of its rows sees
  int t0, t1;              // tiles of this run
  int lo[2], hi[2];        // of them, those that each accumulator takes part in
  int full_lo, full_hi;    // keys that every row sees
  int slot;                // -1: the run holds all of the item; else where its partial goes
  int bad;                 // an infinite or NaN value was replaced by 0 in a tile not seen by every row
};

struct Sequence {
  int first, tokens, n, blocks;    // its rows, keys, blocks of packed rows
};

template <int DP>
struct Control {
  unsigned long long full[Shape<DP>::kStages], empty[Shape<DP>::kStages], raw[Shape<DP>::kStages];
  unsigned long long qfull, qempty, sfull[2], pready[2][2], ofull[2], ifull[2], iempty[2], drain;
  uint32_t valid[16][4];   // per tile: keys whose page could be read
  Item item[2];
  uint32_t tmem;
  int abort;
  int sequence;            // that the run begins in, what it is, units before it and of each of its kv heads
  Sequence found;
  long long at, total;
  long long sum[Shape<DP>::kThreads / 32];
};

// What is left of a cut item for the joining kernel, by the run that holds the item's first tile.
struct alignas(16) Record {
  int valid, first_run, last_run, kv_head, first, row0, rows, pad;
};

struct Args {
  ChunkProblem p;
  int group;
  float scale_log2;        // |scale| * log2(e)
  int negative;            // scale < 0
  unsigned page_mul, page_shift;   // key / page_size = key * page_mul >> page_shift for keys below 2^30
  unsigned group_mul, group_shift; // and packed rows by the group's heads
  unsigned k_page16, k_slot16, k_head16, v_page16, v_slot16, v_head16;   // strides in 16-byte units
  int box_rows;            // keys of a TMA box: 0 where the cache is not read by TMA
  int box_order[3];        // which coordinate is the box's second, third and fourth: 0 slot, 1 head, 2 page
  int q_boxes;             // queries come as boxes of 128 / group tokens with the heads of a group
  Record* records;
  float* partials;
};

// floats of one partial: accumulators [column / 4][row][4], then m and l per row
template <int DP>
__host__ __device__ constexpr size_t partial_floats() { return static_cast<size_t>(Shape<DP>::kRows) * (DP + 2); }

// ------------------------------------------------------------------------------ small pieces
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {   // (of a NaN and numbers, the numbers)
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// x * s + c of two values at a time
__device__ __forceinline__ void fma2(float& a, float& b, float s, float c) {
  uint64_t d;
  const uint64_t x = (static_cast<uint64_t>(__float_as_uint(b)) << 32) | __float_as_uint(a);
  const uint64_t y = (static_cast<uint64_t>(__float_as_uint(s)) << 32) | __float_as_uint(s);
  const uint64_t z = (static_cast<uint64_t>(__float_as_uint(c)) << 32) | __float_as_uint(c);
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
  a = __uint_as_float(static_cast<uint32_t>(d));
  b = __uint_as_float(static_cast<uint32_t>(d >> 32));
}
__device__ __forceinline__ float2 add2(float2 s, float a, float b) {
  uint64_t d;
  const uint64_t x = (static_cast<uint64_t>(__float_as_uint(s.y)) << 32) | __float_as_uint(s.x);
  const uint64_t y = (static_cast<uint64_t>(__float_as_uint(b)) << 32) | __float_as_uint(a);
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
  return make_float2(__uint_as_float(static_cast<uint32_t>(d)), __uint_as_float(static_cast<uint32_t>(d >> 32)));
}
// c + 0 of two values: a NaN where one is not finite
__device__ __forceinline__ void odd2(float (&c)[2], float a, float b) {
  uint64_t d;
  const uint64_t x = (static_cast<uint64_t>(__float_as_uint(b)) << 32) | __float_as_uint(a);
  const uint64_t z = (static_cast<uint64_t>(__float_as_uint(c[1])) << 32) | __float_as_uint(c[0]);
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(0ull), "l"(z));
  c[0] = __uint_as_float(static_cast<uint32_t>(d));
  c[1] = __uint_as_float(static_cast<uint32_t>(d >> 32));
}
template <int N>
__device__ __forceinline__ void grow_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void shrink_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Bounded wait on an mbarrier phase; false if the wait ran out or another role gave up.  All lanes agree.
__device__ __forceinline__ bool wait_one(uint32_t bar, uint32_t parity, volatile int* abort, const ChunkProblem& p) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint32_t t0 = static_cast<uint32_t>(ptx::globaltimer());   // (limits are below 2^32 ns, and 64 bits cost registers)
  while (true) {
    if (ptx::mbar_try_wait_hint(bar, parity, min(p.wait_ns, 200000u))) return true;
    if (*abort) return false;
    if (static_cast<uint32_t>(ptx::globaltimer()) - t0 > p.wait_ns) {
      *abort = 1;
      atomicOr(p.status, kStatusTimeout);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort, const ChunkProblem& p) {
  return __all_sync(0xFFFFFFFFu, wait_one(bar, parity, abort, p));
}

// x / y of nonnegative numbers: mostly they fit 32 bits
__device__ __forceinline__ long long divide(long long x, long long y) {
  if (((x | y) >> 32) == 0) return static_cast<unsigned>(x) / static_cast<unsigned>(y);
  return x / y;
}

// The token of a packed row (a division costs some 200 cycles, and an item takes a dozen).
__device__ __forceinline__ int token_of(const Args& a, int row) {
  return static_cast<int>(static_cast<unsigned long long>(static_cast<unsigned>(max(row, 0))) * a.group_mul >> a.group_shift);
}

// ------------------------------------------------------------------------------ the line
template <int DP>
__device__ __forceinline__ Sequence sequence_of(const Args& a, int b, bool report) {
  const ChunkProblem& p = a.p;
  Sequence s;
  const int c0 = p.cu[b], c1 = p.cu[b + 1], raw = p.lens[b], most = p.table_width * p.page_size;
  s.first = min(max(c0, 0), p.tokens);
  const int end = max(s.first, min(c1, p.tokens));
  s.tokens = end - s.first;
  s.n = min(max(raw, 0), most);
  s.blocks = (s.tokens * a.group + Shape<DP>::kRows - 1) / Shape<DP>::kRows;
  if (report) {
    if (s.first != c0 || end != c1) atomicOr(p.status, kStatusTokenRows);
    if (s.n != raw) atomicOr(p.status, kStatusSeqLen);
  }
  return s;
}

// Keys [lo, hi) that the packed rows r0 .. r1 of a sequence see.
__device__ __forceinline__ void keys_of(const Args& a, const Sequence& s, int r0, int r1, int* lo, int* hi) {
  const int position0 = s.n - s.tokens;
  *hi = max(0, position0 + token_of(a, r1) + 1);
  *lo = a.p.window > 0 ? max(0, position0 + token_of(a, r0) - a.p.window + 1) : 0;
}

template <int DP>
__device__ __forceinline__ int units_of(const Args& a, const Sequence& s, int block) {
  using S = Shape<DP>;
  const int r0 = block * S::kRows, r1 = min(r0 + S::kRows, s.tokens * a.group) - 1;
  int lo, hi;
  keys_of(a, s, r0, r1, &lo, &hi);
  const int tiles = hi > lo ? (hi + S::kKeys - 1) / S::kKeys - lo / S::kKeys : 0;
  return kItemUnits + max(tiles, 1);       // (an item without keys still writes its zeros)
}

// Units of one kv head's items of each lane's sequence; sequences of many blocks are summed by the warp.
template <int DP>
__device__ __forceinline__ long long head_units(const Args& a, const Sequence& s, int lane) {
  long long sum = 0;
  if (s.blocks <= 4)
    for (int i = 0; i < s.blocks; ++i) sum += units_of<DP>(a, s, i);
  unsigned many = __ballot_sync(0xFFFFFFFFu, s.blocks > 4);
  while (many) {
    const int from = __ffs(many) - 1;
    many &= many - 1;
    Sequence o;
    o.first = __shfl_sync(0xFFFFFFFFu, s.first, from);
    o.tokens = __shfl_sync(0xFFFFFFFFu, s.tokens, from);
    o.n = __shfl_sync(0xFFFFFFFFu, s.n, from);
    o.blocks = __shfl_sync(0xFFFFFFFFu, s.blocks, from);
    long long part = 0;
    for (int i = lane; i < o.blocks; i += 32) part += units_of<DP>(a, o, i);
#pragma unroll
    for (int x = 16; x; x >>= 1) part += __shfl_xor_sync(0xFFFFFFFFu, part, x);
    if (lane == from) sum = part;
  }
  return sum;
}

// ------------------------------------------------------------------------------ the kernel
template <typename T, int DP>
__global__ void __launch_bounds__(Shape<DP>::kThreads, 1) k_chunk(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                                                              const __grid_constant__ CUtensorMap map_q, const __grid_constant__ Args a) {
  using S = Shape<DP>;
  using C = Control<DP>;
  using Tr = F16Traits<T>;
  constexpr int kKeys = S::kKeys, kNQ = S::kNQ;
  const ChunkProblem& p = a.p;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                         ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = ptx::smem_addr(smem);
  C& c = *reinterpret_cast<C*>(smem + S::kOffControl);
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31, run = blockIdx.x;

  decode::pdl_launch_dependents();
  if (warp == S::kLoadWarp0 && lane == 0) {
    if (a.box_rows) {                      // (the others hold nothing)
      ptx::prefetch_tmap(&map_k);
      ptx::prefetch_tmap(&map_v);
    }
    if (a.q_boxes) ptx::prefetch_tmap(&map_q);
  }
  decode::pdl_wait();

  // ---- this CTA's run of the line: a scan over the sequences gives its length, and the sequence that the run
  // begins in
  long long before = 0, upto = 0, units = 0;
  Sequence s = {0, 0, 0, 0};
  auto scan_chunk = [&](int b0, long long base) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    s = {0, 0, 0, 0};
    if (b < p.batch) s = sequence_of<DP>(a, b, run == 0);
    units = head_units<DP>(a, s, lane);
    const long long w = units * p.kv_heads;
    long long x = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += v;
    }
    __syncthreads();                       // what the chunk before left has been read
    if (lane == 31) c.sum[warp] = x;
    if (threadIdx.x == 0) c.sequence = -1;
    __syncthreads();
    long long all = base;
    for (int i = 0; i < S::kThreads / 32; ++i) {
      if (i < warp) x += c.sum[i];
      all += c.sum[i];
    }
    upto = base + x;
    before = upto - w;
    return all;
  };
  long long total = 0;
  for (int b0 = 0; b0 < p.batch; b0 += S::kThreads) total = scan_chunk(b0, total);
  const long long most = total >= kMinShare ? divide(total, kMinShare) : 1;
  const int runs = most < static_cast<long long>(gridDim.x) ? static_cast<int>(most) : static_cast<int>(gridDim.x);
  // runs of `share` units, the first `extra` of them one longer
  const long long share = divide(total, runs), extra = total - share * runs;
  const long long begin = share * run + (run < extra ? run : extra), end = begin + share + (run < extra ? 1 : 0);
  // Or no item is cut: they are dealt out whole, in turns that go to and fro through the CTAs, those of a sequence with the most
  // keys first and its kv heads side by side.  All CTAs then read the same sequence at about the same time and place, so its
  // keys come from DRAM once, in whole rows (of runs each reads a head and a sequence of its own: four prompts of 1300 to
  // 4096 tokens and 32 kv heads took 331 us so, 232 dealt).  That asks for enough items, of which the last ones are small:
  // each sequence's largest at most 1.25 times what each CTA has left from it on, and the last sequence's smallest at
  // most 0.06 of a CTA's work (either with 0.06 of slack).
  bool deal = false;
  if (p.batch <= S::kThreads) {
    bool good = true;
    if (s.blocks > 0) {
      const long long ctas = gridDim.x, rest = total - before;
      good = units_of<DP>(a, s, s.blocks - 1) * ctas * 100 <= rest * 125 + total * 6 &&
             (upto < total || units_of<DP>(a, s, 0) * ctas * 100 <= total * 6);
    }
    deal = __syncthreads_and(good) && total > 0;
  }
  if (!deal && run < runs && total > 0) {
    long long at = 0;
    for (int b0 = 0; b0 < p.batch; b0 += S::kThreads) {
      if (p.batch > S::kThreads) at = scan_chunk(b0, at);
      if (before <= begin && begin < upto) {
        c.sequence = b0 + static_cast<int>(threadIdx.x);
        c.found = s;
        c.at = before;
        c.total = units;
      }
      __syncthreads();
      if (c.sequence >= 0) break;
    }
  }
  if (!deal && (run >= runs || total == 0 || c.sequence < 0)) {   // (the last: lengths written while this ran)
    if (threadIdx.x == 0) a.records[run].valid = 0;
    return;
  }

  // ---- set up
  if (threadIdx.x == 0) {
    auto init = [&](unsigned long long& bar, int count) { ptx::mbar_init(ptx::smem_addr(&bar), count); };
    for (int i = 0; i < S::kStages; ++i) init(c.full[i], 4), init(c.empty[i], 1), init(c.raw[i], 4);
    init(c.qfull, 4);
    init(c.qempty, 1);
    for (int i = 0; i < 2; ++i) {
      init(c.sfull[i], 1);
      init(c.pready[i][0], 4);
      init(c.pready[i][1], 4);
      init(c.ofull[i], 1);
      init(c.ifull[i], 1);
      init(c.iempty[i], 4 * kNQ + 7);      // softmax, loader and look warps, the MMA warp
    }
    init(c.drain, 1);
    c.abort = 0;
    ptx::fence_mbar_init();
  }
  if (p.head_dim % 16) {                   // the MMAs read 16 dimensions at a time: those past head_dim stay zero
    for (uint32_t i = threadIdx.x * 16; i < S::kOffControl; i += S::kThreads * 16)
      *reinterpret_cast<uint4*>(smem + i) = make_uint4(0u, 0u, 0u, 0u);
    ptx::fence_proxy_async_smem();
  }
  if (warp == S::kMmaWarp) {
    ptx::tmem_alloc(ptx::smem_addr(&c.tmem), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, c.tmem, 0);
  volatile int* const abort = &c.abort;
  auto bar = [&](unsigned long long& b) { return ptx::smem_addr(&b); };
  auto wait = [&](unsigned long long& b, uint32_t parity) { return wait_warp(bar(b), parity, abort, p); };
  auto s_col = [&](int s) { return tmem + s * 128; };
  auto o_col = [&](int s) { return tmem + 256 + s * DP; };

  if (warp >= S::kMmaWarp) {
    if constexpr (kNQ == 2) shrink_registers<80>();
    if (warp == S::kWalkWarp) {
      // -------------------------------------------------------------- the line's items, one after the other
      int b = c.sequence, h = 0, block = 0;
      Sequence s = c.found;
      long long start = 0, first_unit = begin, end_unit = end;   // the item's first unit; those of the run
      if (deal) {
        first_unit = 0;
        end_unit = LLONG_MAX;
      } else {
        const long long rel = begin - c.at;
        h = static_cast<int>(divide(rel, c.total));
        long long left = rel - h * c.total;                // units of the head's items before the run
        // the block whose units hold it: a warp's scan at a time
        for (int b0 = 0;; b0 += 32) {
          const int u = b0 + lane < s.blocks ? units_of<DP>(a, s, b0 + lane) : 0;
          int x = u;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += v;
          }
          const unsigned past = __ballot_sync(0xFFFFFFFFu, x > left);
          if (past || b0 + 32 >= s.blocks) {
            const int i = past ? __ffs(past) - 1 : 31;
            block = min(b0 + i, s.blocks - 1);
            left -= __shfl_sync(0xFFFFFFFFu, x - u, i);
            break;
          }
          left -= __shfl_sync(0xFFFFFFFFu, x, 31);
        }
        start = begin - left;
      }
      // dealt items: 32 sequences at a time, a lane each, with the items before them
      Sequence mine = {0, 0, 0, 0};
      int turn = 0, chunk0 = -32, chunk_items = 0, upto_items = 0;
      long long base = 0;
      auto deal_next = [&]() {             // the item of this CTA's next turn; false: there is none
        const long long index = static_cast<long long>(turn) * gridDim.x + (turn & 1 ? gridDim.x - 1 - run : run);
        ++turn;
        while (index - base >= chunk_items) {
          base += chunk_items;
          chunk0 += 32;
          if (chunk0 >= p.batch) return false;
          mine = {0, 0, 0, 0};
          if (chunk0 + lane < p.batch) mine = sequence_of<DP>(a, chunk0 + lane, false);
          upto_items = mine.blocks * p.kv_heads;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, upto_items, o);
            if (lane >= o) upto_items += v;
          }
          chunk_items = __shfl_sync(0xFFFFFFFFu, upto_items, 31);
        }
        const int within = static_cast<int>(index - base);
        const int from = __ffs(__ballot_sync(0xFFFFFFFFu, upto_items > within)) - 1;
        b = chunk0 + from;
        s.first = __shfl_sync(0xFFFFFFFFu, mine.first, from);
        s.tokens = __shfl_sync(0xFFFFFFFFu, mine.tokens, from);
        s.n = __shfl_sync(0xFFFFFFFFu, mine.n, from);
        s.blocks = __shfl_sync(0xFFFFFFFFu, mine.blocks, from);
        const int item = within - (__shfl_sync(0xFFFFFFFFu, upto_items, from) - s.blocks * p.kv_heads);
        block = s.blocks - 1 - item / p.kv_heads;
        h = item % p.kv_heads;
        return true;
      };
      auto run_of = [&](long long unit) {
        const long long cut = extra * (share + 1);
        return static_cast<int>(unit < cut ? divide(unit, share + 1) : extra + divide(unit - cut, share));
      };
      Record record = {};
      uint32_t n = 0;                      // items handed out
      while (true) {
        const bool out = deal && !deal_next();
        const int u = out ? 0 : units_of<DP>(a, s, block);
        const long long tile0 = start + kItemUnits, stop = start + u;
        const bool done = out || tile0 >= end_unit;
        const int slot = n & 1;
        if (!wait(c.iempty[slot], ((n >> 1) & 1) ^ 1)) break;
        Item it;
        it.b = done ? -1 : b;
        if (!done) {
          const int r0 = block * S::kRows, r1 = min(r0 + S::kRows, s.tokens * a.group) - 1;
          it.kv_head = h;
          it.first = s.first;
          it.row0 = r0;
          it.rows = r1 - r0 + 1;
          it.position0 = s.n - s.tokens;
          keys_of(a, s, r0, r1, &it.key_lo, &it.key_hi);
          int x, y;
          keys_of(a, s, r0, r0, &x, &it.full_hi);
          keys_of(a, s, r1, r1, &it.full_lo, &y);
          const bool any = it.key_hi > it.key_lo;
          const int t_lo = it.key_lo / kKeys;
          const long long from = tile0 > first_unit ? 0 : first_unit - tile0, to = (stop < end_unit ? stop : end_unit) - tile0;
          it.t0 = any ? t_lo + static_cast<int>(from) : 0;
          it.t1 = any ? t_lo + static_cast<int>(to) : 0;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            it.lo[q] = it.hi[q] = 0;
            if (q < kNQ && r0 + q * 128 <= r1) {
              keys_of(a, s, r0 + q * 128, min(r0 + q * 128 + 127, r1), &x, &y);
              if (y > x) {
                it.lo[q] = max(x / kKeys, it.t0);
                it.hi[q] = min((y + kKeys - 1) / kKeys, it.t1);
              }
            }
          }
          const bool whole = tile0 >= first_unit && stop <= end_unit;
          const int first_run = whole ? run : run_of(tile0);
          it.slot = whole ? -1 : 2 * run + (first_run == run ? 1 : 0);
          it.bad = 0;
          if (!whole && first_run == run)
            record = {1, first_run, run_of(stop - 1), h, s.first, r0, it.rows, 0};
        }
        if (lane == 0) {
          c.item[slot] = it;
          ptx::mbar_arrive(bar(c.ifull[slot]));
        }
        __syncwarp();
        if (done) break;
        ++n;
        if (deal) continue;
        start = stop;
        if (++block >= s.blocks) {
          block = 0;
          if (++h == p.kv_heads) {
            h = 0;
            do {
              if (++b >= p.batch) break;
              s = sequence_of<DP>(a, b, false);
            } while (s.blocks == 0);
            if (b >= p.batch) {            // the line's end: nothing follows
              b = p.batch - 1;
              start = end_unit;
            }
          }
        }
      }
      if (lane == 0) a.records[run] = record;
    } else if (warp == S::kMmaWarp) {
      // -------------------------------------------------------------- MMAs
      const int kd = (p.head_dim + 15) / 16;
      constexpr uint32_t type = std::is_same<T, __half>::value ? 0u : 1u;
      // a negative scale is that of -q
      const uint32_t idesc_s = ptx::umma_idesc_f16(type, 128u, kKeys) | (a.negative ? ptx::kUmmaNegateA : 0u);
      const uint32_t idesc_o = ptx::umma_idesc_f16(type, 128u, kd * 16u) | ptx::kUmmaBMajorMN;
      const uint32_t leader = ptx::elect_one();
      auto commit = [&](unsigned long long& b) { ptx::umma_commit_by(leader, bar(b)); };
      int stage = 0;
      uint32_t phase = 0, items = 0, queries = 0, p_phase[2] = {0, 0};
      bool ok = true;
      // Descriptors hold addresses in units of 16 bytes in their lowest bits: a step is an addition of a constant.
      const uint64_t q_desc = ptx::umma_desc_sw128_kmajor(sbase), k_desc = ptx::umma_desc_sw128_kmajor(sbase + S::kOffKV);
      const uint64_t v_desc = ptx::umma_desc_sw128_mnmajor(sbase + S::kOffKV, kKeys * 128);
      auto scores = [&](int s, int at, auto steps) {       // S[s] = q[s] k^T
        const uint64_t qd = q_desc + s * (S::kQBytes >> 4), kt = k_desc + at * (S::kTileBytes >> 4);
        auto step = [&](int k) {
          ptx::umma_f16_by(leader, s_col(s), qd + ((k >> 2) * 128 * 128 + (k & 3) * 32) / 16,
                           kt + ((k >> 2) * kKeys * 128 + (k & 3) * 32) / 16, idesc_s, k != 0);
        };
        if constexpr (steps.value > 0) {
#pragma unroll
          for (int k = 0; k < steps.value; ++k) step(k);
        } else {
#pragma unroll 1
          for (int k = 0; k < kd; ++k) step(k);
        }
        commit(c.sfull[s]);
      };
      auto values = [&](int s, int at, int half, bool more) {   // O[s] (+)= p[s] v, over half of the tile's keys
        const uint64_t vt = v_desc + at * (S::kTileBytes >> 4) + half * (kKeys / 32) * (2048 / 16);
        const uint32_t pt = s_col(s) + half * (kKeys / 4);
#pragma unroll
        for (int k = 0; k < kKeys / 32; ++k)
          ptx::umma_f16_ta_by(leader, o_col(s), pt + k * 8, vt + k * (2048 / 16), idesc_o, more || k != 0);
      };
      auto next_stage = [&]() {
        if (++stage == S::kStages) stage = 0, phase ^= 1;
      };
      // All items; a scores' product takes `steps` MMAs, as many as kd says where that is 0.  One sequence of MMAs stands in
      // the loop over the tiles, chosen before it.
      auto products = [&](auto steps) {
        while (ok) {
          const int slot = items & 1;
          if (!wait(c.ifull[slot], (items >> 1) & 1)) { ok = false; break; }
          ++items;
          const Item& from = c.item[slot];
          if (from.b < 0) break;
          struct { int t0, t1, lo[2], hi[2]; } it = {from.t0, from.t1, {from.lo[0], from.lo[1]}, {from.hi[0], from.hi[1]}};
          __syncwarp();
          if (leader) ptx::mbar_arrive(bar(c.iempty[slot]));
          if (it.t0 >= it.t1) continue;
          auto live = [&](int s, int t) { return s < kNQ && t >= it.lo[s] && t < it.hi[s]; };
          if (!wait(c.qfull, queries & 1)) { ok = false; break; }
          ++queries;
          // the first tile's scores; from then on p v of a tile, then the scores of the next, accumulator by accumulator
          if (!wait(c.full[stage], phase)) { ok = false; break; }
          ptx::tc_fence_after();
#pragma unroll
          for (int s = 0; s < kNQ; ++s)
            if (live(s, it.t0)) scores(s, stage, steps);
          commit(c.empty[stage]);
          if (it.t0 + 1 == it.t1) commit(c.qempty);
          next_stage();
          for (int t = it.t0; t < it.t1; ++t) {
            const int v_stage = stage;
            if (!wait(c.full[stage], phase)) { ok = false; break; }
            next_stage();
            bool have_k = false;
#pragma unroll
            for (int s = 0; s < kNQ; ++s) {
              if (live(s, t)) {
                if (!wait(c.pready[s][0], p_phase[s])) { ok = false; break; }
                ptx::tc_fence_after();
                values(s, v_stage, 0, t > it.lo[s]);
                if (!wait(c.pready[s][1], p_phase[s])) { ok = false; break; }
                p_phase[s] ^= 1;
                ptx::tc_fence_after();
                values(s, v_stage, 1, true);
                if (t + 1 == it.hi[s]) commit(c.ofull[s]);
              }
              if (live(s, t + 1)) {
                if (!have_k) {
                  if (!wait(c.full[stage], phase)) { ok = false; break; }
                  ptx::tc_fence_after();
                  have_k = true;
                }
                scores(s, stage, steps);
              }
            }
            if (!ok) break;
            commit(c.empty[v_stage]);
            if (t + 1 < it.t1) {
              if (!have_k && !wait(c.full[stage], phase)) { ok = false; break; }
              commit(c.empty[stage]);
              if (t + 2 == it.t1) commit(c.qempty);
              next_stage();
            }
          }
        }
      };
      // (Unrolled where head_dim fills DP, and in a DP of 128 always: a loop makes its descriptors anew for each MMA.
      // 4096 tokens on 28672, 32 heads of 8 caches: at 112 1270-1390 us against 1470-1500 in the loop, at 104 1335
      // against 1495, at 96 1271 against 1391.  At a DP of 64 unrolled forms for the smaller head_dims cost 7 %, at
      // 256 they changed nothing.  Chosen here and not within the tiles' loop: at 128 1283 us against 1308, at 80
      // 1225 against 1319, at 64 1224 against 1246, at 256 990 against 982, a mixed batch 103.5 against 108.)
      if (kd == DP / 16) {
        products(std::integral_constant<int, DP / 16>());
      } else if constexpr (DP == 128) {
        if (kd == 7) products(std::integral_constant<int, 7>());
        else if (kd == 6) products(std::integral_constant<int, 6>());
        else products(std::integral_constant<int, 5>());   // (head_dim is above 64)
      } else {
        products(std::integral_constant<int, 0>());
      }
      if (!ok) {
        // wait (bounded) for the MMAs already issued before tensor memory is released
        commit(c.drain);
        const uint64_t t0 = ptx::globaltimer();
        while (!ptx::mbar_try_wait(bar(c.drain), 0) && ptx::globaltimer() - t0 < kDrainLimitNs) {}
        __syncwarp();
      }
    } else if (warp >= S::kLookWarp0) {
      // -------------------------------------------------------------- values that not every row sees
      // Those of a key that no row sees leave, and so does what is not finite; then the tile is the MMA's.
      int stage = 0;
      uint32_t items = 0, raw_phase = 0;
      bool ok = true;
      while (ok) {
        const int slot = items & 1;
        if (!wait(c.ifull[slot], (items >> 1) & 1)) break;
        ++items;
        const Item& from = c.item[slot];
        const struct { int b, key_lo, key_hi, t0, t1, full_lo, full_hi; } it = {from.b, from.key_lo, from.key_hi, from.t0, from.t1,
                                                                               from.full_lo, from.full_hi};
        if (it.b < 0) break;
        for (int t = it.t0; ok && t < it.t1; ++t) {
          if (++stage == S::kStages) stage = 0;            // past the keys
          const bool full = t * kKeys >= it.full_lo && (t + 1) * kKeys <= it.full_hi;
          if (a.box_rows && !full) {
            if (!wait(c.raw[stage], raw_phase >> stage & 1)) { ok = false; break; }
            raw_phase ^= 1u << stage;
            unsigned bad = 0;
            // 16 bytes a lane, as they lie: a row's pieces are swizzled within its 128 bytes
            const int pieces = kKeys * ((p.head_dim + 63) / 64) / 8;
            unsigned char* tile = smem + S::kOffKV + stage * S::kTileBytes;
#pragma unroll 4
            for (int i = 0; i < pieces; ++i) {
              const int at = (i * 64 + (warp - S::kLookWarp0) * 32 + lane) * 16;
              const int key = t * kKeys + at / 128 % kKeys;
              uint4* v = reinterpret_cast<uint4*>(tile + at);
              uint4 x = *v;
              constexpr uint32_t kExp = std::is_same<T, __half>::value ? 0x7C007C00u : 0x7F807F80u;
              unsigned here = 0;
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const uint32_t hit = __vcmpeq2((&x.x)[w] & kExp, kExp);
                (&x.x)[w] &= ~hit;
                here |= hit;
              }
              if (key < it.key_lo || key >= it.key_hi) {
                *v = make_uint4(0u, 0u, 0u, 0u);
              } else if (here) {
                *v = x;
                bad = 1;
              }
            }
            if (bad) *const_cast<volatile int*>(&c.item[slot].bad) = 1;
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              ptx::mbar_arrive(bar(c.full[stage]));
              ptx::mbar_arrive(bar(c.full[stage]));
            }
          }
          if (++stage == S::kStages) stage = 0;
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(c.iempty[slot]));
      }
    }
  } else if (warp >= S::kLoadWarp0) {
    // ---------------------------------------------------------------- loads
    if constexpr (kNQ == 2) shrink_registers<80>();
    // An instruction copies 128 bytes of 4 rows, 8 lanes each.  Row r's pieces sit at piece ^ r % 8, which for row 4 i + sub
    // is piece ^ sub ^ 4 (i % 2).
    constexpr int kWarpKeys = kKeys / 4, kGroups = kWarpKeys / 4, kHalves = DP / 64;
    const int lw = warp - S::kLoadWarp0;
    const int piece = lane & 7, sub = lane >> 3;
    const int halves = (p.head_dim - piece * 8 + 63) / 64;   // 128-byte blocks of a row that hold a piece of this lane
    const uint32_t lane_at = static_cast<uint32_t>(sub * 128 + ((piece ^ sub) << 4));
    auto place = [&](uint32_t block0, int rows_in, int i, int half) {   // of rows 4 i .. 4 i + 3 of a block of `rows_in`
      return ((block0 + lane_at) ^ static_cast<uint32_t>((i & 1) << 6)) + i * 512 + half * rows_in * 128;
    };
    const uint32_t kv_at = sbase + S::kOffKV + lw * kWarpKeys * 128;
    int stage = 0, open = 0;
    uint32_t phase = 0, items = 0, queries = 0, tiles = 0;
    unsigned long long meta = 0;           // of each open copy a byte, the oldest lowest: kLook, kQueries, the item's slot, the stage
    constexpr unsigned kLook = 1, kQueries = 2, kSlot = 4;
    bool ok = true;
    auto finish = [&]() {                  // the oldest open copy has landed (the caller has waited)
      const unsigned m = meta & 255;
      const int old_stage = m >> 3;
      meta >>= 8;
      --open;
      if (m & kLook) {                     // this thread's own pieces: what is not finite leaves
        unsigned bad = 0;
#pragma unroll 1
        for (int i = 0; i < kGroups; ++i) {
#pragma unroll
          for (int h = 0; h < kHalves; ++h) {
            if (h >= halves) continue;
            uint4* v = reinterpret_cast<uint4*>(smem + (place(kv_at + old_stage * S::kTileBytes, kKeys, i, h) - sbase));
            uint4 x = *v;
            constexpr uint32_t kExp = std::is_same<T, __half>::value ? 0x7C007C00u : 0x7F807F80u;
            unsigned here = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t hit = __vcmpeq2((&x.x)[w] & kExp, kExp);
              (&x.x)[w] &= ~hit;
              here |= hit;
            }
            if (here) *v = x;
            bad |= here;
          }
        }
        if (bad) *const_cast<volatile int*>(&c.item[m & kSlot ? 1 : 0].bad) = 1;
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(m & kQueries ? bar(c.qfull) : bar(c.full[old_stage]));
    };
    auto oldest = [&]() {                  // waits for the oldest open copy and hands it on
      if (open > 5) cp_wait<5>();
      else if (open == 5) cp_wait<4>();
      else if (open == 4) cp_wait<3>();
      else if (open == 3) cp_wait<2>();
      else if (open == 2) cp_wait<1>();
      else cp_wait<0>();
      finish();
    };
    // A wait in which open copies are handed on as they land: who releases the barrier may be waiting for them.
    auto wait_open = [&](unsigned long long& b, uint32_t parity) {
      while (open) {
        if (__all_sync(0xFFFFFFFFu, ptx::mbar_try_wait(bar(b), parity))) return true;
        oldest();
      }
      return wait(b, parity);
    };
    auto close = [&](unsigned m) {         // of a copy that has been issued
      cp_commit();
      meta |= static_cast<unsigned long long>(m) << (8 * open);
      ++open;
      if (open > S::kAhead) oldest();
    };
    const int blocks = (p.head_dim + 63) / 64;
    uint32_t boxed = 0, boxed_phase = 0, looked = 0, raw_phase = ~0u, q_sent = 0;   // stages that boxes were sent to, in which phase, to whom; queries too
    const bool boxes = a.box_rows > 0 && lane < kWarpKeys && lane % max(a.box_rows, 1) == 0;   // this lane's key begins a box
    while (ok) {
      const int slot = items & 1;
      if (!wait_open(c.ifull[slot], (items >> 1) & 1)) { ok = false; break; }
      ++items;
      const Item it = c.item[slot];
      __syncwarp();
      if (it.b < 0) {
        while (open) oldest();
        break;
      }
      if (lane == 0) ptx::mbar_arrive(bar(c.iempty[slot]));
      if (it.t0 >= it.t1) continue;
      const int32_t* table = p.table + static_cast<long long>(it.b) * p.table_width;
      int key = 0, entry = 0, page = -1;
      bool want = false;
      auto fetch = [&](int t) {            // lane's key of tile t: its page
        key = t * kKeys + lw * kWarpKeys + lane;
        want = lane < kWarpKeys && key >= it.key_lo && key < it.key_hi;
        entry = static_cast<int>(static_cast<unsigned long long>(static_cast<unsigned>(key)) * a.page_mul >> a.page_shift);
        // (read once: past the first-level cache.  Not by the read-only path, which asks that nobody writes while this kernel
        // lives: it may have been launched while the plan was still being written, and waits for that above)
        page = want ? __ldcg(table + entry) : -1;
      };
      fetch(it.t0);
      auto queries_of = [&]() {            // row r of the item is token r / group, head r % group
        if (!wait_open(c.qempty, (queries & 1) ^ 1)) return false;
        ++queries;
        if (a.q_boxes) {
          const bool mine = lw == 0 ? it.lo[0] < it.hi[0] : lw < kNQ && it.lo[1] < it.hi[1];
          if (mine && lane == 0) {
            const uint32_t at = sbase + lw * S::kQBytes;
            q_sent |= 1;
            ptx::mbar_arrive_expect_tx(bar(c.qfull), 128 * 128 * blocks);
            for (int h = 0; h < blocks; ++h)
              ptx::tma_load_4d(at + h * 128 * 128, &map_q, 64 * h, 0, it.kv_head, it.first + token_of(a, it.row0 + lw * 128), bar(c.qfull));
          } else if (lane == 0) {
            ptx::mbar_arrive(bar(c.qfull));
          }
          __syncwarp();
          return true;
        }
        const T* q = static_cast<const T*>(p.q);
#pragma unroll
        for (int s = 0; s < kNQ; ++s) {
          if (it.lo[s] >= it.hi[s]) continue;
          const int r = s * 128 + lw * 32 + lane;
          const int packed = it.row0 + r, token = token_of(a, packed), head = packed - token * a.group;
          const long long off = (it.first + token) * p.q_token + static_cast<long long>(it.kv_head * a.group + head) * p.head_dim;
          const unsigned rows = __ballot_sync(0xFFFFFFFFu, r < it.rows);
          const uint32_t at = sbase + s * S::kQBytes + lw * 32 * 128;
#pragma unroll 2
          for (int i = 0; i < 8; ++i) {
            const long long o = __shfl_sync(0xFFFFFFFFu, off, 4 * i + sub);
            const bool on = rows >> (4 * i + sub) & 1;
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
              if (on && h < halves) cp_async16(place(at, 128, i, h), q + o + piece * 8 + 64 * h);
          }
        }
        close(kQueries);
        return true;
      };
      // the queries' place is free once the item before has its last scores: the first tile need not wait for that
      const bool at_once = queries == 0;
      if (at_once) ok = queries_of();
      for (int t = it.t0; ok && t < it.t1; ++t, ++tiles) {
        const bool good = want && page >= 0 && page < p.pages;
        if (want && !good) atomicOr(p.status, kStatusPageRange);
        const unsigned rows = __ballot_sync(0xFFFFFFFFu, good), unread = __ballot_sync(0xFFFFFFFFu, want && !good);
        if (lane == 0) c.valid[tiles & 15][lw] = ~unread;
        const int place_in = key - entry * p.page_size, now = page;
        const unsigned off_k = good ? page * a.k_page16 + place_in * a.k_slot16 + it.kv_head * a.k_head16 : 0u;
        const unsigned off_v = good ? page * a.v_page16 + place_in * a.v_slot16 + it.kv_head * a.v_head16 : 0u;
        // the page of the box that begins at this lane's key: that of any of its keys.  One without a page, or without a key
        // that some row sees, is zeros: a coordinate past the cache
        const unsigned in_box = rows >> lane & ((2u << (a.box_rows - 1 & 31)) - 1u);
        const int some_page = __shfl_sync(0xFFFFFFFFu, now, in_box ? lane + __ffs(in_box) - 1 : lane);
        const int box_page = in_box ? some_page : p.pages;
        if (t + 1 < it.t1) fetch(t + 1);
        const bool full = t * kKeys >= it.full_lo && (t + 1) * kKeys <= it.full_hi;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          if (!wait_open(c.empty[stage], phase ^ 1)) { ok = false; break; }
          const uint4* base = static_cast<const uint4*>(kv ? p.v_cache : p.k_cache);
          const uint32_t at = kv_at + stage * S::kTileBytes;
          const unsigned off = kv ? off_v : off_k;
          const bool all = rows == static_cast<unsigned>((1ull << kWarpKeys) - 1), look = kv && !full;
          if (a.box_rows) {
            // values that not every row sees pass the look warps before the MMA
            const uint32_t to = look ? bar(c.raw[stage]) : bar(c.full[stage]);
            if (lane == 0) ptx::mbar_arrive_expect_tx(to, kWarpKeys * 128 * blocks);
            boxed |= 1u << stage;
            boxed_phase = (boxed_phase & ~(1u << stage)) | phase << stage;
            looked = (looked & ~(1u << stage)) | (look ? 1u << stage : 0u);
            if (look) raw_phase ^= 1u << stage;
            __syncwarp();
            if (boxes) {
              auto coordinate = [&](int which) { return which == 0 ? place_in : (which == 1 ? it.kv_head : box_page); };
              const int y = coordinate(a.box_order[0]), z = coordinate(a.box_order[1]), w = coordinate(a.box_order[2]);
#pragma unroll
              for (int h = 0; h < kHalves; ++h)
                if (h < blocks) ptx::tma_load_4d(at + lane * 128 + h * kKeys * 128, kv ? &map_v : &map_k, 64 * h, y, z, w, to);
            }
          } else if (all) {
            const uint4* from = base + piece;
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
              const uint4* row = from + __shfl_sync(0xFFFFFFFFu, off, 4 * i + sub);
#pragma unroll
              for (int h = 0; h < kHalves; ++h)
                if (h < halves) cp_async16(place(at, kKeys, i, h), row + 8 * h);
            }
          } else {                         // a key without a page, or that no row sees, is zeros
#pragma unroll 2
            for (int i = 0; i < kGroups; ++i) {
              const uint4* row = base + __shfl_sync(0xFFFFFFFFu, off, 4 * i + sub);
              const bool on = rows >> (4 * i + sub) & 1;
#pragma unroll
              for (int h = 0; h < kHalves; ++h)
                if (h < halves) cp_async16(place(at, kKeys, i, h), row + (on ? piece + 8 * h : 0), on ? 16u : 0u);
            }
          }
          if (!a.box_rows) close((look ? kLook : 0u) | (slot ? kSlot : 0u) | static_cast<unsigned>(stage) << 3);
          if (++stage == S::kStages) stage = 0, phase ^= 1;
        }
        if (ok && t == it.t0) {
          if (!at_once) ok = queries_of();
          while (open) oldest();           // (copied: it is waited for before more is asked for)
        }
      }
    }
    if (!ok) {
      // nothing may land after the CTA: wait (bounded) for the copies already issued
      cp_wait<0>();
      const uint64_t t0 = ptx::globaltimer();
      for (int i = 0; i < S::kStages; ++i)
        if (boxed >> i & 1)
          while (!ptx::mbar_try_wait(looked >> i & 1 ? bar(c.raw[i]) : bar(c.full[i]),
                                     looked >> i & 1 ? raw_phase >> i & 1 : boxed_phase >> i & 1) &&
                 ptx::globaltimer() - t0 < kDrainLimitNs) {}
      if (q_sent)
        while (!ptx::mbar_try_wait(bar(c.qfull), (queries & 1) ^ 1) && ptx::globaltimer() - t0 < kDrainLimitNs) {}
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------------- softmax: a thread a row
    if constexpr (kNQ == 2) grow_registers<176>();
    const int s = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;   // the warp's 32 lanes of tensor memory
    const uint32_t sc = s_col(s) + lanes, oc = o_col(s) + lanes;
    const float scale = a.scale_log2;
    uint32_t items = 0, tiles = 0, s_phase = 0, o_phase = 0;
    while (true) {
      const int slot = items & 1;
      if (!wait(c.ifull[slot], (items >> 1) & 1)) break;
      ++items;
      const Item& it = c.item[slot];
      if (it.b < 0) break;
      const int r = s * 128 + row;
      const bool live_row = r < it.rows, live_warp = s * 128 + (warp & 3) * 32 < it.rows;
      const int row_hi = it.position0 + token_of(a, it.row0 + r) + 1;
      const int row_lo = p.window > 0 ? max(0, row_hi - p.window) : 0;
      float m = -CUDART_INF_F, l = 0.f;
      bool ok = true;
      const int t0 = it.t0, t1 = it.t1, lo = it.lo[s], hi = it.hi[s];
      for (int t = t0; t < t1; ++t, ++tiles) {
        if (t < lo || t >= hi) continue;
        if (!wait(c.sfull[s], s_phase)) { ok = false; break; }
        s_phase ^= 1;
        ptx::tc_fence_after();
        if (live_warp) {
          float x[kKeys];
#pragma unroll
          for (int i = 0; i < kKeys / 32; ++i) ptx::tmem_ld_32x32b_x32(sc + 32 * i, *reinterpret_cast<uint32_t(*)[32]>(x + 32 * i));
          ptx::tmem_ld_wait();
          // keys that the row does not see
          const int key0 = t * kKeys;
          if (__any_sync(0xFFFFFFFFu, key0 < row_lo || key0 + kKeys > row_hi)) {
            const int from = row_lo - key0;
            const unsigned count = static_cast<unsigned>(max(row_hi - row_lo, 0));
#pragma unroll
            for (int i = 0; i < kKeys; ++i)
              if (static_cast<unsigned>(i - from) >= count) x[i] = -CUDART_INF_F;
          }
          const uint32_t* valid = c.valid[tiles & 15];
          if ((valid[0] & valid[1] & valid[2] & valid[3]) != 0xFFFFFFFFu) {
#pragma unroll
            for (int i = 0; i < kKeys; ++i)
              if (!(valid[i / (kKeys / 4)] >> (i % (kKeys / 4)) & 1)) x[i] = -CUDART_INF_F;
          }
          float top[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int i = 4; i + 8 <= kKeys; i += 8)
#pragma unroll
            for (int j = 0; j < 4; ++j) top[j] = max3(top[j], x[i + 2 * j], x[i + 2 * j + 1]);
#pragma unroll
          for (int j = 0; j < 4; ++j) top[j] = fmaxf(top[j], x[kKeys - 4 + j]);
          const float now = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * scale;
          const bool grown = now > m + kGrow;
          if (__any_sync(0xFFFFFFFFu, grown)) {
            const float mn = grown ? now : m;
            const float keep = grown ? ex2(m - mn) : 1.f;
            m = mn;
            l *= keep;
            if (t > lo) {                  // o is at rest: the scores' MMA came after its last
#pragma unroll 1
              for (int i = 0; i < p.head_dim; i += 16) {
                uint32_t o[16];
                ptx::tmem_ld_32x32b_x16(oc + i, o);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * keep);
                ptx::tmem_st_32x32b_x16(oc + i, o);
              }
            }
          }
          const float base = lift<T>() - (m == -CUDART_INF_F ? 0.f : m);
          float2 sum[2] = {};
#pragma unroll
          for (int half = 0; half < 2; ++half) {           // p v of the first half starts while the second is made
#pragma unroll
            for (int i = half * kKeys / 64; i < (half + 1) * kKeys / 64; ++i) {
              uint32_t w[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                float u = x[32 * i + 2 * j], v = x[32 * i + 2 * j + 1];
                fma2(u, v, scale, base);
                u = ex2(u);
                v = ex2(v);
                sum[j & 1] = add2(sum[j & 1], u, v);
                w[j] = pack2(u, v, T());
              }
              ptx::tmem_st_32x32b_x16(sc + 16 * i, w);
            }
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(c.pready[s][half]));
          }
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        } else if (lane == 0) {
          ptx::mbar_arrive(bar(c.pready[s][0]));
          ptx::mbar_arrive(bar(c.pready[s][1]));
        }
      }
      if (!ok) break;
      const bool any = hi > lo;
      if (any) {
        if (!wait(c.ofull[s], o_phase)) break;
        o_phase ^= 1;
        ptx::tc_fence_after();
      }
      if (live_warp) {
        const int packed = it.row0 + r, token = token_of(a, packed), head = packed - token * a.group;
        const long long at = static_cast<long long>(it.first + token) * p.heads + it.kv_head * a.group + head;
        const unsigned live_rows = __ballot_sync(0xFFFFFFFFu, live_row);
        const bool bad = *const_cast<const volatile int*>(&it.bad) != 0;
        const float inv = it.slot >= 0 ? 1.f : (l > 0.f || isnan(l) ? 1.f / l : 0.f);
        float* part = a.partials + static_cast<size_t>(max(it.slot, 0)) * partial_floats<DP>();
        float odd[2] = {0.f, 0.f};         // a NaN once a value of o is not finite
#pragma unroll 1
        for (int i = 0; i < p.head_dim; i += 32) {
          uint32_t o[32];
          if (any) {
            ptx::tmem_ld_32x32b_x32(oc + i, o);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
              if (i + j >= p.head_dim) break;              // (columns that hold anything)
#pragma unroll
              for (int y = 0; y < 8; y += 2) odd2(odd, __uint_as_float(o[j + y]), __uint_as_float(o[j + y + 1]));
            }
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = 0;
          }
          if (it.slot < 0) {
            // the 4 lanes of a group exchange 16-byte pieces: lane x then holds piece x of each of their 4 rows, and an
            // instruction writes 64 bytes of 8 rows (16 bytes of 32 took 4 times as long)
            uint32_t w[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int y = 0; y < 4; ++y)
                w[j][y] = pack2(__uint_as_float(o[8 * j + 2 * y]) * inv, __uint_as_float(o[8 * j + 2 * y + 1]) * inv, T());
#pragma unroll
            for (int x = 1; x <= 2; x <<= 1)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if (j & x) continue;
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  const bool up = lane & x;
                  const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, up ? w[j][y] : w[j | x][y], x);
                  if (up) w[j][y] = got;
                  else w[j | x][y] = got;
                }
              }
            const int d = i + 8 * (lane & 3);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int from = (lane & ~3) + j;
              const long long row_at = __shfl_sync(0xFFFFFFFFu, at, from);
              if ((live_rows >> from & 1) && d < p.head_dim)
                *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + row_at * p.head_dim + d) = make_uint4(w[j][0], w[j][1], w[j][2], w[j][3]);
            }
          } else if (any) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              __stcg(reinterpret_cast<uint4*>(part) + (i / 4 + j) * S::kRows + r, make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]));
          }
        }
        if (it.slot < 0) {
          if (p.lse && live_row) p.lse[at] = m * 0.693147180559945f + logf(l * (std::is_same<T, __half>::value ? 1.f / 128.f : 1.f));
        } else {
          __stcg(reinterpret_cast<float2*>(part + static_cast<size_t>(S::kRows) * DP) + r, make_float2(any ? m : -CUDART_INF_F, l));
        }
        __syncwarp();
        const unsigned again = __ballot_sync(0xFFFFFFFFu, live_row && isnan(odd[0] + odd[1]) && !isnan(l));
        if (again) {
          // values that are not finite, of the keys in the tiles seen by all: their sum is the result of the rows that
          // have met them.  A lane takes 8 dimensions of every 32 / pieces-th key.
          const int pieces = p.head_dim / 8, step = 32 / pieces, piece = lane % pieces;
          float f[8] = {};
#pragma unroll 1
          for (int t = max(t0, lo); t < min(t1, hi); ++t) {
            if (t * kKeys < it.full_lo || (t + 1) * kKeys > it.full_hi) continue;
#pragma unroll 4
            for (int key = t * kKeys + lane / pieces; key < (t + 1) * kKeys; key += step) {
              const int page = p.table[static_cast<long long>(it.b) * p.table_width + key / p.page_size];
              if (lane / pieces >= step || page < 0 || page >= p.pages) continue;
              const T* v = static_cast<const T*>(p.v_cache) + page * p.v_page + key % p.page_size * p.v_slot + it.kv_head * p.v_head;
              const uint4 x = *reinterpret_cast<const uint4*>(v + piece * 8);
#pragma unroll
              for (int y = 0; y < 8; ++y) {
                const float one = Tr::to_f32(Tr::from_bits(static_cast<uint16_t>((&x.x)[y / 2] >> (16 * (y & 1)))));
                if (!isfinite(one)) f[y] += one;
              }
            }
          }
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            float sum = 0.f;
            for (int i = 0; i < step; ++i) sum += __shfl_sync(0xFFFFFFFFu, f[y], i * pieces + piece);
            for (int i = 0; i < 32; ++i) {
              const long long row_at = __shfl_sync(0xFFFFFFFFu, at, i);
              if (!(again >> i & 1) || lane >= pieces || sum == 0.f) continue;
              const int d = piece * 8 + y;
              if (it.slot < 0) static_cast<T*>(p.out)[row_at * p.head_dim + d] = Tr::from_f32(sum);
              else __stcg(part + ((d / 4) * S::kRows + r - lane + i) * 4 + d % 4, sum);
            }
          }
          __syncwarp();
        }
        if (bad && live_row) {
          // values that are not finite, of the keys that this row sees in the tiles not seen by all
#pragma unroll 1
          for (int t = t0; t < t1; ++t) {
            if (t * kKeys >= it.full_lo && (t + 1) * kKeys <= it.full_hi) continue;
#pragma unroll 1
            for (int key = max(t * kKeys, row_lo); key < min((t + 1) * kKeys, row_hi); ++key) {
              const int page = p.table[static_cast<long long>(it.b) * p.table_width + key / p.page_size];
              if (page < 0 || page >= p.pages) continue;
              const T* v = static_cast<const T*>(p.v_cache) + page * p.v_page + key % p.page_size * p.v_slot + it.kv_head * p.v_head;
#pragma unroll 1
              for (int d = 0; d < p.head_dim; ++d) {
                const float f = Tr::to_f32(v[d]);
                if (isfinite(f)) continue;
                if (it.slot < 0) {
                  T* to = static_cast<T*>(p.out) + at * p.head_dim + d;
                  *to = Tr::from_f32(Tr::to_f32(*to) + f);
                } else {
                  float* to = part + ((d / 4) * S::kRows + r) * 4 + d % 4;
                  __stcg(to, __ldcg(to) + f);
                }
              }
            }
          }
        }
        ptx::tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(c.iempty[slot]));
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == S::kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// The join: a CTA takes 16 columns of one cut item, a thread a row.
constexpr int kJoinCols = 16;

template <typename T, int DP>
__global__ void __launch_bounds__(Shape<DP>::kRows) k_join(const __grid_constant__ Args a) {
  using S = Shape<DP>;
  const ChunkProblem& p = a.p;
  decode::pdl_launch_dependents();
  decode::pdl_wait();
  Record rec;
  reinterpret_cast<int4*>(&rec)[0] = __ldcg(reinterpret_cast<const int4*>(a.records + blockIdx.x));
  reinterpret_cast<int4*>(&rec)[1] = __ldcg(reinterpret_cast<const int4*>(a.records + blockIdx.x) + 1);
  rec.last_run = min(rec.last_run, static_cast<int>(gridDim.x) - 1);   // (past it only where lengths were written meanwhile)
  const int row = threadIdx.x, col = blockIdx.y * kJoinCols;
  if (!rec.valid || row >= rec.rows || col >= p.head_dim) return;
  auto part_of = [&](int run) {
    return a.partials + static_cast<size_t>(2 * run + (run == rec.first_run ? 1 : 0)) * partial_floats<DP>();
  };
  // kBatch parts in flight at a time (64 tokens on 4000 keys / the mixed batch of 16: 28.5 / 111 us with one after the
  // other, 24.7 / 108 so, 25.3 / 113 with four, which leave fewer CTAs an SM)
  constexpr int kBatch = 2;
  float top = -CUDART_INF_F, l = 0.f, o[kJoinCols] = {};
  for (int run0 = rec.first_run; run0 <= rec.last_run; run0 += kBatch) {
    float2 ml[kBatch];
    float4 v[kBatch][kJoinCols / 4];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const float* part = part_of(min(run0 + j, rec.last_run));
      ml[j] = __ldcg(reinterpret_cast<const float2*>(part + static_cast<size_t>(S::kRows) * DP) + row);
#pragma unroll
      for (int i = 0; i < kJoinCols / 4; ++i)
        v[j][i] = __ldcg(reinterpret_cast<const float4*>(part) + static_cast<size_t>(col / 4 + i) * S::kRows + row);
    }
    float mn = top;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) mn = fmaxf(mn, ml[j].x);   // (a repeated last part changes nothing)
    // (no factor is 0: an infinite value stays infinite; 2^-126 of a finite one is nothing)
    constexpr float kLeast = 1.17549435e-38f;
    const float base = mn == -CUDART_INF_F ? 0.f : mn, keep = fmaxf(ex2(top - base), kLeast);
    top = mn;
    l *= keep;
#pragma unroll
    for (int i = 0; i < kJoinCols; ++i) o[i] *= keep;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      // of a run that had no key of the row o says nothing
      if (run0 + j > rec.last_run || (ml[j].x == -CUDART_INF_F && !isnan(ml[j].y))) continue;
      const float f = fmaxf(ex2(ml[j].x - base), kLeast);
      l += ml[j].y * f;
#pragma unroll
      for (int i = 0; i < kJoinCols / 4; ++i) {
        o[4 * i] += v[j][i].x * f;
        o[4 * i + 1] += v[j][i].y * f;
        o[4 * i + 2] += v[j][i].z * f;
        o[4 * i + 3] += v[j][i].w * f;
      }
    }
  }
  const int packed = rec.row0 + row, token = token_of(a, packed), head = packed - token * a.group;
  const long long at = static_cast<long long>(rec.first + token) * p.heads + rec.kv_head * a.group + head;
  const float inv = l > 0.f || isnan(l) ? 1.f / l : 0.f;
  uint4* to = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + at * p.head_dim + col);
#pragma unroll
  for (int j = 0; j < kJoinCols / 8; ++j) {
    uint4 w;
#pragma unroll
    for (int y = 0; y < 4; ++y) (&w.x)[y] = pack2(o[8 * j + 2 * y] * inv, o[8 * j + 2 * y + 1] * inv, T());
    if (col + 8 * j < p.head_dim) to[j] = w;
  }
  if (p.lse && col == 0) p.lse[at] = top * 0.693147180559945f + logf(l * (std::is_same<T, __half>::value ? 1.f / 128.f : 1.f));
}

// ------------------------------------------------------------------------------ host side
// The tensor map of a cache [slot, head, page, dimension], its dimensions in the order of their strides.
inline bool cache_map(const ChunkProblem& p, const void* cache, long long slot, long long head, long long page, int box_rows,
               int* order, CUtensorMap* map) {
  const uint64_t size[3] = {static_cast<uint64_t>(p.page_size), static_cast<uint64_t>(p.kv_heads), static_cast<uint64_t>(p.pages)};
  uint64_t stride[3] = {static_cast<uint64_t>(slot) * 2, static_cast<uint64_t>(head) * 2, static_cast<uint64_t>(page) * 2};
  const uint32_t rows[3] = {static_cast<uint32_t>(box_rows), 1, 1};
  uint64_t longest = static_cast<uint64_t>(p.head_dim) * 2;
  for (int i = 0; i < 3; ++i) {
    if (size[i] > 1 && stride[i] == 0) return false;
    if (stride[i] > longest) longest = stride[i];
  }
  for (int i = 0; i < 3; ++i) {
    if (size[i] == 1) stride[i] = longest;                 // never stepped over
    order[i] = i;
  }
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (stride[order[j]] > stride[order[j + 1]]) {
        const int x = order[j];
        order[j] = order[j + 1];
        order[j + 1] = x;
      }
  uint64_t dims[4] = {static_cast<uint64_t>(p.head_dim)}, strides[3];
  uint32_t box[4] = {64}, step[4] = {1, 1, 1, 1};
  for (int i = 0; i < 3; ++i) {
    dims[i + 1] = size[order[i]];
    strides[i] = stride[order[i]];
    box[i + 1] = rows[order[i]];
  }
  return encode_tensor_map_nd(map, p.dtype == 0 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                              const_cast<void*>(cache), dims, strides, box, step, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <typename T, int DP>
cudaError_t launch(const Args& args, cudaStream_t stream) {
  using S = Shape<DP>;
  constexpr size_t kSmem = S::kOffControl + sizeof(Control<DP>) + 1024;
  static_assert(kSmem <= 232448, "the layout must fit one CTA's shared memory (227 KB)");
  auto kern = k_chunk<T, DP>;
  const DeviceInfo& dev = device_info();
  static std::atomic<unsigned long long> opted_in{0};       // per device
  if (dev.device >= 64 || !(opted_in.load(std::memory_order_relaxed) & (1ull << dev.device))) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
    if (e != cudaSuccess) return e;
    if (dev.device < 64) opted_in.fetch_or(1ull << dev.device, std::memory_order_relaxed);
  }
  const int grid = dev.sm_count < kMaxRuns ? dev.sm_count : kMaxRuns;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  Args a = args;
  CUtensorMap map_k = {}, map_v = {}, map_q = {};
  // The cache as boxes of consecutive keys of one page and head, 64 dimensions wide: the most keys, a power of two from
  // 8 (whole swizzle atoms) to a loader warp's share, that divide a page.  Other pages, and strides that a tensor map
  // does not take, are copied by cp.async.
  int box = a.p.page_size & -a.p.page_size;
  if (box > S::kKeys / 4) box = S::kKeys / 4;
  if (box >= 8 && cache_map(a.p, a.p.k_cache, a.p.k_slot, a.p.k_head, a.p.k_page, box, a.box_order, &map_k)) {
    int order[3];
    if (cache_map(a.p, a.p.v_cache, a.p.v_slot, a.p.v_head, a.p.v_page, box, order, &map_v) &&
        order[0] == a.box_order[0] && order[1] == a.box_order[1] && order[2] == a.box_order[2])
      a.box_rows = box;
  }
  // A block's 128 packed rows are whole tokens where the group divides it.  (The tail of a sequence's last block reads the
  // next sequence's rows, or zeros: rows that nobody looks at.)
  if (128 % a.group == 0) {
    const uint64_t dims[4] = {static_cast<uint64_t>(a.p.head_dim), static_cast<uint64_t>(a.group),
                              static_cast<uint64_t>(a.p.kv_heads), static_cast<uint64_t>(a.p.tokens)};
    const uint64_t row = static_cast<uint64_t>(a.p.head_dim) * 2;
    const uint64_t strides[3] = {row, row * a.group,
                                 a.p.tokens > 1 ? static_cast<uint64_t>(a.p.q_token) * 2 : row * a.p.heads};
    const uint32_t boxes[4] = {64, static_cast<uint32_t>(a.group), 1, static_cast<uint32_t>(128 / a.group)}, step[4] = {1, 1, 1, 1};
    a.q_boxes = strides[2] > 0 &&
                encode_tensor_map_nd(&map_q, a.p.dtype == 0 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                                     const_cast<void*>(a.p.q), dims, strides, boxes, step, CU_TENSOR_MAP_SWIZZLE_128B);
  }
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, map_k, map_v, map_q, a);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(grid, DP / kJoinCols);
  cfg.blockDim = dim3(S::kRows);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, k_join<T, DP>, a);
}

template <typename T>
cudaError_t launch_dim(const Args& a, cudaStream_t stream) {
  if (a.p.head_dim <= 64) return launch<T, 64>(a, stream);
  if (a.p.head_dim <= 128) return launch<T, 128>(a, stream);
  return launch<T, 256>(a, stream);
}

// One translation unit each (chunk_attention_{f16,bf16}.cu).
cudaError_t launch_f16(const Args& a, cudaStream_t stream);
cudaError_t launch_bf16(const Args& a, cudaStream_t stream);

}  // namespace chunk
}  // namespace gptq
