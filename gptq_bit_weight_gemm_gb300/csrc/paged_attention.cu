// paged_attention.cu -- attention of one new token of each sequence over a paged key-value cache:
//   out = sum_j p_j v_j,  p = softmax_j(scale q . k_j).
//
// Bound: the cache is read once (4 bytes per key, kv head and dimension for 16-bit k and v) against
// 4 flops per key, query head and dimension, so HBM bounds it at any group size the tensor cores
// keep up with.  The running form of the softmax makes one pass of it: with the maximum m, the sum l
// and the accumulator o of the keys so far, a new block of scores s moves them to
//   m' = max(m, max s),  l' = l e^(m - m') + sum e^(s - m'),  o' = o e^(m - m') + e^(s - m') v,
// and two partial results of disjoint keys join the same way.
//
// Split: the work of a call is a line of tiles of 64 keys -- sequence by sequence, kv head by kv head
// (and 16 query heads by 16) -- cut into equal runs, one per resident CTA.  The cut is computed on the
// device from the lengths, so a batch of very different lengths fills the GPU as evenly as an even
// one, and a single long sequence spreads over all of it.  An item (one sequence and kv head) inside
// one run is finished there; of an item that spans several runs each CTA leaves a partial (m, l, o) in
// the workspace, and the last one to arrive joins them in run order (the result does not depend on
// who is last).  A run has at most two partials, so the workspace does not grow with the problem.
//
// Inside a CTA each of 4 warps takes 16 of a tile's 64 keys and streams them through a ring of its
// own (cp.async, 16 bytes a lane, whole rows of consecutive bytes an instruction), so the main loop
// has no CTA barrier.  Measured on the same 512 MB: cp.async moves 6.9 TB/s with 96 KB in flight per
// SM, while one bulk copy per 256-byte row moves 1.4 to 2.7 TB/s (about 50 ns of issue each), so rows
// scattered over pages go through cp.async.  The 16-byte pieces of row r sit at piece ^ swizzle(r), with
// which the three ways a warp touches a stage are free of bank conflicts: whole rows written, k
// fragments read with 16-byte loads, v fragments with ldmatrix.  The k dimension of an MMA may be
// permuted as long as both operands agree: lane (g, t) = (lane / 4, lane % 4) reads 8 consecutive
// dimensions of key g as the B fragments of two k-steps of q k^T, and the query fragments are loaded in
// the same order.  The scores' C fragment is the A fragment of p v as it stands.
//
// The probabilities go to the tensor cores in two parts, 16 bits of a little less than each and what is left
// (15 significant bits for bf16, 20 for fp16; one part shows in the output: relative error 2.2e-3 in bf16, 1.7e-3
// so).  Both are above 0, so an infinite value stays infinite.  The second parts are the A rows 8 .. 15 where an item has at most 8 query heads, and products of their
// own where it has more.  They are taken 2^15 times as large, as l and o are throughout: one part in 2^25
// of the largest, of which a long flat tail may have thousands, would be nothing in fp16.
//
// Measured (GB300, bf16, 32 query and 8 kv heads of 128): 64 sequences of 512 to 8192 keys 124 us,
// 6.1 TB/s; one of 131072 keys 90 us, 6.0 TB/s; one of 997 keys 8.5 us, the latencies of launch, lengths,
// table, keys, partial and join one after the other.
#include <math_constants.h>

#include <atomic>
#include <type_traits>

#include "decode.cuh"
#include "gptq_device.cuh"
#include "gptq_internal.h"
#include "serving_internal.h"

namespace gptq {
namespace attention {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kWarpKeys = 16, kTileKeys = kWarps * kWarpKeys;
constexpr int kMaxRows = 16;             // query heads of one item
constexpr float kLift = 15.f;            // probabilities are taken times 2^kLift
constexpr int kMaxCtas = 512;            // runs, at most
constexpr size_t kControlBytes = 4096;   // arrival counters, one per run

// Dimensions padded to DP (64, 128, 256); R = 1 or 2 blocks of 8 query rows.
template <int DP, int R>
struct Shape {
  static constexpr int kBlocks = DP / 32;                  // 32-dimension blocks of k
  static constexpr int kCols = DP / 8;                     // column tiles of v, 16-byte pieces of a row
  static constexpr int kRowBytes = DP * 2;
  static constexpr int kLaneRows = DP / 16;                // rows one lane copies: 16 rows, 32 / kCols lanes each
  static constexpr int kStageBytes = 2 * kWarpKeys * kRowBytes;   // k rows, then v rows
  static constexpr int kStages = DP == 64 ? 4 : 3;
  static constexpr int kCtas = DP == 256 ? 1 : (DP == 128 ? 2 : 3);   // per SM
  static constexpr size_t kRing = static_cast<size_t>(kStages) * kWarps * kStageBytes;
  static constexpr size_t kMerge = static_cast<size_t>(kWarps - 1) * kCols * 2 * 128;   // one block of 8 rows
  static constexpr size_t kSmem = kRing + kMerge;
};

__host__ __device__ constexpr int swizzle(int row) {
  return ((row >> 1 & 1) * 5) ^ ((row >> 2 & 1) * 2) ^ ((row & 1) * 4);
}

// floats of one partial: accumulators, then m and l per row
constexpr size_t partial_floats(int dp) { return static_cast<size_t>(kMaxRows) * dp + 2 * kMaxRows; }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// 16 bytes from L2 (a partial another SM has written); volatile, so that a batch of them is issued
// before the first is used
__device__ __forceinline__ float4 ldcg4(const float* p) {
  float4 v;
  asm volatile("ld.global.cg.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ float2 ldcg2(const float* p) {
  float2 v;
  asm volatile("ld.global.cg.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&v)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(a)
               : "memory");
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1, __half) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1, __nv_bfloat16) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct Args {
  AttentionProblem p;
  int group;          // query heads per kv head
  int row_blocks;     // items per (sequence, kv head): 16 query heads each
  int items;          // items per sequence
  float scale_log2;   // scale * log2(e)
  // key / page_size = key * page_mul >> page_shift for keys below 2^30
  unsigned page_mul, page_shift;
  // cache strides in 16-byte units
  unsigned k_page16, k_slot16, k_head16, v_page16, v_slot16, v_head16;
  unsigned* counters;
  float* partials;
};

__device__ __forceinline__ int clamp_len(const AttentionProblem& p, int n) {
  const int most = p.table_width * p.page_size;
  return n < 0 ? 0 : (n > most ? most : n);
}
// first live key, first key of the tiles (a multiple of 16), tiles (at least one: an item without
// keys still writes its zeros)
__device__ __forceinline__ int first_key(const AttentionProblem& p, int n) {
  return p.window > 0 && n > p.window ? n - p.window : 0;
}
__device__ __forceinline__ int tile_count(const AttentionProblem& p, int n) {
  const int base = first_key(p, n) & ~(kWarpKeys - 1);
  const int nt = (n - base + kTileKeys - 1) / kTileKeys;
  return nt > 0 ? nt : 1;
}

// An item counts as its tiles and kItemUnits more on the line that is cut into runs: what opening,
// joining and writing it takes, in tiles.  Without it a run of many short items ends last (16
// sequences of 40 to 2048 keys, 32 kv heads: the last run at 39 us, the median at 30 us).
constexpr int kItemUnits = 2;
// Units of a run, at least: shorter runs leave more parts to join than they save (one sequence of 4000
// keys: 14.3 us at 1, 11.6 at 2, 12.1 at 4; of 997: 8.3, 8.4, 10.3, a tile alone taking about 1 us).
constexpr int kMinShare = 2;

// A place on the line: u units after the run's begin, tile t of nt of item h of sequence b, whose live
// keys are [lo, n).
struct Cursor {
  int u, b, h, t, nt, n, lo, n_next;
  __device__ __forceinline__ void set_len(const AttentionProblem& p, int raw) {
    n = clamp_len(p, raw);
    lo = first_key(p, n);
    nt = tile_count(p, n);
  }
  __device__ __forceinline__ void set(const AttentionProblem& p, int seq, int raw) {
    b = seq;
    set_len(p, raw);
    n_next = seq + 1 < p.batch ? p.lens[seq + 1] : 0;      // fetched a sequence ahead
  }
  __device__ __forceinline__ bool advance(const Args& a) {   // true: a new item begins
    ++u;
    if (++t < nt) return false;
    t = 0;
    u += kItemUnits;
    if (++h == a.items) {
      h = 0;
      if (b + 1 < a.p.batch) set(a.p, b + 1, n_next);
    }
    return true;
  }
};

// x / y of nonnegative numbers: a 64-bit division costs a few hundred cycles, and tile counts mostly
// fit 32 bits
__device__ __forceinline__ long long divide(long long x, long long y) {
  if (((x | y) >> 32) == 0) return static_cast<unsigned>(x) / static_cast<unsigned>(y);
  return x / y;
}

template <typename T, int DP, int R>
__global__ void __launch_bounds__(kThreads, (Shape<DP, R>::kCtas)) k_attention(const Args a) {
  using S = Shape<DP, R>;
  using Tr = F16Traits<T>;
  const AttentionProblem& p = a.p;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float sm_m[kWarps][kMaxRows], sm_l[kWarps][kMaxRows];
  __shared__ __align__(16) unsigned sm_rows[kWarps][2][kWarpKeys];
  __shared__ long long sm_sum[kWarps];
  __shared__ long long sm_at;
  __shared__ int sm_seq, sm_last, sm_lens[kThreads];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;

  decode::pdl_launch_dependents();
  decode::pdl_wait();

  // ---- this CTA's run: a scan of the sequences' tiles, a chunk of kThreads at a time, gives the total
  // and then the sequence its first tile falls into (a batch of one chunk is read and scanned once)
  long long before = 0, upto = 0;                          // tiles before and with this thread's sequence
  int raw = 0;
  auto scan_chunk = [&](int b0, long long base) {          // returns the tiles up to the chunk's end
    const int b = b0 + static_cast<int>(threadIdx.x);
    raw = b < p.batch ? p.lens[b] : 0;
    const int n = clamp_len(p, raw);
    if (n != raw && blockIdx.x == 0) atomicOr(p.status, kStatusSeqLen);
    const long long w = b < p.batch ? static_cast<long long>(tile_count(p, n) + kItemUnits) * a.items : 0;
    long long c = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xFFFFFFFFu, c, o);
      if (lane >= o) c += v;
    }
    __syncthreads();                                       // sm_sum, sm_lens and sm_seq of the chunk before are read
    if (lane == 31) sm_sum[warp] = c;
    if (threadIdx.x == 0) sm_seq = -1;
    sm_lens[threadIdx.x] = raw;
    __syncthreads();
    long long all = base;
    for (int x = 0; x < kWarps; ++x) {
      if (x < warp) c += sm_sum[x];
      all += sm_sum[x];
    }
    upto = base + c;
    before = upto - w;
    return all;
  };
  long long total = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kThreads) total = scan_chunk(b0, total);
  const long long most = total >= kMinShare ? divide(total, kMinShare) : 1;
  const int runs = most < static_cast<long long>(gridDim.x) ? static_cast<int>(most) : static_cast<int>(gridDim.x);
  const int run = blockIdx.x;
  if (run >= runs) return;
  // runs of `share` tiles, the first `extra` of them one longer
  const long long share = divide(total, runs), extra = total - share * runs;
  const long long begin = share * run + (run < extra ? run : extra), end = begin + share + (run < extra ? 1 : 0);
  auto run_of = [&](long long tile) {
    const long long cut = extra * (share + 1);
    return static_cast<int>(tile < cut ? divide(tile, share + 1) : extra + divide(tile - cut, share));
  };
  {
    long long at = 0;
    for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
      if (p.batch > kThreads) at = scan_chunk(b0, at);
      if (before <= begin && begin < upto) {
        sm_seq = b0 + static_cast<int>(threadIdx.x);
        sm_at = before;
      }
      __syncthreads();
      if (sm_seq >= 0) break;
    }
  }
  if (sm_seq < 0) return;                                  // lengths written while this ran
  Cursor put, get;
  put.b = sm_seq;
  put.set_len(p, sm_lens[sm_seq % kThreads]);
  put.n_next = sm_seq + 1 < p.batch ? ((sm_seq + 1) % kThreads ? sm_lens[(sm_seq + 1) % kThreads] : p.lens[sm_seq + 1]) : 0;
  const int limit = static_cast<int>(end - begin);
  long long tiles_begin;                                   // the consumer's item: its first tile on the line
  {
    const long long rel = begin - sm_at;
    const int units = put.nt + kItemUnits;
    put.h = static_cast<int>(divide(rel, units));
    const int at = static_cast<int>(rel - static_cast<long long>(put.h) * units);
    put.t = at > kItemUnits ? at - kItemUnits : 0;
    put.u = at > kItemUnits ? 0 : kItemUnits - at;
    tiles_begin = begin - at + kItemUnits;
  }
  if (put.u >= limit) return;                              // no tile of an item, only its extra units
  get = put;

  // ---- the ring of this warp.  The offsets of a stage's 16 rows (in 16-byte units, 32 bits: the host
  // refuses caches past 2^32 of them) go through shared memory from the lanes that look them up.
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * (S::kStages * S::kStageBytes);
  unsigned long long live = 0;                             // 16 key bits per stage in flight, oldest first
  const int piece = lane % S::kCols, row0 = lane / S::kCols * S::kLaneRows;
  const bool in_dim = piece * 8 < p.head_dim;
  // lane l < 16 looks up key l of the producer's place: its page (fetched a tile ahead) and slot
  int page = -1, slot = 0, kb = 0, put_hk = put.h / a.row_blocks;
  bool want = false;
  constexpr int kFresh = (2 * S::kCols + 31) / 32;         // 16-byte pieces of the new token's k and v per lane
  uint4 fresh[kFresh];
  int fresh_row = -1;                                      // its place among the 16 keys
  auto fetch_page = [&]() {
    kb = (put.lo & ~(kWarpKeys - 1)) + put.t * kTileKeys + warp * kWarpKeys;
    const int key = kb + lane;
    want = lane < kWarpKeys && key >= put.lo && key < put.n;
    const int entry = static_cast<int>(static_cast<unsigned long long>(static_cast<unsigned>(key)) * a.page_mul >> a.page_shift);
    slot = key - entry * p.page_size;
    page = want ? __ldg(p.table + static_cast<long long>(put.b) * p.table_width + entry) : -1;
    // the new token's own row comes from k_new and v_new: fetched here, a tile ahead.  Past the block table
    // it has no slot: the last one holds an older key
    fresh_row = p.k_new && put.n > kb && put.n <= kb + kWarpKeys ? put.n - 1 - kb : -1;
    if (fresh_row >= 0 && put.n == p.table_width * p.page_size && p.lens[put.b] != put.n) fresh_row = -1;
    if (fresh_row >= 0) {
#pragma unroll
      for (int i = 0; i < kFresh; ++i) {
        const int kv = (lane + 32 * i) / S::kCols, d = (lane + 32 * i) % S::kCols * 8;
        const T* from = kv ? static_cast<const T*>(p.v_new) + put.b * p.vn_batch : static_cast<const T*>(p.k_new) + put.b * p.kn_batch;
        fresh[i] = make_uint4(0u, 0u, 0u, 0u);
        if (kv < 2 && d < p.head_dim) fresh[i] = __ldg(reinterpret_cast<const uint4*>(from + put_hk * p.head_dim + d));
      }
    }
  };
  auto issue = [&](int s, int pos) {
    const bool ok = want && page >= 0 && page < p.pages;
    if (want && !ok) atomicOr(p.status, kStatusPageRange);
    const unsigned mask = __ballot_sync(0xFFFFFFFFu, ok);
    live |= static_cast<unsigned long long>(mask) << (16 * pos);
    if (mask == 0) return;
    if (lane < kWarpKeys) {
      sm_rows[warp][0][lane] = ok ? page * a.k_page16 + slot * a.k_slot16 + put_hk * a.k_head16 : 0u;
      sm_rows[warp][1][lane] = ok ? page * a.v_page16 + slot * a.v_slot16 + put_hk * a.v_head16 : 0u;
    }
    __syncwarp();
    // row row0 + j lands at piece ^ swizzle(row0 + j); the swizzle is linear, and rows start at
    // multiples of 128 bytes, so it is an exclusive or on the lane's own address
    const uint32_t dst = ring + s * S::kStageBytes + row0 * S::kRowBytes + ((piece ^ swizzle(row0)) << 4);
    const int skip = fresh_row >= 0 && (mask >> fresh_row & 1) ? fresh_row : -1;
    if (mask == 0xFFFFu && skip < 0) {
      if (in_dim) {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const uint4* base = static_cast<const uint4*>(kv ? p.v_cache : p.k_cache) + piece;
#pragma unroll
          for (int j4 = 0; j4 < S::kLaneRows; j4 += 4) {
            const uint4 off = *reinterpret_cast<const uint4*>(&sm_rows[warp][kv][row0 + j4]);
#pragma unroll
            for (int j = j4; j < j4 + 4; ++j)
              cp_async16((dst ^ (swizzle(j) << 4)) + (kv * kWarpKeys + j) * S::kRowBytes, base + (&off.x)[j - j4]);
          }
        }
      }
    } else {
      // rows without a live key are filled with zeros: what the cache holds there may be NaN
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint4* base = static_cast<const uint4*>(kv ? p.v_cache : p.k_cache);
#pragma unroll
        for (int j4 = 0; j4 < S::kLaneRows; j4 += 4) {
          const uint4 off = *reinterpret_cast<const uint4*>(&sm_rows[warp][kv][row0 + j4]);
#pragma unroll
          for (int j = j4; j < j4 + 4; ++j) {
            const bool on = in_dim && (mask >> (row0 + j) & 1);
            if (row0 + j != skip)
              cp_async16((dst ^ (swizzle(j) << 4)) + (kv * kWarpKeys + j) * S::kRowBytes,
                         on ? base + (&off.x)[j - j4] + piece : base, on ? 16u : 0u);
          }
        }
      }
      if (skip >= 0) {                                     // into the stage, and once into the cache's slot
#pragma unroll
        for (int i = 0; i < kFresh; ++i) {
          const int kv = (lane + 32 * i) / S::kCols, c = (lane + 32 * i) % S::kCols;
          if (kv < 2) {
            *reinterpret_cast<uint4*>(smem + warp * (S::kStages * S::kStageBytes) + s * S::kStageBytes +
                                      (kv * kWarpKeys + skip) * S::kRowBytes + ((c ^ swizzle(skip)) << 4)) = fresh[i];
            if (c * 8 < p.head_dim && put.h % a.row_blocks == 0)
              static_cast<uint4*>(kv ? p.v_cache : p.k_cache)[sm_rows[warp][kv][skip] + c] = fresh[i];
          }
        }
      }
    }
    __syncwarp();                                          // sm_rows is free again
  };
  if (!in_dim) {                                           // columns past head_dim stay zero
    for (int s = 0; s < S::kStages; ++s)
      for (int j = 0; j < 2 * kWarpKeys; ++j)
        if (j % kWarpKeys / S::kLaneRows == row0 / S::kLaneRows)
          *reinterpret_cast<uint4*>(smem + warp * (S::kStages * S::kStageBytes) + s * S::kStageBytes + j * S::kRowBytes +
                                    ((piece ^ swizzle(j)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
  }
  fetch_page();
  auto produce = [&](int s, int pos) {                     // one tile into stage s, the fifo's place pos
    if (put.u < limit) {
      issue(s, pos);
      if (put.advance(a)) put_hk = put.h / a.row_blocks;
      if (put.u < limit) fetch_page();
    }
    cp_commit();
  };
#pragma unroll
  for (int s = 0; s < S::kStages; ++s) produce(s, s);

  // ---- the consumer: queries, running maximum and sum (log2 units) of rows g and g + 8, accumulator
  uint32_t q[R][S::kBlocks * 4];
  float m[R], l[R], o[S::kCols][4];
  auto rows_of = [&](int h) {                              // live query rows of item h
    const int r = a.group - (h % a.row_blocks) * kMaxRows;
    return r < kMaxRows ? r : kMaxRows;
  };
  auto q_head = [&](int h) { return (h / a.row_blocks) * a.group + (h % a.row_blocks) * kMaxRows; };
  auto load_q = [&]() {
    const T* qp = static_cast<const T*>(p.q) + get.b * p.q_batch + static_cast<long long>(q_head(get.h)) * p.head_dim;
    const int rows = rows_of(get.h);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int blk = 0; blk < S::kBlocks; ++blk) {
        const int row = g + 8 * r, d = 32 * blk + 8 * t;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (row < rows && d < p.head_dim) v = __ldg(reinterpret_cast<const uint4*>(qp + row * p.head_dim + d));
        q[r][4 * blk] = v.x; q[r][4 * blk + 1] = v.y; q[r][4 * blk + 2] = v.z; q[r][4 * blk + 3] = v.w;
      }
  };
  auto clear = [&]() {
#pragma unroll
    for (int r = 0; r < R; ++r) m[r] = -CUDART_INF_F, l[r] = 0.f;
#pragma unroll
    for (int i = 0; i < S::kCols; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[i][c] = 0.f;
  };
  // this lane's k piece of key g: blocks 2 i and 2 i + 1 at k_at[0] and k_at[1] + 128 i; its ldmatrix
  // row: v tiles 8 i + 2 x and 8 i + 2 x + 1 at v_at[x] + 128 i
  uint32_t k_at[2], v_at[4];
#pragma unroll
  for (int x = 0; x < 2; ++x) k_at[x] = ring + g * S::kRowBytes + ((t ^ swizzle(g) ^ (4 * x)) << 4);
#pragma unroll
  for (int x = 0; x < 4; ++x)
    v_at[x] = ring + (kWarpKeys + (lane & 15)) * S::kRowBytes + (((lane >> 4) ^ swizzle(lane & 7) ^ (2 * x)) << 4);

  auto compute = [&](int s, unsigned mask) {
    const uint32_t at = s * S::kStageBytes;
    float sc[2][4] = {};
#pragma unroll
    for (int blk = 0; blk < S::kBlocks; ++blk) {
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const uint4 v = lds128(k_at[blk & 1] + at + (blk >> 1) * 128 + nt * 8 * S::kRowBytes);
        mma(sc[nt], q[0][4 * blk], R == 2 ? q[R - 1][4 * blk] : 0u, q[0][4 * blk + 1], R == 2 ? q[R - 1][4 * blk + 1] : 0u,
            v.x, v.y, T());
        mma(sc[nt], q[0][4 * blk + 2], R == 2 ? q[R - 1][4 * blk + 2] : 0u, q[0][4 * blk + 3],
            R == 2 ? q[R - 1][4 * blk + 3] : 0u, v.z, v.w, T());
      }
    }
    uint32_t pa[2][2], rest[R][2];                         // [row block][key half]: the A fragment of p v
    bool moved = false;
    float alpha[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = 8 * (i >> 1) + 2 * t + (i & 1);
        x[i] = sc[i >> 1][2 * r + (i & 1)] * a.scale_log2;
        if (mask != 0xFFFFu && !(mask >> key & 1)) x[i] = -CUDART_INF_F;
      }
      float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      const float mn = fmaxf(m[r], top), base = mn == -CUDART_INF_F ? 0.f : mn, low = base - kLift;
      alpha[r] = exp2f(m[r] - base);
      moved |= mn != m[r];
      m[r] = mn;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = exp2f(x[i] - low);
      l[r] = l[r] * alpha[r] + ((x[0] + x[1]) + (x[2] + x[3]));
      // below p whichever way it rounds, by u = 2^-8 (bf16) or 2^-11 (fp16) of itself at most: for u taken off
      // p (1 - u) (1 + u / (1 + u)) = p (1 - 2 u^2 / (1 + u))
      constexpr float kLess = std::is_same<T, __half>::value ? 1.f - 1.f / 1024.f : 1.f - 1.f / 256.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t h = pack2(x[2 * i] * kLess, x[2 * i + 1] * kLess, T());
        pa[r][i] = h;
        rest[r][i] = pack2(x[2 * i] - Tr::to_f32(Tr::from_bits(lo16(h))), x[2 * i + 1] - Tr::to_f32(Tr::from_bits(hi16(h))), T());
      }
    }
    if (R == 1) pa[1][0] = rest[0][0], pa[1][1] = rest[0][1];
    if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
      for (int i = 0; i < S::kCols; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[i][c] *= alpha[R == 2 ? c >> 1 : 0];
    }
#pragma unroll
    for (int i = 0; i < S::kCols; i += 2) {                // keys 0..7 and 8..15 of two column tiles
      uint32_t v[4];
      ldsm4_trans(v, v_at[(i >> 1) & 3] + at + (i >> 3) * 128);
      mma(o[i], pa[0][0], pa[1][0], pa[0][1], pa[1][1], v[0], v[1], T());
      mma(o[i + 1], pa[0][0], pa[1][0], pa[0][1], pa[1][1], v[2], v[3], T());
      if (R == 2) {
        mma(o[i], rest[0][0], rest[R - 1][0], rest[0][1], rest[R - 1][1], v[0], v[1], T());
        mma(o[i + 1], rest[0][0], rest[R - 1][0], rest[0][1], rest[R - 1][1], v[2], v[3], T());
      }
    }
  };

  // The item's keys of this run are done: the 4 warps join, and the result or a partial is written.
  // (b, h): the item; the cursor may already be at the next one.  Thread (warp w, lane (g, t)) sums,
  // for row g of a block of 8, column tiles w kMine .. of the 4 warps' accumulators.
  constexpr int kMine = S::kCols / kWarps;
  float* const merge = reinterpret_cast<float*>(smem + S::kRing);
  auto close_item = [&](int b, int h, long long tiles_begin, long long tiles_end) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 1);
      l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 2);
      if (t == 0) {
        sm_m[warp][g + 8 * r] = m[r];
        sm_l[warp][g + 8 * r] = l[r];
      }
    }
    __syncthreads();
    const bool whole = tiles_begin >= begin && tiles_end <= end;
    // part of an item: runs first .. last hold it; the first leaves its part in its slot 1, the
    // others in slot 0
    const int first = whole ? run : run_of(tiles_begin), last = whole ? run : run_of(tiles_end - 1);
    auto slot_of = [&](int r) { return a.partials + (static_cast<size_t>(r) * 2 + (r == first ? 1 : 0)) * partial_floats(DP); };
    const int rows = rows_of(h);
    auto write = [&](int r, float M, float L, const float (&sum)[kMine][2]) {
      const int row = g + 8 * r;
      if (row >= rows) return;
      const long long at = static_cast<long long>(b) * p.heads + q_head(h) + row;
      const float inv = L > 0.f || isnan(L) ? 1.f / L : 0.f;
      T* out = static_cast<T*>(p.out) + at * p.head_dim;
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int d = (warp * kMine + i) * 8 + 2 * t;
        if (d < p.head_dim) *reinterpret_cast<uint32_t*>(out + d) = pack2(sum[i][0] * inv, sum[i][1] * inv, T());
      }
      if (p.lse && warp == 0 && t == 0) p.lse[at] = M * 0.693147180559945f + logf(L * (1.f / 32768.f));   // 2^-kLift
    };
    float M[R], L[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      M[r] = -CUDART_INF_F;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M[r] = fmaxf(M[r], sm_m[w][g + 8 * r]);
      const float base = M[r] == -CUDART_INF_F ? 0.f : M[r];
      L[r] = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) L[r] += sm_l[w][g + 8 * r] * exp2f(sm_m[w][g + 8 * r] - base);
      const float f = exp2f(m[r] - base);
      if (r) __syncthreads();                              // the block before has been read
      // every warp hands the column tiles that others sum to them, and keeps its own
      float sum[kMine][2];
#pragma unroll
      for (int i = 0; i < S::kCols; ++i) {
        const float2 v = R == 2 ? make_float2(o[i][2 * r] * f, o[i][2 * r + 1] * f)
                                : make_float2((o[i][0] + o[i][2]) * f, (o[i][1] + o[i][3]) * f);
        const int owner = i / kMine, from = (warp - owner + kWarps - 1) % kWarps;   // 0 .. 2, 3 for the owner
        if (warp == owner) {
          sum[i % kMine][0] = v.x;
          sum[i % kMine][1] = v.y;
        } else {
          *reinterpret_cast<float2*>(merge + ((i * (kWarps - 1) + from) * 32 + lane) * 2) = v;
        }
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kMine; ++i)
#pragma unroll
        for (int w = 0; w < kWarps - 1; ++w) {
          const float2 x = *reinterpret_cast<const float2*>(merge + (((warp * kMine + i) * (kWarps - 1) + w) * 32 + lane) * 2);
          sum[i][0] += x.x;
          sum[i][1] += x.y;
        }
      if (whole) {
        write(r, M[r], L[r], sum);
      } else {
        // [row block][pair of column tiles][lane]: 4 floats; then (m, l) of each row
        float* to = slot_of(run);
        if (g + 8 * r < rows) {
#pragma unroll
          for (int i = 0; i < kMine; i += 2)
            __stcg(reinterpret_cast<float4*>(to + r * 8 * DP) + (warp * kMine + i) / 2 * 32 + lane,
                   make_float4(sum[i][0], sum[i][1], sum[i + 1][0], sum[i + 1][1]));
          if (warp == 0 && t == 0) __stcg(reinterpret_cast<float2*>(to + kMaxRows * DP) + g + 8 * r, make_float2(M[r], L[r]));
        }
      }
    }
    if (whole) return;
    __syncthreads();
    // the counter wraps to zero at the last arrival, ready for the next call; thread 0's fences stand
    // for the CTA (ordered with the other threads' accesses by the barriers)
    if (threadIdx.x == 0) {
      __threadfence();
      sm_last = atomicInc(a.counters + first, static_cast<unsigned>(last - first)) == static_cast<unsigned>(last - first);
      __threadfence();
    }
    __syncthreads();
    if (!sm_last) return;
    // the last arrival joins the parts in run order, a batch of them in flight at a time
    constexpr int kBatch = DP == 256 ? 3 : 8;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (g + 8 * r >= rows) continue;
      float top = -CUDART_INF_F, l_all = 0.f, sum[kMine][2] = {};
      for (int c0 = first; c0 <= last; c0 += kBatch) {
        float2 ml[kBatch];
        float4 x[kBatch][kMine / 2];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const float* from = slot_of(c0 + j <= last ? c0 + j : last);
          ml[j] = ldcg2(from + kMaxRows * DP + 2 * (g + 8 * r));
#pragma unroll
          for (int i = 0; i < kMine / 2; ++i) x[j][i] = ldcg4(from + r * 8 * DP + ((warp * kMine / 2 + i) * 32 + lane) * 4);
        }
        float mn = top;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) mn = fmaxf(mn, ml[j].x);   // (a repeated last part changes nothing)
        const float base = mn == -CUDART_INF_F ? 0.f : mn, keep = exp2f(top - base);
        top = mn;
        l_all *= keep;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          sum[i][0] *= keep;
          sum[i][1] *= keep;
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          if (c0 + j <= last) {
            const float f = exp2f(ml[j].x - base);
            l_all += ml[j].y * f;
#pragma unroll
            for (int i = 0; i < kMine / 2; ++i) {
              sum[2 * i][0] += x[j][i].x * f;
              sum[2 * i][1] += x[j][i].y * f;
              sum[2 * i + 1][0] += x[j][i].z * f;
              sum[2 * i + 1][1] += x[j][i].w * f;
            }
          }
        }
      }
      write(r, top, l_all, sum);
    }
  };

  load_q();
  clear();
  int stage = 0;
  while (get.u < limit) {
    cp_wait<S::kStages - 1>();
    __syncwarp();                                          // every lane's copies of the stage have landed
    const unsigned mask = static_cast<unsigned>(live & 0xFFFFu);
    if (mask) compute(stage, mask);
    live >>= 16;
    __syncwarp();                                          // every lane has read the stage
    produce(stage, S::kStages - 1);
    stage = stage + 1 == S::kStages ? 0 : stage + 1;
    const int b = get.b, h = get.h;
    const long long tiles_end = tiles_begin + get.nt;
    const bool next = get.advance(a), more = get.u < limit;
    if (next || !more) {
      if (more) load_q();                                  // on its way while the warps join
      close_item(b, h, tiles_begin, tiles_end);
      if (more) clear();
      tiles_begin = tiles_end + kItemUnits;
    }
  }
  cp_wait<0>();
}

template <typename T, int DP, int R>
cudaError_t launch(const Args& a, cudaStream_t stream) {
  using S = Shape<DP, R>;
  auto kern = k_attention<T, DP, R>;
  const DeviceInfo& dev = device_info();
  static std::atomic<unsigned long long> opted_in{0};       // per device
  if (dev.device >= 64 || !(opted_in.load(std::memory_order_relaxed) & (1ull << dev.device))) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(S::kSmem));
    if (e != cudaSuccess) return e;
    if (dev.device < 64) opted_in.fetch_or(1ull << dev.device, std::memory_order_relaxed);
  }
  int grid = dev.sm_count * S::kCtas;
  if (grid > kMaxCtas) grid = kMaxCtas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <typename T, int DP>
cudaError_t launch_rows(const Args& a, cudaStream_t stream) {
  return a.group <= 8 ? launch<T, DP, 1>(a, stream) : launch<T, DP, 2>(a, stream);
}

template <typename T>
cudaError_t launch_dim(const Args& a, cudaStream_t stream) {
  if (a.p.head_dim <= 64) return launch_rows<T, 64>(a, stream);
  if (a.p.head_dim <= 128) return launch_rows<T, 128>(a, stream);
  return launch_rows<T, 256>(a, stream);
}

}  // namespace attention

size_t attention_workspace_bytes(int, int, int head_dim) {
  const int dp = head_dim <= 64 ? 64 : (head_dim <= 128 ? 128 : 256);
  return attention::kControlBytes + static_cast<size_t>(attention::kMaxCtas) * 2 * attention::partial_floats(dp) * 4;
}

cudaError_t launch_paged_attention(const AttentionProblem& p, cudaStream_t stream) {
  attention::Args a;
  a.p = p;
  a.group = p.heads / p.kv_heads;
  a.row_blocks = (a.group + attention::kMaxRows - 1) / attention::kMaxRows;
  a.items = p.kv_heads * a.row_blocks;
  a.scale_log2 = p.scale * 1.44269504088896341f;
  // m = ceil(2^(30 + L) / d) with 2^L >= d: n m / 2^(30 + L) is off by less than 1 / d for n < 2^30
  unsigned log = 0;
  while ((1ull << log) < static_cast<unsigned>(p.page_size)) ++log;
  a.page_shift = 30 + log;
  a.page_mul = static_cast<unsigned>(((1ull << a.page_shift) + p.page_size - 1) / p.page_size);
  a.k_page16 = static_cast<unsigned>(p.k_page / 8);
  a.k_slot16 = static_cast<unsigned>(p.k_slot / 8);
  a.k_head16 = static_cast<unsigned>(p.k_head / 8);
  a.v_page16 = static_cast<unsigned>(p.v_page / 8);
  a.v_slot16 = static_cast<unsigned>(p.v_slot / 8);
  a.v_head16 = static_cast<unsigned>(p.v_head / 8);
  a.counters = static_cast<unsigned*>(p.workspace);
  a.partials = reinterpret_cast<float*>(static_cast<char*>(p.workspace) + attention::kControlBytes);
  return p.dtype == 0 ? attention::launch_dim<__half>(a, stream) : attention::launch_dim<__nv_bfloat16>(a, stream);
}

}  // namespace gptq
