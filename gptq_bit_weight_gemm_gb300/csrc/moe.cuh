// moe.cuh -- the expert products of the mixture-of-experts layer (gptq_moe) for up to 32 tokens.
//
// An expert's rows are taken in blocks of 8 NB; a block, with its expert, is a slot.
//
// Three launches after the router's (moe.cu, which leaves the logits): UP writes h = silu(x Wg) * (x Wu) for every
// (expert, token) row, DOWN out[t] = sum over t's experts of w * (h Wd), in parts that the third adds
// (k_sum_parts).  UP and DOWN are a stream of packed weights -- those of the chosen experts, each read once --
// against a few activations.  HBM is their floor; what they take more goes to the instructions that unpack,
// multiply and fold, to the ends of items and to the chain of launches.  One kernel template runs both.
//
// Split: a call's work is a line of chunks (32 columns x 8 warps wide, kRows packed rows deep).  UP's
// items are (expert, 128 gate and the same 128 up columns), DOWN's are 256 output columns, whose line
// runs through all experts one after the other, so that the sum over experts stays in the CTA and needs
// no atomics.  The line is cut into equal runs, one per resident CTA, whatever the experts the tokens
// chose; an item that spans runs leaves one partial tile per run in the workspace.  UP's are added in run
// order by the last CTA to arrive, DOWN's by k_sum_parts.
//
// A CTA is one producer warp and 8 consumer warps around a ring of chunks.  Two CTAs share an SM, so that
// one computes while the other writes an item: one CTA of 16 or 24 consumer warps took 75 and 83 us for
// one token against 62, three CTAs 67.  The producer copies a
// chunk's weights (one or two TMA boxes of slots of 32 columns with the 128-byte swizzle), its rows of
// activations and its groups' scales and zeros (cp.async), all arriving on one mbarrier.  (A box for
// each 32 columns and a bulk copy for each row cost the producer about 100 cycles each, which bounded
// everything: one token 83 us.)  A consumer warp owns 32 columns and multiplies on the tensor cores (m16n8k16, weights as
// the A operand).  Unpacking is what the SM runs out of first.  A code masked into the low mantissa bits of
// a half, s bits up, reads as the subnormal q 2^(s - 24), and one fma with 2^(14 - s) and -z 2^-10 makes
// it (q - z) 2^-10, exactly: 9 operations per word of 8 codes.  (Without the fma, with the zero taken off
// per group as sum q a - z sum a, a group whose codes equal its zero would leave the fp32 error of two
// sums of up to 255 |a| where the result is 0: 0.2 at 8 bits with outlier channels.)
//
// Activations are fp16 in both stages: every row's run of 128 values is stored as fp16 times a power
// of two chosen for the run (11 bits of each value above 2^-28 of the run's largest; exact for fp16 and
// bf16 input in that range), already in the pair order of the codes.  So h may exceed fp16's range, and
// bf16 models lose nothing to the multiply.  Where the output is fp16 too, 11 bits of h would show in it
// (relative error 2.9e-4 against the 2.1e-4 of the output's own rounding), so h goes in two parts there,
// its rounding and what the rounding left: as two rows of the products, free where a block of 8 rows has
// room for them, or multiplied one after the other (TWICE).
#pragma once

#include <cuda.h>

#include <atomic>

#include "decode_mma.cuh"
#include "serving_internal.h"

namespace gptq {
namespace moe {

constexpr int kWarps = 8, kConsumers = kWarps * 32, kThreads = kConsumers + 32;
constexpr int kCols = kWarps * 32;       // columns of a CTA's tile
constexpr int kRun = 128;                // activations that share a power of two
constexpr int kMaxRuns = 480;            // CTAs, at most
constexpr int kItemUnits = 2;            // what opening and writing an item takes, in chunks
constexpr int kMinShare = 2;             // chunks and units of a run, at least (5 tokens on 6 small experts: 23 us; 4: 27, 8: 36)
constexpr int kMaxStages = 12;

constexpr int kCtas = 2;                 // on an SM

template <int BITS>
struct Chunk {
  static constexpr int kTiles = BITS == 3 ? 1 : 4;                        // k-tiles
  static constexpr int kTileK = 4 * Pack<BITS>::kPerUnit;                 // k values of a k-tile
  static constexpr int kK = kTiles * kTileK;
  static constexpr int kRows = kTiles * 4 * Pack<BITS>::kRowsPerUnit;     // packed rows
  static constexpr int kSlot = kRows * 128;                               // one warp's 32 columns
  static constexpr int kRunsOf = (kK + kRun - 1) / kRun;                  // activation runs of a chunk
  // bytes of an activation row in the ring: padded so that the B fragments of 4 units and 8 rows
  // fall into distinct banks
  static constexpr int kActRow = kK * 2 + (BITS == 4 ? 64 : BITS == 8 ? 32 : 16);
  static constexpr int kZeroWords = kWarps * BITS;                        // zeros of 256 columns
  static constexpr int kInfo = kRunsOf;                                   // floats per row: run scales
  // tiles that share a run of activations (and a group, where groups are multiples of their length)
  static constexpr int kSegTiles = kTileK * kTiles < kRun ? kTiles : kRun / kTileK;
  static constexpr int kSegK = kSegTiles * kTileK;
};

// The routing of a call in shared memory: every CTA derives it from the logits (identical in all of
// them), so that no index ever comes from memory another CTA had to write first.
struct Routing {
  int* id;               // [pairs] expert of (token, choice)
  float* w;              // [pairs] its weight
  int* count;            // [experts] rows, then first row
  int* slot_expert;      // [slots] chosen experts in order, as often as they have blocks of rows
  int* slot_off;         // [slots + 1] their rows: [slot_off[s], slot_off[s + 1])
  int* row_token;        // [pairs] rows by expert, an expert's by token
  float* row_weight;
  __host__ __device__ static int most_slots(int pairs, int experts) {
    return (pairs < experts ? pairs : experts) + pairs / 4;   // (4 rows a slot at least, unless there are fewer)
  }
  __host__ __device__ static int bytes(int pairs, int experts) {
    return (16 * pairs + 4 * experts + 8 * most_slots(pairs, experts) + 4 + 15) & ~15;
  }
};

struct Args {
  int K, N, group, G, zero_offset, zwords, units;
  const int32_t* qzeros;
  const __half* scales;
  int tokens;
  int rows;              // of a slot, at most
  int parts;             // fp16 rows of a row's activations: 1, or 2 (DOWN)
  int ring_rows;         // of the ring's activation part: rows * parts
  int h_parts;           // UP: DOWN's parts
  int experts, topk, renormalize;
  const float* logits;   // [tokens][experts]
  int32_t* ids;          // UP, nullable: the caller's copies
  float* weights;
  const __half* act;     // UP: [tokens][K] in pair order; DOWN: [rows][parts][K]
  const float* act_scale;   // [row][act_runs]
  int act_runs;
  int jblocks;           // column blocks: UP ceil(inter / 128), DOWN ceil(hidden / 256)
  int inter;
  __half* h;             // UP
  float* h_scale;
  int h_runs;
  void* out;             // DOWN
  int dtype;
  int* slots;            // DOWN: the number of chosen experts, for the sum of the parts
  unsigned* counters;    // UP
  float* partials;
  unsigned* status;
  int stages, gmax, stage_bytes;
};

// Position of value k of a unit among its halfwords.
template <int BITS>
__device__ __forceinline__ int pair_pos(int k) {
  if constexpr (BITS == 3) {
    int at = 0;
#pragma unroll
    for (int p = 0; p < 16; ++p) {
      if (code3_pair(p, 0) == k) at = 2 * p;
      if (code3_pair(p, 1) == k) at = 2 * p + 1;
    }
    return at;
  } else {
    constexpr int half = Pack<BITS>::kPerUnit / 2;
    return k < half ? 2 * k : 2 * (k - half) + 1;
  }
}

// How far up (bits) the code at halfword `pos` of a unit sits in its half once masked (ScaledPairs).
template <int BITS>
__host__ __device__ constexpr int pair_shift(int pos) {
  const int p = pos >> 1;
  if (BITS == 2) return 2 * (p & 3);
  if (BITS == 4) return 4 * (p & 1);
  if (BITS == 3) return pos & 1 ? CodePairs<__half, 3>::shift_hi(p) : CodePairs<__half, 3>::shift_lo(p);
  return 0;
}

// fp16 bits of (2^(14 - s), 2^(14 - s')), s and s' the shifts of pair p's codes
template <int BITS>
__host__ __device__ constexpr uint32_t pair_scale(int p) {
  return static_cast<uint32_t>(29 - pair_shift<BITS>(2 * p)) << 10 | static_cast<uint32_t>(29 - pair_shift<BITS>(2 * p + 1)) << 26;
}
// -z 2^-10 in both halves: z as a subnormal, z 2^-24, times -2^14
__device__ __forceinline__ uint32_t zero_pair(uint32_t z) { return fma2(z * 0x00010001u, 0xF400F400u, 0x80008000u, __half()); }

// (q - z) 2^-10 of the codes of a unit as pairs of halves, in DiffPairs' order; zero: zero_pair(z).
template <int BITS>
struct ScaledPairs {
  static constexpr int kPairs = 16 / BITS;
  __device__ static __forceinline__ void run(uint32_t w, uint32_t zero, uint32_t (&d)[kPairs]) {
    constexpr uint32_t mask = Pack<BITS>::kMask * 0x00010001u;
    constexpr int low = 8 / BITS;                          // pairs below bit 8
#pragma unroll
    for (int p = 0; p < low; ++p) {
      d[p] = fma2(w & (mask << (BITS * p)), pair_scale<BITS>(p), zero, __half());
      d[low + p] = fma2((w >> 8) & (mask << (BITS * p)), pair_scale<BITS>(low + p), zero, __half());
    }
  }
};
template <>
struct ScaledPairs<3> {
  static constexpr int kPairs = 16;
  __device__ static __forceinline__ void run3(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t zero, uint32_t (&d)[kPairs]) {
    const uint32_t x[9] = {w0, w0 >> 4, __funnelshift_r(w0, w1, 10), w1, w1 >> 3, w1 >> 6, __funnelshift_r(w1, w2, 26), w2, w2 >> 6};
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
      const int s = code3_pair(p, 2);
      const int xi = s == 0 ? 0 : s == 4 ? 1 : s == 10 ? 2 : s == 32 ? 3 : s == 35 ? 4 : s == 38 ? 5 : s == 58 ? 6 : s == 64 ? 7 : 8;
      d[p] = fma2(x[xi] & ((7u << CodePairs<__half, 3>::shift_lo(p)) | (7u << (16 + CodePairs<__half, 3>::shift_hi(p)))), pair_scale<3>(p), zero, __half());
    }
  }
};

// The power of two (as its exponent) that takes a run's largest magnitude to [2^14, 2^15).
__device__ __forceinline__ int run_exponent(float largest) {
  int e = largest > 0.f ? static_cast<int>(__float_as_uint(largest) >> 23) - 127 - 14 : 0;
  return e < -126 ? -126 : (e > 126 ? 126 : e);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<unsigned>(e + 127) << 23); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int x, int y, int z, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory"); }

// One warp stores a run of a row: lane l holds values 4 l .. 4 l + 3 (zeros past K).  act: the row, or in
// two parts the two rows of its roundings and of what they left; the run's power of two goes to *scale.
template <int BITS>
__device__ __forceinline__ void store_run(const float (&v)[4], int j0, int K, int parts, __half* act, float* scale) {
  constexpr int per = Pack<BITS>::kPerUnit;
  const int lane = threadIdx.x & 31, j = j0 + 4 * lane;
  float top = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  const int e = run_exponent(top);
  const float inv = pow2(-e);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = (j + i) / per * per + pair_pos<BITS>((j + i) % per);
    const __half x = __float2half_rn(v[i] * inv);
    if (j < K) {
      act[at] = x;
      if (parts == 2) act[K + at] = __float2half_rn(v[i] * inv - __half2float(x));
    }
  }
  if (lane == 0) *scale = pow2(e);
}

// Loads from shared memory by 32-bit address (a generic pointer costs 64-bit additions in the main loop);
// volatile, so that none moves ahead of the wait for its stage.
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

// Not volatile: the products of one k-tile move freely among the loads and unpacking of the next.
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Shared memory: [stages][weights | activations | their scales | group scales | group zeros], the
// output tile [tokens (DOWN) or rows][kCols] floats, 2 mbarriers per stage, the routing.
template <int BITS>
struct Layout {
  using C = Chunk<BITS>;
  __host__ __device__ static constexpr int act() { return kWarps * C::kSlot; }
  __host__ __device__ static int info(int rows) { return act() + rows * C::kActRow; }
  __host__ __device__ static int scales(int rows) { return (info(rows) + rows * C::kInfo * 4 + 15) & ~15; }
  __host__ __device__ static int zeros(int rows, int gmax) { return scales(rows) + gmax * kCols * 2; }
  __host__ __device__ static int stage(int rows, int gmax) {
    return (zeros(rows, gmax) + gmax * C::kZeroWords * 4 + 1023) & ~1023;
  }
  __host__ __device__ static int tile_bytes(int rows) { return rows * kCols * 4; }
  // less the stages and their mbarriers
  __host__ __device__ static int fixed(int tile_rows, int pairs, int experts) {
    return 1024 + tile_bytes(tile_rows) + Routing::bytes(pairs, experts);
  }
};

__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned* status) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer();
  while (true) {
    if (ptx::mbar_try_wait_hint(bar, parity, 100000u)) return true;
    if (*abort_flag) return false;
    if (ptx::globaltimer() - t0 > 2000000000ull) {
      *abort_flag = 1;
      atomicOr(status, kStatusTimeout);
      return false;
    }
  }
}

// Order-preserving bits of a logit, never 0; a NaN as -inf, -0 as 0.
__device__ __forceinline__ unsigned key_of(float v) {
  const unsigned b = __float_as_uint(isnan(v) ? __int_as_float(0xFF800000) : v + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(unsigned key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// Softmax, top-k (equal logits: the lower index; a NaN ranks as -inf) and grouping by expert, by the
// whole CTA; returns the number of chosen experts.  scratch: a row of `experts` floats per warp.
__device__ __forceinline__ int route(const Args& a, const Routing& r, float* scratch, int* scan, bool publish) {
  constexpr int kAll = kThreads / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float inf = __int_as_float(0x7F800000);
  for (int e = threadIdx.x; e < a.experts; e += kThreads) r.count[e] = 0;
  for (int t = warp; t < a.tokens; t += kAll) {
    // keys order the logits (a NaN as -inf); 0 marks absent and taken ones.  Up to kHeld experts a lane stay
    // in registers, more in shared memory.
    constexpr int kHeld = 4;
    const float* logits = a.logits + t * a.experts;
    float* row = scratch + warp * a.experts;
    const bool held = a.experts <= 32 * kHeld;
    unsigned key[kHeld];
    float m = -inf, sum = 0.f, kept = 0.f, mine = 0.f;
    if (held) {
      float v[kHeld];
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        v[i] = lane + 32 * i < a.experts ? __ldcg(logits + lane + 32 * i) : -inf;
        m = fmaxf(m, v[i]);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        const bool in = lane + 32 * i < a.experts;
        if (in) sum += expf(v[i] - m);
        key[i] = in ? key_of(v[i]) : 0u;
      }
    } else {
      for (int e = lane; e < a.experts; e += 32) {
        const float v = __ldcg(logits + e);
        row[e] = v;
        m = fmaxf(m, v);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      for (int e = lane; e < a.experts; e += 32) {
        sum += expf(row[e] - m);
        row[e] = __uint_as_float(key_of(row[e]));
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    // topk times the largest key, its lowest index first
    for (int j = 0; j < a.topk; ++j) {
      unsigned bk = 0u;
      int be = 0x7FFFFFFF;
      if (held) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
          if (key[i] > bk) {
            bk = key[i];
            be = lane + 32 * i;
          }
      } else {
        for (int e = lane; e < a.experts; e += 32) {
          const unsigned k = __float_as_uint(row[e]);
          if (k > bk) {
            bk = k;
            be = e;
          }
        }
      }
      const unsigned top = __reduce_max_sync(0xFFFFFFFFu, bk);
      be = __reduce_min_sync(0xFFFFFFFFu, bk == top ? be : 0x7FFFFFFF);
      const float pr = expf(logit_of(top) - m) / sum;
      kept += pr;
      if (lane == j) mine = pr;
      if (lane == 0) r.id[t * a.topk + j] = be;
      if (held) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
          if (be == lane + 32 * i) key[i] = 0u;
      } else {
        if (lane == (be & 31)) row[be] = 0.f;
        __syncwarp();
      }
    }
    if (a.renormalize) mine /= kept;
    if (lane < a.topk) r.w[t * a.topk + lane] = mine;
  }
  __syncthreads();
  // a pair's place among its expert's rows: warp 0 takes the pairs in order, 32 at a time
  const int pairs = a.tokens * a.topk;
  int* rank = reinterpret_cast<int*>(scratch);
  if (warp == 0) {
    for (int p0 = 0; p0 < pairs; p0 += 32) {
      const int p = p0 + lane, e = p < pairs ? r.id[p] : 0x7FFFFFFF;
      const unsigned same = __match_any_sync(0xFFFFFFFFu, e);
      const int before = __popc(same & ((1u << lane) - 1u));
      if (p < pairs) {
        const int base = r.count[e];
        rank[p] = base + before;
        if (publish && a.ids) a.ids[p] = e;
        if (publish && a.weights) a.weights[p] = r.w[p];
      }
      __syncwarp();
      if (p < pairs && before == 0) r.count[e] += __popc(same);
      __syncwarp();
    }
  }
  __syncthreads();
  // experts with rows, in order: a scan of (blocks, rows), a CTA's threads at a time
  int slots = 0, rows = 0;
  for (int e0 = 0; e0 < a.experts; e0 += kThreads) {
    const int e = e0 + static_cast<int>(threadIdx.x), n = e < a.experts ? r.count[e] : 0;
    const int mine = n | (n + a.rows - 1) / a.rows << 16;  // rows, and blocks of them
    int c = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, c, o);
      if (lane >= o) c += v;
    }
    if (lane == 31) scan[warp] = c;
    __syncthreads();
    int at = c - mine;
    for (int w = 0; w < kAll; ++w) {
      if (w < warp) at += scan[w];
    }
    at += slots << 16 | rows;
    for (int w = 0; w < kAll; ++w) {
      slots += scan[w] >> 16;
      rows += scan[w] & 0xFFFF;
    }
    if (n > 0) {
      const int off = at & 0xFFFF;
      int s = at >> 16;
      for (int m = 0; m < n; m += a.rows, ++s) {
        r.slot_expert[s] = e;
        r.slot_off[s] = off + m;
      }
      r.count[e] = off;
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) r.slot_off[slots] = rows;
  for (int p = threadIdx.x; p < pairs; p += kThreads) {
    const int at = r.count[r.id[p]] + rank[p];
    r.row_token[at] = p / a.topk;
    r.row_weight[at] = r.w[p];
  }
  ptx::fence_proxy_async_smem();                           // the scratch lies where the ring's copies will land
  __syncthreads();
  return slots;
}

// A line of `total` units cut into runs of `share`, the first `extra` of them one longer.
struct Line {
  int runs, share, extra;
  __device__ __forceinline__ Line(long long total, int grid) {
    const long long want = total / kMinShare;
    runs = want < 1 ? 1 : (want < grid ? static_cast<int>(want) : grid);
    share = static_cast<int>(total / runs);
    extra = static_cast<int>(total - static_cast<long long>(share) * runs);
  }
  __device__ __forceinline__ long long begin(int run) const { return static_cast<long long>(share) * run + (run < extra ? run : extra); }
  __device__ __forceinline__ int length(int run) const { return share + (run < extra ? 1 : 0); }
  __device__ __forceinline__ int run_of(long long u) const {
    const long long cut = static_cast<long long>(extra) * (share + 1);
    return static_cast<int>(u < cut ? u / (share + 1) : extra + (u - cut) / share);
  }
};

// A place on the line: u units after the run's begin, chunk c of the item, which is chunk kc of slot s.
struct Cursor {
  int u, item, c, s, kc;
};

// TWICE: the activations' two parts are multiplied one after the other into the same sums, instead of as two
// rows.
template <int BITS, int NB, bool DOWN, bool TWICE>
__global__ void __launch_bounds__(kThreads, kCtas) k_experts(const __grid_constant__ CUtensorMap tmW, const Args a) {
  using P = Pack<BITS>;
  using C = Chunk<BITS>;
  using L = Layout<BITS>;
  using RP = ScaledPairs<BITS>;
  constexpr int NP = RP::kPairs, ROWS = P::kRowsPerUnit;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  __shared__ int sm_abort, sm_last, sm_scan[kThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  uint8_t* smem = smem_raw + ((1024u - (ptx::smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t smem_a = ptx::smem_addr(smem);
  const int stage_bytes = a.stage_bytes;
  float* tile = reinterpret_cast<float*>(smem + a.stages * stage_bytes);
  const uint32_t bars = ptx::smem_addr(tile) + L::tile_bytes(DOWN ? a.tokens : a.rows);
  auto full = [&](int s) { return bars + 16u * s; };
  auto empty = [&](int s) { return bars + 16u * s + 8u; };
  Routing rt;
  {
    const int pairs = a.tokens * a.topk;
    rt.id = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(tile) + L::tile_bytes(DOWN ? a.tokens : a.rows) + 16 * a.stages);
    rt.w = reinterpret_cast<float*>(rt.id + pairs);
    rt.row_token = reinterpret_cast<int*>(rt.w + pairs);
    rt.row_weight = reinterpret_cast<float*>(rt.row_token + pairs);
    rt.count = reinterpret_cast<int*>(rt.row_weight + pairs);
    rt.slot_expert = rt.count + a.experts;
    rt.slot_off = rt.slot_expert + Routing::most_slots(pairs, a.experts);
  }
  // UP waits for the router's kernel and only then lets DOWN start; so the logits are final for DOWN from
  // its first instruction.  A DOWN CTA starts where a UP CTA has left its SM (either's ring takes half of it)
  // and streams its first weights while the last runs of UP end.
  if (!DOWN) decode::pdl_wait();
  decode::pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      ptx::mbar_init(full(s), 33);                         // the byte count's arrival and 32 lanes' cp.async
      ptx::mbar_init(empty(s), kWarps);
    }
    sm_abort = 0;
    ptx::fence_mbar_init();
  }
  // ---- this CTA's run.  All items of a call are equally long.
  const int slots = route(a, rt, reinterpret_cast<float*>(smem), sm_scan, !DOWN && blockIdx.x == 0);
  if (DOWN && blockIdx.x == 0 && threadIdx.x == 0) *a.slots = slots;   // (its run may hold no chunk)
  const int nk = (a.K + C::kK - 1) / C::kK;                // chunks of one expert's K
  const int per = DOWN ? slots * nk : nk;                  // chunks of an item
  const int items = DOWN ? a.jblocks : slots * a.jblocks;
  const Line line(static_cast<long long>(items) * (per + kItemUnits), gridDim.x);
  const int run = blockIdx.x;
  if (run >= line.runs) return;
  const long long begin = line.begin(run);
  const int limit = line.length(run);
  auto run_of = [&](long long u) { return line.run_of(u); };
  Cursor start;
  {
    start.item = static_cast<int>(begin / (per + kItemUnits));
    const int at = static_cast<int>(begin - static_cast<long long>(start.item) * (per + kItemUnits));
    start.c = at > kItemUnits ? at - kItemUnits : 0;
    start.u = at > kItemUnits ? 0 : kItemUnits - at;
    start.s = DOWN ? start.c / nk : start.item / a.jblocks;
    start.kc = DOWN ? start.c - start.s * nk : start.c;
  }
  if (start.u >= limit) return;                            // no chunk, only an item's extra units
  auto advance = [&](Cursor& x) {                          // true: a new item begins
    ++x.u;
    if (++x.c == per) {
      x.u += kItemUnits;
      ++x.item;
      x.c = x.kc = 0;
      x.s = DOWN ? 0 : x.item / a.jblocks;
      return true;
    }
    if (++x.kc == nk) {                                    // DOWN: the next expert
      x.kc = 0;
      ++x.s;
    }
    return false;
  };
  // first column (of the packed weight) of warp w's 32, or -1 past the end
  auto col_of = [&](int item, int w) {
    if (DOWN) {
      const int n = item * kCols + 32 * w;
      return n < a.N ? n : -1;
    }
    const int j = (item % a.jblocks) * (kCols / 2) + 32 * (w & 3);
    return j < a.inter ? (w < 4 ? j : a.inter + j) : -1;
  };

  if (warp == kWarps) {
    // ---------------------------------------------------------------- producer
    const uint64_t policy = ptx::policy_evict_first();     // weights are read once
    // Everything that changes with the item or the expert only is kept, and a chunk moves it on: with
    // the divisions in here the one producer warp took longer over a chunk than the consumers did
    // (one token, 4096 x 14336: 85 us).
    struct Put {
      Cursor x;
      int item, slot, rows, off, w_row, g, g_at;           // g: the chunk's first group, g_at: k of the chunk in it
      int block, sc_col, zc[2];                            // block: the item's first 32 columns
      const __half* sc;
      const int32_t* zr[2];
      const float* act_sc;
    };
    auto place = [&](Put& p) {                             // after a new item or expert
      if (p.item != p.x.item) {
        p.item = p.x.item;
        p.block = DOWN ? p.item * kWarps : (p.item % a.jblocks) * (kWarps / 2);
        p.sc_col = col_of(p.item, lane >> 2);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int w = lane + 32 * i;
          p.zc[i] = w < C::kZeroWords ? col_of(p.item, w / BITS) : -1;
        }
      }
      p.slot = p.x.s;
      const int expert = rt.slot_expert[p.slot], off = rt.slot_off[p.slot];
      p.off = off * a.parts;
      p.rows = (rt.slot_off[p.slot + 1] - off) * a.parts;
      const int k0 = p.x.kc * C::kK;
      p.g = k0 / a.group;
      p.g_at = k0 - p.g * a.group;
      p.w_row = expert * (a.units * ROWS) + p.x.kc * C::kRows;
      const long long grow = static_cast<long long>(expert) * a.G + p.g;
      p.sc = a.scales + grow * a.N + p.sc_col + 8 * (lane & 3);
#pragma unroll
      for (int i = 0; i < 2; ++i) p.zr[i] = a.qzeros + grow * a.zwords + p.zc[i] / 32 * BITS + (lane + 32 * i) % BITS;
      const int row = lane < p.rows ? (DOWN ? off + (a.parts == 2 ? lane >> 1 : lane) : rt.row_token[off + lane]) : 0;
      p.act_sc = a.act_scale + static_cast<long long>(row) * a.act_runs + k0 / kRun;
    };
    auto step = [&](Put& p) {                              // to the next chunk
      const int item = p.x.item, slot = p.x.s;
      advance(p.x);
      if (p.x.item != item || p.x.s != slot) {
        if (p.x.u < limit) place(p);
        return;
      }
      p.w_row += C::kRows;
      p.act_sc += C::kK >= kRun ? C::kRunsOf : 1 - (p.x.kc & 1);
      p.g_at += C::kK;
      while (p.g_at >= a.group) {
        p.g_at -= a.group;
        ++p.g;
        p.sc += a.N;
        p.zr[0] += a.zwords;
        p.zr[1] += a.zwords;
      }
    };
    static_assert(C::kK % kRun == 0 || 2 * C::kK == kRun, "a chunk is whole runs or half of one");
    // a chunk's weights, scales and zeros; then its activations
    auto put_weights = [&](const Put& p, int st) {
      const uint32_t to = smem_a + st * stage_bytes;
      const int left = a.K - p.x.kc * C::kK, ck = left < C::kK ? left : C::kK;
      if (lane == 0) {
        // box rows past the matrix and columns past its end arrive as zeros, and count
        ptx::mbar_arrive_expect_tx(full(st), kWarps * C::kRows * 128);
        tma_load_3d(to, &tmW, 0, p.w_row, p.block, full(st), policy);
        if (!DOWN) tma_load_3d(to + kWarps / 2 * C::kSlot, &tmW, 0, p.w_row, a.inter / 32 + p.block, full(st), policy);
      }
      __syncwarp();
      const __half* sc = p.sc;
      const int32_t* z0 = p.zr[0];
      const int32_t* z1 = p.zr[1];
      uint32_t sc_to = to + L::scales(a.ring_rows) + lane * 16, z_to = to + L::zeros(a.ring_rows, a.gmax) + lane * 4;
      for (int at = -p.g_at; at < ck; at += a.group) {      // the groups that the chunk touches
        if (p.sc_col >= 0) cp_async16(sc_to, sc);
        if (p.zc[0] >= 0) cp_async4(z_to, z0);
        if (C::kZeroWords > 32 && p.zc[1] >= 0) cp_async4(z_to + 128, z1);
        sc += a.N;
        z0 += a.zwords;
        z1 += a.zwords;
        sc_to += kCols * 2;
        z_to += C::kZeroWords * 4;
      }
    };
    auto put_acts = [&](const Put& p, int st) {
      const uint32_t to = smem_a + st * stage_bytes;
      const int left = a.K - p.x.kc * C::kK, ck = left < C::kK ? left : C::kK;
      // 16-byte pieces of the rows, then each row's scales
      constexpr int kPieces = C::kK / 8;
      const int pieces = p.rows * kPieces;
      for (int i = lane; i < pieces; i += 32) {
        const int m = i / kPieces, piece = i % kPieces;
        const int row = DOWN ? p.off + m : rt.row_token[p.off + m];
        if (piece * 8 < ck)
          cp_async16(to + L::act() + m * C::kActRow + piece * 16,
                     a.act + static_cast<long long>(row) * a.K + p.x.kc * C::kK + piece * 8);
      }
      if (lane < p.rows) {
        const uint32_t info = to + L::info(a.ring_rows) + lane * C::kInfo * 4;
#pragma unroll
        for (int i = 0; i < C::kRunsOf; ++i)
          if (i * kRun < ck) cp_async4(info + 4 * i, p.act_sc + i);
      }
      cp_async_arrive(full(st));
    };
    Put p = {};
    p.x = start;
    p.item = -1;
    place(p);
    int issued = 0;
    // the first chunks; DOWN's weights go out before UP has finished
    if (DOWN) {
      Put y = p;
      for (; issued < a.stages && p.x.u < limit; ++issued) {
        put_weights(p, issued);
        step(p);
      }
      decode::pdl_wait();
      for (int i = 0; i < issued; ++i) {
        put_acts(y, i);
        step(y);
      }
    } else {
      for (; issued < a.stages && p.x.u < limit; ++issued) {
        put_weights(p, issued);
        put_acts(p, issued);
        step(p);
      }
    }
    int st = 0;
    unsigned round = 0;                                    // parity of the stage's last emptying
    for (; p.x.u < limit; ++issued) {
      if (!wait(empty(st), round, &sm_abort, a.status)) break;
      put_weights(p, st);
      put_acts(p, st);
      step(p);
      if (++st == a.stages) {
        st = 0;
        round ^= 1;
      }
    }
    // let every copy land before shared memory is released (after a timeout no consumer waits for them)
    if (sm_abort) {
      const uint64_t t0 = ptx::globaltimer();
      for (int i = issued > a.stages ? issued - a.stages : 0; i < issued; ++i)
        while (!ptx::mbar_try_wait(full(i % a.stages), (i / a.stages) & 1) && ptx::globaltimer() - t0 < 2000000000ull) {}
    }
    return;
  }

  // ------------------------------------------------------------------ consumers
  const int gq = lane >> 2, tq = lane & 3;
  const int quad = decode::col_quad(gq), col0 = warp * 32 + quad * 4;   // this thread's 4 columns of the tile
  float acc[2][NB][4], cg[2][NB][4];
  auto clear = [](float (&x)[2][NB][4]) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[t][nb][i] = 0.f;
  };
  Cursor x = start;
  const int row_parts = TWICE ? 1 : a.parts;               // rows of the products to a row
  int cur = -1, rows = 0, off = 0;                         // rows: of the products
  int tok[NB][2];
  float wt[NB][2];
  auto open_slot = [&]() {
    cur = x.s;
    off = rt.slot_off[cur];
    const int count = rt.slot_off[cur + 1] - off;
    rows = count * row_parts;
    if constexpr (DOWN) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int m = row_parts == 2 ? 4 * nb + tq : 8 * nb + 2 * tq + i;
          tok[nb][i] = m < count ? rt.row_token[off + m] : 0;
          wt[nb][i] = m < count ? rt.row_weight[off + m] : 0.f;
        }
    }
    clear(acc);
  };
  // the finished rows of a slot into the tile: UP stores [row][column], DOWN adds w * y to [token] (both
  // parts of a row are one thread's)
  auto close_slot = [&]() {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int m = 8 * nb + 2 * tq + (i & 1), c = col0 + 2 * t + (i >> 1);
          if (m < rows) {
            const float v = acc[t][nb][i] * 1024.f;        // the differences' 2^-10
            if constexpr (DOWN) tile[tok[nb][i & 1] * kCols + c] += wt[nb][i & 1] * v;
            else tile[m * kCols + c] = v;
          }
        }
  };
  auto open_item = [&]() {
    if constexpr (DOWN) {                                  // this warp's own columns
      for (int t = 0; t < a.tokens; ++t) tile[t * kCols + warp * 32 + lane] = 0.f;
      __syncwarp();
    }
  };

  // the tile is complete.  DOWN: the layer's output; UP: one warp per row, 4 of the run's 128 columns
  // per lane
  auto finish = [&](int item) {
    if constexpr (DOWN) {
      const int n = item * kCols + static_cast<int>(threadIdx.x);
      if (n < a.N)
        for (int t = 0; t < a.tokens; ++t) {
          const float v = tile[t * kCols + threadIdx.x];
          const long long at = static_cast<long long>(t) * a.N + n;
          if (a.dtype == 0) static_cast<__half*>(a.out)[at] = __float2half_rn(v);
          else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
        }
      return;
    }
    const int j0 = (item % a.jblocks) * kRun, j = j0 + 4 * lane;
    for (int m = warp; m < rows; m += kWarps) {
      const float4 g = *reinterpret_cast<const float4*>(tile + m * kCols + 4 * lane);
      const float4 u = *reinterpret_cast<const float4*>(tile + m * kCols + kCols / 2 + 4 * lane);
      float h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float gi = (&g.x)[i];
        h[i] = j < a.inter ? gi / (1.f + expf(-gi)) * (&u.x)[i] : 0.f;
      }
      const long long row = off + m;
      store_run<BITS>(h, j0, a.inter, a.h_parts, a.h + row * a.h_parts * a.inter, a.h_scale + row * a.h_runs + j0 / kRun);
    }
  };
  // runs first .. last hold an item; the first leaves its part in its slot 1, the others in slot 0
  auto slot_of = [&](int r, int first) {
    return a.partials + (static_cast<size_t>(r) * 2 + (r == first ? 1 : 0)) * (static_cast<size_t>(a.tokens) * kCols);
  };
  auto close_item = [&](int item, long long first_chunk) {
    close_slot();
    consumer_sync();
    const int live = DOWN ? a.tokens : rows;
    const bool whole = first_chunk >= begin && first_chunk + per <= begin + limit;
    if (whole) {
      finish(item);
      consumer_sync();                                     // the tile is free again
      return;
    }
    // the part goes to the workspace; threads take (row, 4 columns)
    const int first = run_of(first_chunk);
    const int c4 = 4 * (threadIdx.x % (kCols / 4)), m0 = threadIdx.x / (kCols / 4);
    constexpr int kStep = kConsumers / (kCols / 4);
    float* to = slot_of(run, first);
    for (int m = m0; m < live; m += kStep)
      __stcg(reinterpret_cast<float4*>(to + m * kCols + c4), *reinterpret_cast<const float4*>(tile + m * kCols + c4));
    if (DOWN) {                                            // summed by a kernel of its own
      consumer_sync();
      return;
    }
    const int last = run_of(first_chunk + per - 1);
    consumer_sync();
    if (threadIdx.x == 0) {
      __threadfence();
      sm_last = atomicInc(a.counters + first, static_cast<unsigned>(last - first)) == static_cast<unsigned>(last - first);
      __threadfence();
    }
    consumer_sync();
    if (sm_last) {                                         // the last to arrive adds the parts in run order
      constexpr int kBatch = 8;
      for (int m = m0; m < live; m += kStep) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c0 = first; c0 <= last; c0 += kBatch) {
          float4 p[kBatch];
#pragma unroll
          for (int j = 0; j < kBatch; ++j)
            p[j] = __ldcg(reinterpret_cast<const float4*>(slot_of(c0 + j <= last ? c0 + j : last, first) + m * kCols + c4));
#pragma unroll
          for (int j = 0; j < kBatch; ++j)
            if (c0 + j <= last) {
              v.x += p[j].x;
              v.y += p[j].y;
              v.z += p[j].z;
              v.w += p[j].w;
            }
        }
        *reinterpret_cast<float4*>(tile + m * kCols + c4) = v;
      }
      consumer_sync();
      finish(item);
    }
    consumer_sync();
  };
  long long first_chunk = begin + start.u - start.c;       // of the current item, on the line
  open_item();
  // this thread's places in a stage: its pieces of the weights (tile l at w_at[l & 1] + 512 l; the swizzle
  // goes by the 128-byte line within the stage), scales and zeros, and its rows' activations and scales
  int w_at[BITS == 3 ? ROWS : 2], act_at[NB], info_at[NB][2];
  const int scales_at = L::scales(a.ring_rows) + 2 * col0;
  const int zeros_at = L::zeros(a.ring_rows, a.gmax) + 4 * (warp * BITS + BITS * quad * 4 / 32), zero_shift = BITS * quad * 4 % 32;
#pragma unroll
  for (int i = 0; i < (BITS == 3 ? ROWS : 2); ++i) {
    const int row = BITS == 3 ? tq * ROWS + i : 4 * i + tq, line = warp * C::kRows + row;
    w_at[i] = line * 128 + ((quad ^ (line & 7)) << 4) - (BITS == 3 ? 0 : 512 * i);
  }
  uint32_t base = smem_a;                                  // of the stage
  int st = 0, g_at = 0;                                    // g_at: k of the chunk within its first group
  unsigned round = 0;
  while (x.u < limit) {
    if (x.s != cur) {
      open_slot();
      g_at = x.kc * C::kK % a.group;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {                    // rows past the slot's read its last one
        const int m = 8 * nb + gq;
        act_at[nb] = L::act() + (m < rows ? m : rows - 1) * (TWICE ? 2 * C::kActRow : C::kActRow) + tq * (NP * 4);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int mi = 8 * nb + 2 * tq + i;
          info_at[nb][i] = L::info(a.ring_rows) + (mi < rows ? mi : rows - 1) * ((TWICE ? 2 : 1) * C::kInfo * 4);
        }
      }
    }
    if (__all_sync(0xFFFFFFFFu, wait(full(st), round, &sm_abort, a.status))) {
      const int k0 = x.kc * C::kK;
      const int tiles = a.K - k0 < C::kK ? (a.K - k0) / C::kTileK : C::kTiles;
      float gs[4];                                         // scales and zeros of this thread's 4 columns
      uint32_t gz[4];
      auto load_group = [&](int g) {
        const uint2 s = lds64(base + scales_at + g * (kCols * 2));
        gs[0] = __half2float(__ushort_as_half(lo16(s.x)));
        gs[1] = __half2float(__ushort_as_half(hi16(s.x)));
        gs[2] = __half2float(__ushort_as_half(lo16(s.y)));
        gs[3] = __half2float(__ushort_as_half(hi16(s.y)));
        const uint32_t zw = base + zeros_at + g * (C::kZeroWords * 4);
        uint32_t zf = lds32(zw) >> zero_shift;
        if (BITS == 3) zf = zero_shift + 12 > 32 ? zf | lds32(zw + 4) << (32 - zero_shift) : zf;
#pragma unroll
        for (int c = 0; c < 4; ++c) gz[c] = zero_pair(((zf >> (BITS * c)) & P::kMask) + a.zero_offset);
      };
      auto load_tile = [&](int l, uint4 (&w)[ROWS]) {
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          if constexpr (BITS == 3) w[r] = lds128(base + w_at[r]);
          else w[r] = lds128(base + w_at[l & 1] + l * 512);
        }
      };
      auto load_acts = [&](int l, int nb, uint32_t (&b)[NP], int part = 0) {
        const uint32_t src = base + act_at[nb] + l * (NP * 16) + part * C::kActRow;
        if constexpr (NP % 4 == 0) {
#pragma unroll
          for (int i = 0; i < NP / 4; ++i) {
            const uint4 v = lds128(src + 16 * i);
            b[4 * i] = v.x; b[4 * i + 1] = v.y; b[4 * i + 2] = v.z; b[4 * i + 3] = v.w;
          }
        } else {
          const uint2 v = lds64(src);
          b[0] = v.x; b[1] = v.y;
        }
      };
      // the products of one k-tile; b0: its activations of the first 8 rows
      auto multiply = [&](int l, const uint4 (&w)[ROWS], const uint32_t (&b0)[NP]) {
        uint32_t d[4][NP];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if constexpr (BITS == 3) RP::run3((&w[0].x)[c], (&w[1].x)[c], (&w[2].x)[c], gz[c], d[c]);
          else RP::run((&w[0].x)[c], gz[c], d[c]);
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          if (nb == 0 || 8 * nb < rows) {
            uint32_t b[NP];
            if (nb == 0) {
#pragma unroll
              for (int i = 0; i < NP; ++i) b[i] = b0[i];
            } else {
              load_acts(l, nb, b);
            }
#pragma unroll
            for (int part = 0; part < (TWICE ? 2 : 1); ++part) {
              if (part) load_acts(l, nb, b, 1);
#pragma unroll
              for (int j = 0; j < NP / 2; ++j)
#pragma unroll
                for (int t = 0; t < 2; ++t)
                  mma(cg[t][nb], d[2 * t][2 * j], d[2 * t + 1][2 * j], d[2 * t][2 * j + 1], d[2 * t + 1][2 * j + 1], b[2 * j], b[2 * j + 1]);
            }
          }
        }
      };
      auto tile_mma = [&](int l) {
        uint4 w[ROWS];
        uint32_t b[NP];
        load_tile(l, w);
        load_acts(l, 0, b);
        multiply(l, w, b);
      };
      // tiles of the run that tile l0 lies in are done: acc += scale act_scale c
      auto fold = [&](int l0) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          if (nb == 0 || 8 * nb < rows) {
            float s[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) s[i] = __uint_as_float(lds32(base + info_at[nb][i] + 4 * (l0 * C::kTileK / kRun)));
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                acc[t][nb][i] = fmaf(gs[2 * t + (i >> 1)], s[i & 1] * cg[t][nb][i], acc[t][nb][i]);
          }
        }
      };
      if (a.group % C::kSegK == 0 && tiles == C::kTiles) {
        // every segment of kSegTiles tiles lies in one group and one run
#pragma unroll
        for (int l0 = 0; l0 < C::kTiles; l0 += C::kSegTiles) {
          load_group(l0 == 0 || g_at + l0 * C::kTileK < a.group ? 0 : (g_at + l0 * C::kTileK) / a.group);
          clear(cg);
          // a segment's tiles are loaded ahead of their products (2-bit tiles hold 64 k and go one by one)
          if constexpr (BITS == 4 || BITS == 8) {
            uint4 w[C::kSegTiles][ROWS];
            uint32_t b[C::kSegTiles][NP];
#pragma unroll
            for (int l = 0; l < C::kSegTiles; ++l) {
              load_tile(l0 + l, w[l]);
              load_acts(l0 + l, 0, b[l]);
            }
#pragma unroll
            for (int l = 0; l < C::kSegTiles; ++l) multiply(l0 + l, w[l], b[l]);
          } else {
#pragma unroll
            for (int l = l0; l < l0 + C::kSegTiles; ++l) tile_mma(l);
          }
          fold(l0);
        }
      } else {
        int g = 0, g_end = k0 - g_at + a.group;
        clear(cg);
        load_group(0);
#pragma unroll
        for (int l = 0; l < C::kTiles; ++l) {
          if (l < tiles) {
            tile_mma(l);
            const int k = k0 + (l + 1) * C::kTileK;
            if (k == g_end || k % kRun == 0 || l + 1 == tiles) {   // a group, a run or the chunk ends
              fold(l);
              clear(cg);
              if (k == g_end && l + 1 < tiles) {
                load_group(++g);
                g_end += a.group;
              }
            }
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(empty(st));
    base += stage_bytes;
    if (++st == a.stages) {
      st = 0;
      round ^= 1;
      base = smem_a;
    }
    g_at += C::kK;
    while (g_at >= a.group) g_at -= a.group;
    // to the next chunk
    const int item = x.item;
    const bool next = advance(x);
    if (next || x.u >= limit) {
      close_item(item, first_chunk);
      first_chunk += per + kItemUnits;
      cur = -1;
      if (x.u < limit) open_item();
    } else if (x.s != cur) {
      close_slot();
    }
  }
}

// out = the parts of each 256 columns, rounded once.  A CTA takes a token of an item, a thread 4 columns
// and a quarter of the parts, each quarter in run order and the quarters in theirs, so the sum does not
// depend on timing.  (In DOWN itself the last CTA to arrive would add up to 40 parts of tokens x 256
// values alone: 16 tokens of 2048 columns took 60 us that way.)
template <typename T>
__global__ void __launch_bounds__(kCols) k_sum_parts(const float* partials, const int* slots, int nk, int items, int grid,
                                                     int tokens, int hidden, T* out) {
  constexpr int kQuads = kCols / 4, kShares = 4, kBatch = 16;
  __shared__ float4 sm[kShares - 1][kQuads];
  decode::pdl_wait();
  decode::pdl_launch_dependents();
  const int per = *slots * nk, item = blockIdx.x, m = blockIdx.y;
  const Line line(static_cast<long long>(items) * (per + kItemUnits), grid);
  const long long first_chunk = static_cast<long long>(item) * (per + kItemUnits) + kItemUnits;
  const int first = line.run_of(first_chunk), last = line.run_of(first_chunk + per - 1);
  if (first == last) return;   // (DOWN wrote an item inside one run itself)
  const int quad = threadIdx.x % kQuads, share = threadIdx.x / kQuads, n = item * kCols + 4 * quad;
  const int each = (last - first + kShares) / kShares, from = first + share * each;
  const int to = from + each <= last ? from + each : last + 1;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c0 = from; c0 < to; c0 += kBatch) {
    float4 p[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int r = c0 + j;
      p[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < to)
        p[j] = __ldcg(reinterpret_cast<const float4*>(
            partials + ((static_cast<size_t>(r) * 2 + (r == first ? 1 : 0)) * tokens + m) * kCols + 4 * quad));
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      v.x += p[j].x;
      v.y += p[j].y;
      v.z += p[j].z;
      v.w += p[j].w;
    }
  }
  if (share > 0) sm[share - 1][quad] = v;
  __syncthreads();
  if (share > 0 || n >= hidden) return;
#pragma unroll
  for (int i = 0; i < kShares - 1; ++i) {
    v.x += sm[i][quad].x;
    v.y += sm[i][quad].y;
    v.z += sm[i][quad].z;
    v.w += sm[i][quad].w;
  }
  *reinterpret_cast<uint2*>(out + static_cast<long long>(m) * hidden + n) = make_uint2(pack2(v.x, v.y, T()), pack2(v.z, v.w, T()));
}

template <int BITS, int NB, bool DOWN, bool TWICE = false>
cudaError_t launch_experts(Args a, const int32_t* qweight, int experts, int* runs, cudaStream_t stream) {
  using C = Chunk<BITS>;
  using L = Layout<BITS>;
  auto kern = k_experts<BITS, NB, DOWN, TWICE>;
  const DeviceInfo& dev = device_info();
  a.units = a.K / Pack<BITS>::kPerUnit;
  a.zwords = a.N / 32 * BITS;
  const int room = 8 * NB / (TWICE ? 1 : a.parts);
  a.rows = a.tokens < room ? a.tokens : room;
  a.ring_rows = a.rows * a.parts;
  a.gmax = (C::kK - 1) / a.group + 2;
  if (a.group % C::kK == 0) a.gmax = 1;
  else if (C::kK % a.group == 0) a.gmax = C::kK / a.group;
  a.stage_bytes = L::stage(a.ring_rows, a.gmax);
  const int pairs = a.tokens * a.topk;
  int per_sm = kCtas;
  auto fit = [&](int ctas) {
    const int budget = ctas > 1 ? 233472 / ctas - 1024 - 512 : 227 * 1024 - 512;   // less the static part
    return (budget - L::fixed(DOWN ? a.tokens : a.rows, pairs, experts)) / (a.stage_bytes + 16);
  };
  a.stages = fit(per_sm);
  while (per_sm > 1 && a.stages < 3) a.stages = fit(--per_sm);
  if (a.stages > kMaxStages) a.stages = kMaxStages;
  // the router's scratch lies over the ring
  if (a.stages < 2 || a.stages * a.stage_bytes < kThreads / 32 * experts * 4 || a.stages * a.stage_bytes < pairs * 4) return cudaErrorInvalidConfiguration;
  const int smem = L::fixed(DOWN ? a.tokens : a.rows, pairs, experts) + a.stages * (a.stage_bytes + 16);
  static std::atomic<unsigned long long> opted_in{0};       // per device
  if (dev.device >= 64 || !(opted_in.load(std::memory_order_relaxed) & (1ull << dev.device))) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024 - 512);
    if (e != cudaSuccess) return e;
    if (dev.device < 64) opted_in.fetch_or(1ull << dev.device, std::memory_order_relaxed);
  }
  CUtensorMap tmW = {};
  // (column of 32, packed row, block of 32 columns): a box lands block by block, as the warps read it
  const uint64_t dims[3] = {32, static_cast<uint64_t>(a.units) * Pack<BITS>::kRowsPerUnit * experts, static_cast<uint64_t>(a.N) / 32};
  const uint64_t strides[2] = {static_cast<uint64_t>(a.N) * 4, 128};
  const uint32_t box[3] = {32, static_cast<uint32_t>(C::kRows), DOWN ? kWarps : kWarps / 2};
  const uint32_t estr[3] = {1, 1, 1};
  if (!encode_tensor_map_nd(&tmW, CU_TENSOR_MAP_DATA_TYPE_INT32, 3, const_cast<int32_t*>(qweight), dims, strides, box, estr,
                            CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  int grid = dev.sm_count * per_sm;
  if (grid > kMaxRuns) grid = kMaxRuns;
  *runs = grid;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, tmW, a);
}

template <int BITS, bool DOWN>
cudaError_t launch_blocks(const Args& a, const int32_t* qweight, int experts, int* runs, cudaStream_t stream) {
  // Single blocks (8 rows, or 4 in two parts) unless the experts have as many rows on average: a further block
  // of an expert reads its weights again, a double one multiplies rows that are not there and has 96 registers
  // for twice the accumulators.  At 8 bits, where reading is most of it, unless they have half as many.
  // Single and double, wide layer of 8 experts, top-2, bf16: 18 tokens 182 and 217 us, 24 206 and 232, 32 250 and
  // 247; 24 at 2, 3 and 8 bits 198 and 263, 224 and 385, 362 and 324.
  // In two parts a double block holds 8 rows as well, and so does a single one whose parts are multiplied one
  // after the other.  Blocks of 4, double and single of 8 (fp16): 8 tokens 172, 183 and 173 us, 12 185, 193 and
  // 186, 16 196, 199 and 195, 24 246, 227 and 220; 32 at 2, 3 and 8 bits, the last two, 331 and 293, 458 and
  // 408, 383 and 370.
  constexpr int kBlock = 8;
  const int room = kBlock / a.parts, pairs = a.tokens * a.topk;
  if (a.tokens <= room || (BITS == 8 ? 2 * pairs <= room * a.experts : pairs < room * a.experts))
    return launch_experts<BITS, 1, DOWN>(a, qweight, experts, runs, stream);
  if constexpr (DOWN)
    if (a.parts == 2) return launch_experts<BITS, 1, DOWN, true>(a, qweight, experts, runs, stream);
  return launch_experts<BITS, 2, DOWN>(a, qweight, experts, runs, stream);
}

template <int BITS>
cudaError_t launch_bits(const Args& up, const int32_t* up_qweight, const Args& down, const int32_t* down_qweight, int experts,
                        int* down_grid, cudaStream_t stream) {
  int up_grid = 0;
  const cudaError_t e = launch_blocks<BITS, false>(up, up_qweight, experts, &up_grid, stream);
  return e != cudaSuccess ? e : launch_blocks<BITS, true>(down, down_qweight, experts, down_grid, stream);
}

}  // namespace moe
}  // namespace gptq
