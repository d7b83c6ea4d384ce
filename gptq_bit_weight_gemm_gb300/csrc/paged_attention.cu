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
// own: every lane copies (cp.async, 16 bytes) exactly the pieces of k and v that it will feed to the
// tensor cores, so the ring needs no barrier, only the lane's own wait.  The k dimension of an MMA
// may be permuted as long as both operands agree: lane (g, t) = (lane / 4, lane % 4) reads 8
// consecutive dimensions of key g as the B fragments of two k-steps of q k^T (the query fragments are
// loaded in the same order), and 8 consecutive dimensions 8 g .. 8 g + 7 of keys 2t, 2t+1, 2t+8, 2t+9
// as the B fragments of eight column tiles of p v, tile j taking column 8 g + j.  The scores' C
// fragment is the A fragment of p v as it stands.
#include <math_constants.h>

#include "decode.cuh"
#include "gptq_device.cuh"
#include "gptq_internal.h"
#include "serving_internal.h"

namespace gptq {
namespace attention {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kWarpKeys = 16, kTileKeys = kWarps * kWarpKeys;
constexpr int kMaxRows = 16;             // query heads of one item
constexpr int kMaxCtas = 512;            // runs, at most
constexpr size_t kControlBytes = 4096;   // arrival counters, one per run

// Dimensions padded to DP (64, 128, 256); R = 1 or 2 blocks of 8 query rows.
template <int DP, int R>
struct Shape {
  static constexpr int kBlocks = DP / 32;                  // 32-dimension blocks of k
  static constexpr int kHalves = DP / 64;                  // 64-dimension blocks of v
  static constexpr int kPieces = 2 * kBlocks + 4 * kHalves;   // 16-byte pieces per lane and stage
  static constexpr int kStages = DP == 64 ? 4 : 3;
  static constexpr int kCtas = DP == 256 ? 1 : (DP == 128 ? 2 : 3);   // per SM
  static constexpr int kAcc = kHalves * 8 * 2 * R;         // live accumulators per thread
  static constexpr size_t kRing = static_cast<size_t>(kStages) * kWarps * kPieces * 512;
  static constexpr size_t kMerge = 2 * static_cast<size_t>(kAcc) * 128;
  static constexpr size_t kSmem = kRing + kMerge;
};

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
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
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

// A place on the line of tiles.
struct Cursor {
  int b, h, t, nt, n, n_next;
  __device__ __forceinline__ void set(const AttentionProblem& p, int seq, int raw) {
    b = seq;
    n = clamp_len(p, raw);
    nt = tile_count(p, n);
    n_next = seq + 1 < p.batch ? p.lens[seq + 1] : 0;      // fetched a sequence ahead
  }
  __device__ __forceinline__ bool advance(const Args& a) {   // true: a new item begins
    if (++t < nt) return false;
    t = 0;
    if (++h == a.items) {
      h = 0;
      if (b + 1 < a.p.batch) set(a.p, b + 1, n_next);
    }
    return true;
  }
};

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

template <typename T, int DP, int R>
__global__ void __launch_bounds__(kThreads, (Shape<DP, R>::kCtas)) k_attention(const Args a) {
  using S = Shape<DP, R>;
  using Tr = F16Traits<T>;
  const AttentionProblem& p = a.p;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float sm_m[kWarps][kMaxRows], sm_l[kWarps][kMaxRows];
  __shared__ long long sm_sum[kWarps];
  __shared__ long long sm_at;
  __shared__ int sm_seq, sm_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;

  decode::pdl_launch_dependents();
  decode::pdl_wait();

  // ---- this CTA's run: the tiles of all sequences, then the sequence its first tile falls into
  long long total = 0;
  {
    long long mine = 0;
    for (int b = threadIdx.x; b < p.batch; b += kThreads) {
      const int raw = p.lens[b], n = clamp_len(p, raw);
      if (n != raw && blockIdx.x == 0) atomicOr(p.status, kStatusSeqLen);
      mine += tile_count(p, n);
    }
    mine = warp_sum(mine);
    if (lane == 0) sm_sum[warp] = mine;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) total += sm_sum[w];
    total *= a.items;
  }
  const int runs = total < static_cast<long long>(gridDim.x) ? static_cast<int>(total) : static_cast<int>(gridDim.x);
  const int run = blockIdx.x;
  if (run >= runs) return;
  const long long begin = total * run / runs, end = total * (run + 1) / runs;
  {
    long long before = 0;                                  // tiles of the sequences before this chunk
    for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
      const int b = b0 + static_cast<int>(threadIdx.x);
      const long long w = b < p.batch ? static_cast<long long>(tile_count(p, clamp_len(p, p.lens[b]))) * a.items : 0;
      long long c = w;                                     // inclusive scan over the CTA
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xFFFFFFFFu, c, o);
        if (lane >= o) c += v;
      }
      __syncthreads();
      if (lane == 31) sm_sum[warp] = c;
      if (threadIdx.x == 0) sm_seq = -1;
      __syncthreads();
      long long all = 0;
      for (int x = 0; x < kWarps; ++x) {
        if (x < warp) c += sm_sum[x];
        all += sm_sum[x];
      }
      const long long lo = before + c - w;
      if (lo <= begin && begin < lo + w) {
        sm_seq = b;
        sm_at = lo;
      }
      __syncthreads();
      if (sm_seq >= 0) break;
      before += all;
    }
  }
  if (sm_seq < 0) return;                                  // lengths written while this ran
  Cursor put, get;
  put.set(p, sm_seq, p.lens[sm_seq]);
  {
    const long long rel = begin - sm_at;
    put.h = static_cast<int>(rel / put.nt);
    put.t = static_cast<int>(rel - static_cast<long long>(put.h) * put.nt);
  }
  get = put;

  // ---- the ring: stage s of this warp, piece i of this lane
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * S::kPieces * 512 + lane * 16;
  auto stage_at = [&](int s) { return ring + s * (kWarps * S::kPieces * 512); };
  unsigned long long live = 0;                             // 16 key bits per stage in flight, oldest first
  int page = -1;                                           // lanes 0..15: the page of this lane's next key
  // lane l < 16 looks up key `key0 + l` of the producer's place
  auto place = [&](int& key, int& kb) {
    kb = (first_key(p, put.n) & ~(kWarpKeys - 1)) + put.t * kTileKeys + warp * kWarpKeys;
    key = kb + (lane & 15);
  };
  auto fetch_page = [&]() {
    int key, kb;
    place(key, kb);
    page = -1;
    if (lane < kWarpKeys && key >= first_key(p, put.n) && key < put.n)
      page = __ldg(p.table + static_cast<long long>(put.b) * p.table_width + key / p.page_size);
  };
  auto issue = [&](int s, int pos) {
    int key, kb;
    place(key, kb);
    const bool wanted = lane < kWarpKeys && key >= first_key(p, put.n) && key < put.n;
    const bool ok = wanted && page >= 0 && page < p.pages;
    if (wanted && !ok) atomicOr(p.status, kStatusPageRange);
    const unsigned mask = __ballot_sync(0xFFFFFFFFu, ok);
    live |= static_cast<unsigned long long>(mask) << (16 * pos);
    if (mask == 0) return;
    const int hk = put.h / a.row_blocks;
    // addresses of this lane's key's rows; the new token's rows come from k_new and v_new
    const T* krow = static_cast<const T*>(p.k_cache);
    const T* vrow = static_cast<const T*>(p.v_cache);
    if (ok) {
      const int slot = key % p.page_size;
      krow += page * p.k_page + slot * p.k_slot + hk * p.k_head;
      vrow += page * p.v_page + slot * p.v_slot + hk * p.v_head;
    }
    if (p.k_new) {
      const int last = put.n - 1 - kb;                     // the new token's place among the 16 keys
      if (last >= 0 && last < kWarpKeys && (mask >> last & 1)) {
        const T* kn = static_cast<const T*>(p.k_new) + put.b * p.kn_batch + hk * p.head_dim;
        const T* vn = static_cast<const T*>(p.v_new) + put.b * p.vn_batch + hk * p.head_dim;
        T* kd = const_cast<T*>(reinterpret_cast<const T*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(krow), last)));
        T* vd = const_cast<T*>(reinterpret_cast<const T*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(vrow), last)));
        if (put.h % a.row_blocks == 0) {                   // one item of the kv head appends
          const int pieces = p.head_dim / 8;
          for (int i = lane; i < 2 * pieces; i += 32) {
            if (i < pieces) reinterpret_cast<uint4*>(kd)[i] = reinterpret_cast<const uint4*>(kn)[i];
            else reinterpret_cast<uint4*>(vd)[i - pieces] = reinterpret_cast<const uint4*>(vn)[i - pieces];
          }
        }
        if (lane == last) {
          krow = kn;
          vrow = vn;
        }
      }
    }
    const unsigned long long ka = reinterpret_cast<unsigned long long>(krow), va = reinterpret_cast<unsigned long long>(vrow);
    const uint32_t dst = stage_at(s);
#pragma unroll
    for (int i = 0; i < 2; ++i) {                          // keys g and g + 8
      const int k = g + 8 * i;
      const T* src = reinterpret_cast<const T*>(__shfl_sync(0xFFFFFFFFu, ka, k));
      const bool on = mask >> k & 1;
#pragma unroll
      for (int blk = 0; blk < S::kBlocks; ++blk) {
        const int d = 32 * blk + 8 * t;
        const bool in = on && d < p.head_dim;
        cp_async16(dst + (i * S::kBlocks + blk) * 512, in ? src + d : src, in ? 16u : 0u);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {                          // keys 2t, 2t + 1, 2t + 8, 2t + 9
      const int k = 2 * t + (i & 1) + 8 * (i >> 1);
      const T* src = reinterpret_cast<const T*>(__shfl_sync(0xFFFFFFFFu, va, k));
      const bool on = mask >> k & 1;
#pragma unroll
      for (int hb = 0; hb < S::kHalves; ++hb) {
        const int d = 64 * hb + 8 * g;
        const bool in = on && d < p.head_dim;
        cp_async16(dst + (2 * S::kBlocks + i * S::kHalves + hb) * 512, in ? src + d : src, in ? 16u : 0u);
      }
    }
  };
  const int ntiles = static_cast<int>(end - begin < 0x7FFFFFFF ? end - begin : 0x7FFFFFFF);
  int put_left = ntiles;
  fetch_page();
  auto produce = [&](int s, int pos) {                     // one tile into stage s, the fifo's place pos
    if (put_left > 0) {
      issue(s, pos);
      if (--put_left > 0) {
        put.advance(a);
        fetch_page();
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int s = 0; s < S::kStages; ++s) produce(s, s);

  // ---- the consumer: queries, running maximum and sum (log2 units) of rows g and g + 8, accumulator
  uint32_t q[R][S::kBlocks * 4];
  float m[R], l[R], o[S::kHalves * 8][4];
  auto rows_of = [&](int h) {                              // live query rows of item h
    const int r = a.group - (h % a.row_blocks) * kMaxRows;
    return r < kMaxRows ? r : kMaxRows;
  };
  auto q_head = [&](int h) { return (h / a.row_blocks) * a.group + (h % a.row_blocks) * kMaxRows; };
  auto open_item = [&]() {
    const T* qp = static_cast<const T*>(p.q) + get.b * p.q_batch + static_cast<long long>(q_head(get.h)) * p.head_dim;
    const int rows = rows_of(get.h);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = -CUDART_INF_F;
      l[r] = 0.f;
#pragma unroll
      for (int blk = 0; blk < S::kBlocks; ++blk) {
        const int row = g + 8 * r, d = 32 * blk + 8 * t;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (row < rows && d < p.head_dim) v = __ldg(reinterpret_cast<const uint4*>(qp + row * p.head_dim + d));
        q[r][4 * blk] = v.x; q[r][4 * blk + 1] = v.y; q[r][4 * blk + 2] = v.z; q[r][4 * blk + 3] = v.w;
      }
    }
#pragma unroll
    for (int i = 0; i < S::kHalves * 8; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[i][c] = 0.f;
  };

  auto compute = [&](int s, unsigned mask) {
    const uint32_t src = stage_at(s);
    float sc[2][4] = {};
#pragma unroll
    for (int blk = 0; blk < S::kBlocks; ++blk) {
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const uint4 v = lds128(src + (nt * S::kBlocks + blk) * 512);
        mma(sc[nt], q[0][4 * blk], R == 2 ? q[R - 1][4 * blk] : 0u, q[0][4 * blk + 1], R == 2 ? q[R - 1][4 * blk + 1] : 0u,
            v.x, v.y, T());
        mma(sc[nt], q[0][4 * blk + 2], R == 2 ? q[R - 1][4 * blk + 2] : 0u, q[0][4 * blk + 3],
            R == 2 ? q[R - 1][4 * blk + 3] : 0u, v.z, v.w, T());
      }
    }
    uint32_t pa[2][2];                                     // [row block][key half]: the A fragment of p v
    bool moved = false;
    float alpha[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = 8 * (i >> 1) + 2 * t + (i & 1);
        x[i] = mask >> key & 1 ? sc[i >> 1][2 * r + (i & 1)] * a.scale_log2 : -CUDART_INF_F;
      }
      float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      const float mn = fmaxf(m[r], top), base = mn == -CUDART_INF_F ? 0.f : mn;
      alpha[r] = exp2f(m[r] - base);
      moved |= mn != m[r];
      m[r] = mn;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = exp2f(x[i] - base);
      l[r] = l[r] * alpha[r] + ((x[0] + x[1]) + (x[2] + x[3]));
      // the probabilities are rounded to 16 bits for the tensor cores (relative 2^-11 / 2^-8, as the
      // values they multiply); their sum l is not
      pa[r][0] = pack2(x[0], x[1], T());
      pa[r][1] = pack2(x[2], x[3], T());
    }
    if (R == 1) pa[1][0] = pa[1][1] = 0u;
    if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
      for (int i = 0; i < S::kHalves * 8; ++i)
#pragma unroll
        for (int c = 0; c < 2 * R; ++c) o[i][c] *= alpha[c >> 1];
    }
#pragma unroll
    for (int hb = 0; hb < S::kHalves; ++hb) {
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = lds128(src + (2 * S::kBlocks + i * S::kHalves + hb) * 512);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
        const uint32_t b0 = __byte_perm((&v[0].x)[j >> 1], (&v[1].x)[j >> 1], sel);
        const uint32_t b1 = __byte_perm((&v[2].x)[j >> 1], (&v[3].x)[j >> 1], sel);
        mma(o[hb * 8 + j], pa[0][0], pa[1][0], pa[0][1], pa[1][1], b0, b1, T());
      }
    }
  };

  // One row of an item: the running sum's factor and the place of its values.  Warp 0's lane (g, t)
  // holds, of row g + 8 r and half hb, dimensions 64 hb + 16 t .. + 15.
  auto write_row = [&](int b, int h, int r, float mr, float lr) {
    const int row = g + 8 * r;
    if (row >= rows_of(h)) return;
    const long long at = static_cast<long long>(b) * p.heads + q_head(h) + row;
    const float inv = lr > 0.f || isnan(lr) ? 1.f / lr : 0.f;
    T* out = static_cast<T*>(p.out) + at * p.head_dim;
#pragma unroll
    for (int hb = 0; hb < S::kHalves; ++hb)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int d = 64 * hb + 16 * t + 8 * c;
        if (d < p.head_dim) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = pack2(o[hb * 8 + 2 * j][2 * r + c] * inv, o[hb * 8 + 2 * j + 1][2 * r + c] * inv, T());
          *reinterpret_cast<uint4*>(out + d) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    if (p.lse && t == 0) p.lse[at] = mr * 0.693147180559945f + logf(lr);
  };
  float* const merge = reinterpret_cast<float*>(smem + S::kRing);
  auto acc = [&](int i) -> float& { return o[i / (2 * R)][i % (2 * R)]; };

  // The item's keys of this run are done: the 4 warps join, and warp 0 writes the result or a partial.
  auto close_item = [&](long long item_begin, long long item_end) {
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
    float M[R], L[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      M[r] = -CUDART_INF_F;
      for (int w = 0; w < kWarps; ++w) M[r] = fmaxf(M[r], sm_m[w][g + 8 * r]);
      const float base = M[r] == -CUDART_INF_F ? 0.f : M[r];
      L[r] = 0.f;
      for (int w = 0; w < kWarps; ++w) L[r] += sm_l[w][g + 8 * r] * exp2f(sm_m[w][g + 8 * r] - base);
      const float f = exp2f(m[r] - base);
#pragma unroll
      for (int i = 0; i < S::kHalves * 8; ++i) {
        o[i][2 * r] *= f;
        o[i][2 * r + 1] *= f;
      }
    }
#pragma unroll
    for (int step = 2; step >= 1; step >>= 1) {
      if (warp >= step && warp < 2 * step)
#pragma unroll
        for (int i = 0; i < S::kAcc; ++i) merge[((warp - step) * S::kAcc + i) * 32 + lane] = acc(i);
      __syncthreads();
      if (warp < step)
#pragma unroll
        for (int i = 0; i < S::kAcc; ++i) acc(i) += merge[(warp * S::kAcc + i) * 32 + lane];
      __syncthreads();
    }
    const bool whole = item_begin >= begin && item_end <= end;
    if (whole) {
      if (warp == 0)
#pragma unroll
        for (int r = 0; r < R; ++r) write_row(get.b, get.h, r, M[r], L[r]);
      return;
    }
    // ---- part of an item: runs first .. last hold it; the first leaves its part in its slot 1,
    // the others in slot 0
    const int first = static_cast<int>(((item_begin + 1) * runs - 1) / total);
    const int last = static_cast<int>((item_end * runs - 1) / total);
    auto slot = [&](int r) { return a.partials + (static_cast<size_t>(r) * 2 + (r == first ? 1 : 0)) * partial_floats(DP); };
    if (warp == 0) {
      float* to = slot(run);
#pragma unroll
      for (int i = 0; i < S::kAcc; ++i) __stcg(to + i * 32 + lane, acc(i));
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (t == 0) {
          __stcg(to + kMaxRows * DP + g + 8 * r, M[r]);
          __stcg(to + kMaxRows * DP + kMaxRows + g + 8 * r, L[r]);
        }
      __threadfence();
      __syncwarp();
      // the counter wraps to zero at the last arrival, ready for the next call
      if (lane == 0) sm_last = atomicInc(a.counters + first, static_cast<unsigned>(last - first)) == static_cast<unsigned>(last - first);
    }
    __syncthreads();
    if (!sm_last) return;
    __threadfence();
    // the last arrival joins the parts in run order; warp w takes a quarter of the accumulators
    constexpr int kMine = (S::kAcc + kWarps - 1) / kWarps;
    float sum[kMine] = {};
#pragma unroll
    for (int r = 0; r < R; ++r) M[r] = -CUDART_INF_F, L[r] = 0.f;
    for (int c = first; c <= last; ++c)
#pragma unroll
      for (int r = 0; r < R; ++r) M[r] = fmaxf(M[r], __ldcg(slot(c) + kMaxRows * DP + g + 8 * r));
#pragma unroll 4
    for (int c = first; c <= last; ++c) {
      const float* from = slot(c);
      float f[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        f[r] = exp2f(__ldcg(from + kMaxRows * DP + g + 8 * r) - (M[r] == -CUDART_INF_F ? 0.f : M[r]));
        L[r] += __ldcg(from + kMaxRows * DP + kMaxRows + g + 8 * r) * f[r];
      }
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int e = warp * kMine + i;
        sum[i] += __ldcg(from + e * 32 + lane) * f[R == 2 ? (i % 4) >> 1 : 0];
      }
    }
    // back through shared memory, so that warp 0's lanes hold whole rows
    static_assert(S::kAcc % kWarps == 0 && (R == 1 || kMine % 4 == 0), "quarters of whole fragments");
#pragma unroll
    for (int i = 0; i < kMine; ++i) merge[(warp * kMine + i) * 32 + lane] = sum[i];
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int i = 0; i < S::kAcc; ++i) acc(i) = merge[i * 32 + lane];
#pragma unroll
      for (int r = 0; r < R; ++r) write_row(get.b, get.h, r, M[r], L[r]);
    }
    __syncthreads();
  };

  open_item();
  long long item_begin = begin - get.t;
  int stage = 0;
  for (int i = 0; i < ntiles; ++i) {
    cp_wait<S::kStages - 1>();
    const unsigned mask = static_cast<unsigned>(live & 0xFFFFu);
    if (mask) compute(stage, mask);
    live >>= 16;
    produce(stage, S::kStages - 1);
    stage = stage + 1 == S::kStages ? 0 : stage + 1;
    const bool item_done = get.t + 1 == get.nt;
    if (item_done || i + 1 == ntiles) close_item(item_begin, item_begin + get.nt);
    if (i + 1 == ntiles) break;
    item_begin += item_done ? get.nt : 0;
    if (get.advance(a)) open_item();
  }
  cp_wait<0>();
}

template <typename T, int DP, int R>
cudaError_t launch(const Args& a, cudaStream_t stream) {
  using S = Shape<DP, R>;
  auto kern = k_attention<T, DP, R>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(S::kSmem));
  if (e != cudaSuccess) return e;
  int grid = device_info().sm_count * S::kCtas;
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
  a.counters = static_cast<unsigned*>(p.workspace);
  a.partials = reinterpret_cast<float*>(static_cast<char*>(p.workspace) + attention::kControlBytes);
  return p.dtype == 0 ? attention::launch_dim<__half>(a, stream) : attention::launch_dim<__nv_bfloat16>(a, stream);
}

}  // namespace gptq
