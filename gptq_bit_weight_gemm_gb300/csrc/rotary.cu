// rotary.cu -- rotary embedding of a step's queries and keys, and the append of its keys and values to
// the paged cache.
//
// The angle of pair i at position p is p f_i.  In fp32 its product is off by up to p f_i 2^-24 rad: 0.008 at
// position 131072.  Here f_i / (2 pi) is a whole number of 2^-64 turns, so that p times it, modulo 2^64, is
// the angle modulo a turn, exactly: one integer multiplication.  Its upper 32 bits, as a signed number, are the
// argument of sincospi in units of 2^-31 (rounding it to fp32 moves the angle by pi 2^-25 at most).
//
// Bound: q, k and v are read once and written once.
//
// A CTA takes a token.  Each sine and cosine is made once, by one thread, and kept in shared memory; a thread
// then holds those of the pairs it turns and goes through the heads with them, V neighbouring values (16 bytes
// where the layout of the pairs allows it) at a time, 4 heads' loads in flight, the first of them issued
// before the sines are made.
#include "decode.cuh"
#include "gptq_device.cuh"
#include "gptq_internal.h"
#include "prompt_internal.h"

namespace gptq {
namespace rotary {

constexpr int kBatch = 4;                // heads in flight of a thread

struct Args {
  RotaryProblem p;
  int pair_chunks;     // pieces of V pairs (halves) or of V values (interleaved) that are turned
  int chunks;          // with those that are copied
};

__device__ __forceinline__ float2 turn(unsigned long long turns, int position, float amplitude) {
  const unsigned long long at = turns * static_cast<unsigned long long>(static_cast<long long>(position));
  float s, c;
  sincospif(static_cast<float>(static_cast<int>(at >> 32)) * 4.656612873077393e-10f, &s, &c);   // 2^-31
  return make_float2(c * amplitude, s * amplitude);
}

template <int V>
struct Piece;
template <>
struct Piece<8> { using type = uint4; };
template <>
struct Piece<4> { using type = uint2; };
template <>
struct Piece<2> { using type = uint32_t; };
template <>
struct Piece<1> { using type = uint16_t; };

// V values as they lie in memory
template <int V>
union Values {
  typename Piece<V>::type raw;
  uint16_t u[V];
};

// V values at a time.  Halves: a piece is V values of the first half and their partners of the second.  Interleaved:
// V / 2 pairs side by side.
template <typename T, int V, bool INTERLEAVED>
__global__ void __launch_bounds__(256) k_rotary(const __grid_constant__ Args a) {
  using Tr = F16Traits<T>;
  using P = typename Piece<V>::type;
  const RotaryProblem& p = a.p;
  __shared__ float2 cs[128];
  __shared__ long long k_row, v_row;
  decode::pdl_launch_dependents();
  decode::pdl_wait();
  const int t = blockIdx.x, half = p.rot_dim / 2, D = p.head_dim;
  const int lanes = blockDim.x / a.chunks;               // heads at a time
  const int chunk = threadIdx.x % a.chunks, head0 = threadIdx.x / a.chunks;
  const bool mine = head0 < lanes, turned = chunk < a.pair_chunks;
  // the piece's first values and, of halves, their partners: copied pieces lie one after the other
  const int at = INTERLEAVED || turned ? chunk * V : p.rot_dim + (chunk - a.pair_chunks) * V;
  const bool two = !INTERLEAVED && turned;
  const int rows = p.heads + p.kv_heads * (p.slots ? 2 : 1);
  // row: q's heads, then k's, then v's
  auto source = [&](int row) {
    if (row < p.heads) return static_cast<const T*>(p.q) + t * p.q_token + static_cast<long long>(row) * D;
    if (row < p.heads + p.kv_heads) return static_cast<const T*>(p.k) + t * p.k_token + static_cast<long long>(row - p.heads) * D;
    return static_cast<const T*>(p.v) + t * p.v_token + static_cast<long long>(row - p.heads - p.kv_heads) * D;
  };
  Values<V> x[kBatch], y[kBatch];
  auto load = [&](int row0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int row = row0 + i * lanes;
      if (mine && row < rows) {
        const T* from = source(row) + at;
        x[i].raw = *reinterpret_cast<const P*>(from);
        if (two) y[i].raw = *reinterpret_cast<const P*>(from + half);
      }
    }
  };
  load(head0);
  for (int i = threadIdx.x; i < half; i += blockDim.x) cs[i] = turn(p.turns[i], p.positions[t], p.amplitude);
  if (threadIdx.x == blockDim.x - 1) {
    k_row = v_row = -1;
    if (p.slots) {
      const long long slot = p.slots[t];
      if (slot >= static_cast<long long>(p.pages) * p.page_size) {
        atomicOr(p.status, kStatusSlotRange);
      } else if (slot >= 0) {
        // (a 64-bit division costs a few hundred cycles, and slots mostly fit 32 bits)
        const long long page = slot >> 32 ? slot / p.page_size : static_cast<unsigned>(slot) / static_cast<unsigned>(p.page_size);
        const long long place = slot - page * p.page_size;
        k_row = page * p.k_page + place * p.k_slot;
        v_row = page * p.v_page + place * p.v_slot;
      }
    }
  }
  __syncthreads();
  constexpr int kPairs = INTERLEAVED ? (V + 1) / 2 : V;
  float2 r[kPairs];
  if (turned) {
#pragma unroll
    for (int j = 0; j < kPairs; ++j) r[j] = cs[(INTERLEAVED ? chunk * (V / 2) : chunk * V) + j];
  }
  const long long k_at = k_row, v_at = v_row;
  for (int row0 = head0; mine && row0 < rows; row0 += kBatch * lanes) {
    if (row0 != head0) load(row0);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int row = row0 + i * lanes;
      if (row >= rows) continue;
      const bool value = row >= p.heads + p.kv_heads;
      if (turned && !value) {
        auto f = [](uint16_t u) { return Tr::to_f32(Tr::from_bits(u)); };
        auto g = [](float v) { return Tr::bits(Tr::from_f32(v)); };
        if constexpr (INTERLEAVED) {
#pragma unroll
          for (int j = 0; j < V / 2; ++j) {
            const float c = f(x[i].u[2 * j]), d = f(x[i].u[2 * j + 1]);
            x[i].u[2 * j] = g(c * r[j].x - d * r[j].y);
            x[i].u[2 * j + 1] = g(c * r[j].y + d * r[j].x);
          }
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float c = f(x[i].u[j]), d = f(y[i].u[j]);
            x[i].u[j] = g(c * r[j].x - d * r[j].y);
            y[i].u[j] = g(c * r[j].y + d * r[j].x);
          }
        }
      }
      auto put = [&](T* to) {
        *reinterpret_cast<P*>(to + at) = x[i].raw;
        if (two) *reinterpret_cast<P*>(to + at + half) = y[i].raw;
      };
      if (row < p.heads) {
        put(static_cast<T*>(p.q_out) + t * p.qo_token + static_cast<long long>(row) * D);
      } else if (!value) {
        const int h = row - p.heads;
        if (p.k_out) put(static_cast<T*>(p.k_out) + t * p.ko_token + static_cast<long long>(h) * D);
        if (k_at >= 0) put(static_cast<T*>(p.k_cache) + k_at + h * p.k_head);
      } else if (v_at >= 0) {
        put(static_cast<T*>(p.v_cache) + v_at + (row - p.heads - p.kv_heads) * p.v_head);
      }
    }
  }
}

template <typename T, int V, bool INTERLEAVED>
cudaError_t launch(const RotaryProblem& p, cudaStream_t stream) {
  Args a;
  a.p = p;
  a.pair_chunks = INTERLEAVED ? p.rot_dim / V : p.rot_dim / 2 / V;
  a.chunks = a.pair_chunks + (p.head_dim - p.rot_dim) / V;
  // as many threads as take the heads at kBatch a thread, in whole warps, from 64 to 256 (which hold any head's pieces)
  const int rows = p.heads + p.kv_heads * (p.slots ? 2 : 1);
  long long want = static_cast<long long>((rows + kBatch - 1) / kBatch) * a.chunks;
  want = (want + 31) / 32 * 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.tokens);
  cfg.blockDim = dim3(static_cast<unsigned>(want < 64 ? 64 : (want > 256 ? 256 : want)));
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_rotary<T, V, INTERLEAVED>, a);
}

template <typename T>
cudaError_t launch_layout(const RotaryProblem& p, cudaStream_t stream) {
  // rows, head_dim and so the copied part's end are multiples of 8 values; the pieces' size goes by the turned part
  if (p.interleaved)
    return p.rot_dim % 8 == 0 ? launch<T, 8, true>(p, stream) : launch<T, 2, true>(p, stream);
  const int half = p.rot_dim / 2;
  if (half % 8 == 0) return launch<T, 8, false>(p, stream);
  if (half % 4 == 0) return launch<T, 4, false>(p, stream);
  return launch<T, 1, false>(p, stream);
}

}  // namespace rotary

cudaError_t launch_rotary(const RotaryProblem& p, cudaStream_t stream) {
  return p.dtype == 0 ? rotary::launch_layout<__half>(p, stream) : rotary::launch_layout<__nv_bfloat16>(p, stream);
}

}  // namespace gptq
