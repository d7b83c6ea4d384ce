// prompt_internal.h -- host-side launch interface between the C ABI of a prompt step's operators
// (prompt_api.cu) and their kernels.  Not installed; the public interface is include/gptq_prompt.h.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "serving_internal.h"

namespace gptq {

constexpr unsigned kStatusNoPage = 0x100u;
constexpr unsigned kStatusSlotRange = 0x200u;
constexpr unsigned kStatusTokenRows = 0x400u;

constexpr int kMaxPlanBatch = 8192;

// Every field checked by the C ABI before a launcher sees it.
struct PlanProblem {
  const int32_t* cached;
  const int32_t* added;
  int batch, page_size;
  int32_t* table;
  int table_width;
  int32_t* free_pages;
  int free_capacity;
  const int32_t* free_count;
  int32_t* free_count_out;
  int32_t* seq_lens;
  int32_t* cu_tokens;
  int32_t* positions;
  long long* slots;
  int max_tokens;
  unsigned* status;
};
cudaError_t launch_page_plan(const PlanProblem& p, cudaStream_t stream);

struct NormProblem {
  const void* x;
  int rows, hidden;
  long long x_stride;
  int dtype;                       // 0 fp16, 1 bf16, 2 fp32, here and below
  const void* residual;
  long long residual_stride;
  int residual_dtype;
  void* residual_out;
  long long residual_out_stride;
  const void* weight;
  int weight_dtype;
  float eps;
  void* out;
  long long out_stride;
  int out_dtype;
};
cudaError_t launch_rms_norm(const NormProblem& p, cudaStream_t stream);

struct RotaryProblem {
  const void* q;
  const void* k;
  const void* v;
  int tokens, heads, kv_heads, head_dim, rot_dim, interleaved, dtype;
  long long q_token, k_token, v_token, qo_token, ko_token;
  long long k_page, k_slot, k_head, v_page, v_slot, v_head;
  const int32_t* positions;
  const unsigned long long* turns;
  float amplitude;
  void* q_out;
  void* k_out;
  void* k_cache;
  void* v_cache;
  int pages, page_size;
  const long long* slots;
  unsigned* status;
};
cudaError_t launch_rotary(const RotaryProblem& p, cudaStream_t stream);

struct ChunkProblem {
  const void* q;
  int tokens, heads, dtype;
  const void* k_cache;
  const void* v_cache;
  int pages, page_size, kv_heads, head_dim;
  long long q_token, k_page, k_slot, k_head, v_page, v_slot, v_head;
  const int32_t* table;
  int table_width;
  const int32_t* lens;
  const int32_t* cu;
  int batch;
  float scale;
  int window;
  void* out;
  float* lse;
  void* workspace;
  unsigned* status;
  unsigned wait_ns;                // after which a wait inside the kernel gives up
};
constexpr unsigned kChunkWaitNs = 2000000000u;
size_t chunk_attention_workspace_bytes(int heads, int kv_heads, int head_dim);
cudaError_t launch_chunk_attention(const ChunkProblem& p, cudaStream_t stream);

}  // namespace gptq

// The library's own test hook: gptq_chunk_attention calls of this thread give up their waits after limit_ns (1 ns to 4 s;
// 0: as long as ever), so that a test can have a valid call run into its failure path: GPTQ_DEV_TIMEOUT, results
// that mean nothing, everything in flight waited for, and a context that stays usable.
extern "C" int gptq_selftest_chunk_attention_wait(unsigned limit_ns);
