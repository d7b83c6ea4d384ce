// serving_internal.h -- host-side launch interface between the C ABI of the decode-step operators
// (serving_api.cu) and their kernels.  Not installed; the public interface is
// include/gptq_serving.h.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gptq {

constexpr unsigned kStatusPageRange = 0x20u;
constexpr unsigned kStatusSeqLen = 0x40u;
constexpr unsigned kStatusNoToken = 0x80u;

// The status word of the current device, GPTQ_OK or a negative gptq_status (not an sm_103 part, a
// failed runtime call).
int device_status_word(unsigned** status);

// Every field checked by the C ABI before a launcher sees it.
struct AttentionProblem {
  const void* q;
  int batch, heads, dtype;
  void* k_cache;
  void* v_cache;
  int pages, page_size, kv_heads, head_dim;
  long long q_batch, kn_batch, vn_batch, k_page, k_slot, k_head, v_page, v_slot, v_head;
  const int32_t* table;
  int table_width;
  const int32_t* lens;
  const void* k_new;
  const void* v_new;
  float scale;
  int window;
  void* out;
  float* lse;
  void* workspace;
  unsigned* status;
};
size_t attention_workspace_bytes(int heads, int kv_heads, int head_dim);
cudaError_t launch_paged_attention(const AttentionProblem& p, cudaStream_t stream);

struct PackedExperts {
  const int32_t* qweight;
  const int32_t* qzeros;
  const void* scales;
};
struct MoeProblem {
  const void* x;
  int tokens, hidden, inter, dtype;
  const void* router;
  int experts, topk, renormalize;
  PackedExperts up, down;
  int bits, group_up, group_down, zero_offset;   // group: K where the caller passed -1
  void* out;
  int32_t* ids;
  float* weights;
  void* workspace;
  unsigned* status;
};
size_t moe_workspace_bytes(int tokens, int hidden, int inter, int experts, int topk);
cudaError_t launch_moe(const MoeProblem& p, cudaStream_t stream);

struct SampleProblem {
  const void* logits;
  int batch, vocab;
  long long row_stride;
  int dtype;                       // 0 fp16, 1 bf16, 2 fp32
  const float* uniform;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int32_t* token;
  float* logprob;
  unsigned* status;
};
cudaError_t launch_sample(const SampleProblem& p, cudaStream_t stream);

}  // namespace gptq
