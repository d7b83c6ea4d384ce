// chunk_attention_bf16.cu -- chunk attention of bf16 models.
#include "chunk_attention.cuh"

namespace gptq {
namespace chunk {

cudaError_t launch_bf16(const Args& a, cudaStream_t stream) { return launch_dim<__nv_bfloat16>(a, stream); }

}  // namespace chunk
}  // namespace gptq
