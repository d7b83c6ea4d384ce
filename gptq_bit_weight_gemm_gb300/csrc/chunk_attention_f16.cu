// chunk_attention_f16.cu -- chunk attention of f16 models.
#include "chunk_attention.cuh"

namespace gptq {
namespace chunk {

cudaError_t launch_f16(const Args& a, cudaStream_t stream) { return launch_dim<__half>(a, stream); }

}  // namespace chunk
}  // namespace gptq
