// moe_b2.cu -- 2-bit instantiations of the expert products, in their own translation unit so that
// they compile in parallel with the rest.
#include "moe.cuh"

namespace gptq {
cudaError_t launch_moe_b2(const moe::Args& up, const int32_t* up_qweight, const moe::Args& down,
                          const int32_t* down_qweight, int experts, int* down_grid, cudaStream_t stream) {
  return moe::launch_bits<2>(up, up_qweight, down, down_qweight, experts, down_grid, stream);
}
}  // namespace gptq
