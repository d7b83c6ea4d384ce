// chunk_attention.cu -- host side of chunk attention (chunk_attention.cuh).
#include "chunk_attention.cuh"

namespace gptq {

size_t chunk_attention_workspace_bytes(int, int, int head_dim) {
  const size_t floats = head_dim <= 64 ? chunk::partial_floats<64>()
                                       : (head_dim <= 128 ? chunk::partial_floats<128>() : chunk::partial_floats<256>());
  return chunk::kRecordBytes + static_cast<size_t>(chunk::kMaxRuns) * 2 * floats * 4;
}

cudaError_t launch_chunk_attention(const ChunkProblem& p, cudaStream_t stream) {
  chunk::Args a = {};
  a.p = p;
  a.group = p.heads / p.kv_heads;
  a.negative = p.scale < 0.f;
  a.scale_log2 = (a.negative ? -p.scale : p.scale) * 1.44269504088896341f;
  // hidden scores are -inf, which times 0 is no number
  if (a.scale_log2 == 0.f) a.scale_log2 = 1.17549435e-38f;
  // m = ceil(2^(30 + L) / d) with 2^L >= d: n m / 2^(30 + L) is off by less than 1 / d for n < 2^30
  auto divisor = [](unsigned d, unsigned* mul, unsigned* shift) {
    unsigned log = 0;
    while ((1ull << log) < d) ++log;
    *shift = 30 + log;
    *mul = static_cast<unsigned>(((1ull << *shift) + d - 1) / d);
  };
  divisor(static_cast<unsigned>(p.page_size), &a.page_mul, &a.page_shift);
  divisor(static_cast<unsigned>(a.group), &a.group_mul, &a.group_shift);
  a.k_page16 = static_cast<unsigned>(p.k_page / 8);
  a.k_slot16 = static_cast<unsigned>(p.k_slot / 8);
  a.k_head16 = static_cast<unsigned>(p.k_head / 8);
  a.v_page16 = static_cast<unsigned>(p.v_page / 8);
  a.v_slot16 = static_cast<unsigned>(p.v_slot / 8);
  a.v_head16 = static_cast<unsigned>(p.v_head / 8);
  a.records = static_cast<chunk::Record*>(p.workspace);
  a.partials = reinterpret_cast<float*>(static_cast<char*>(p.workspace) + chunk::kRecordBytes);
  return p.dtype == 0 ? chunk::launch_f16(a, stream) : chunk::launch_bf16(a, stream);
}

}  // namespace gptq
