// serving_api.cu -- the C ABI of the decode-step operators (include/gptq_serving.h): host-side
// validation and dispatch.
#include <cuda_runtime.h>

#include "../../include/gptq_serving.h"
#include "gptq_internal.h"
#include "serving_internal.h"

namespace gptq {
namespace {

bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int to_status(cudaError_t e) { return e == cudaSuccess ? GPTQ_OK : GPTQ_ERR_CUDA; }

constexpr int kMaxMoeTokens = kDecodeMaxM, kMaxMoeExperts = 1024, kMaxMoeTopk = 16;
constexpr int kMaxVocab = 1 << 22;

bool moe_shape_ok(int tokens, int hidden, int inter, int experts, int topk) {
  return tokens >= 1 && tokens <= kMaxMoeTokens && hidden > 0 && inter > 0 && hidden % 32 == 0 && inter % 32 == 0 &&
         inter <= (1 << 29) && experts >= 1 && experts <= kMaxMoeExperts && topk >= 1 && topk <= experts &&
         topk <= kMaxMoeTopk;
}

}  // namespace
}  // namespace gptq

extern "C" size_t gptq_paged_attention_workspace_size(int heads, int kv_heads, int head_dim) {
  if (heads <= 0 || kv_heads <= 0 || heads % kv_heads || head_dim <= 0 || head_dim > 256 || head_dim % 8) return 0;
  return gptq::attention_workspace_bytes(heads, kv_heads, head_dim);
}

extern "C" int gptq_paged_attention(const void* q, int batch, int heads, int dtype, void* k_cache, void* v_cache,
                                    int pages, int page_size, int kv_heads, int head_dim, const long long* strides,
                                    const int32_t* block_table, int table_width, const int32_t* seq_lens,
                                    const void* k_new, const void* v_new, float scale, int window, void* out,
                                    float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  using gptq::aligned_to;
  if (dtype != GPTQ_F16 && dtype != GPTQ_BF16) return GPTQ_ERR_ARG;
  if (!strides || (k_new == nullptr) != (v_new == nullptr)) return GPTQ_ERR_ARG;
  if (batch < 0 || heads <= 0 || kv_heads <= 0 || heads % kv_heads || head_dim <= 0 || head_dim > 256 || head_dim % 8 ||
      pages <= 0 || page_size <= 0 || table_width <= 0 || window < 0)
    return GPTQ_ERR_SHAPE;
  // key positions are 32-bit, and so is the count of (sequence, kv head, 16 query heads) items
  if (static_cast<long long>(table_width) * page_size > (1ll << 30)) return GPTQ_ERR_SHAPE;
  if (static_cast<long long>(batch) * heads > (1ll << 24)) return GPTQ_ERR_SHAPE;
  if (batch == 0) return GPTQ_OK;
  if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !out || !workspace) return GPTQ_ERR_ARG;
  // a dimension of one is never stepped over, whatever its stride
  const int steps[9] = {batch, batch, batch, pages, page_size, kv_heads, pages, page_size, kv_heads};
  long long st[9];
  for (int i = 0; i < 9; ++i) {
    st[i] = steps[i] > 1 ? strides[i] : 0;
    if (st[i] < 0 || st[i] % 8) return GPTQ_ERR_ALIGN;
  }
  // rows of a cache are found by 32-bit offsets in 16-byte units
  for (int i = 3; i < 9; i += 3) {
    if (st[i] > (1ll << 40) || st[i + 1] > (1ll << 40) || st[i + 2] > (1ll << 40)) return GPTQ_ERR_SHAPE;
    const __int128 last = static_cast<__int128>(pages - 1) * st[i] + static_cast<__int128>(page_size - 1) * st[i + 1] +
                          static_cast<__int128>(kv_heads - 1) * st[i + 2] + head_dim;
    if (last > (static_cast<__int128>(1) << 35)) return GPTQ_ERR_SHAPE;
  }
  if (!aligned_to(q, 16) || !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) || !aligned_to(k_new, 16) ||
      !aligned_to(v_new, 16) || !aligned_to(out, 16) || !aligned_to(workspace, 16) || !aligned_to(block_table, 4) ||
      !aligned_to(seq_lens, 4) || !aligned_to(lse, 4))
    return GPTQ_ERR_ALIGN;
  if (workspace_bytes < gptq_paged_attention_workspace_size(heads, kv_heads, head_dim)) return GPTQ_ERR_WORKSPACE;
  gptq::AttentionProblem p = {};
  const int rc = gptq::device_status_word(&p.status);
  if (rc) return rc;
  p.q = q; p.batch = batch; p.heads = heads; p.dtype = dtype;
  p.k_cache = k_cache; p.v_cache = v_cache; p.pages = pages; p.page_size = page_size;
  p.kv_heads = kv_heads; p.head_dim = head_dim;
  p.q_batch = st[0]; p.kn_batch = st[1]; p.vn_batch = st[2];
  p.k_page = st[3]; p.k_slot = st[4]; p.k_head = st[5];
  p.v_page = st[6]; p.v_slot = st[7]; p.v_head = st[8];
  p.table = block_table; p.table_width = table_width; p.lens = seq_lens;
  p.k_new = k_new; p.v_new = v_new; p.scale = scale; p.window = window;
  p.out = out; p.lse = lse; p.workspace = workspace;
  return gptq::to_status(gptq::launch_paged_attention(p, static_cast<cudaStream_t>(stream)));
}

extern "C" size_t gptq_moe_workspace_size(int tokens, int hidden, int inter, int experts, int topk) {
  if (!gptq::moe_shape_ok(tokens, hidden, inter, experts, topk)) return 0;
  return gptq::moe_workspace_bytes(tokens, hidden, inter, experts, topk);
}

extern "C" int gptq_moe(const void* x, int tokens, int hidden, int inter, int dtype, const void* router, int experts,
                        int topk, int renormalize, const int32_t* up_qweight, const int32_t* up_qzeros,
                        const void* up_scales, const int32_t* down_qweight, const int32_t* down_qzeros,
                        const void* down_scales, int bits, int group, int fmt, void* out, int32_t* ids, float* weights,
                        void* workspace, size_t workspace_bytes, void* stream) {
  using gptq::aligned_to;
  if (bits != 2 && bits != 3 && bits != 4 && bits != 8) return GPTQ_ERR_ARG;
  if (fmt != GPTQ_FMT_V1 && fmt != GPTQ_FMT_V2) return GPTQ_ERR_ARG;
  if (dtype != GPTQ_F16 && dtype != GPTQ_BF16) return GPTQ_ERR_ARG;
  if (renormalize != 0 && renormalize != 1) return GPTQ_ERR_ARG;
  if (tokens < 0) return GPTQ_ERR_SHAPE;
  if (!gptq::moe_shape_ok(tokens > 0 ? tokens : 1, hidden, inter, experts, topk)) return GPTQ_ERR_SHAPE;
  const int tile = bits == 3 ? 128 : 128 / bits;      // k values of one k-tile
  if (group != -1 && (group <= 0 || hidden % group || inter % group || group % tile)) return GPTQ_ERR_SHAPE;
  if (hidden % tile || inter % tile) return GPTQ_ERR_SHAPE;
  // rows of the stacked packed weights are 32-bit coordinates
  if (static_cast<long long>(experts) * (hidden > inter ? hidden : inter) / 32 * bits > 0x7FFFFFFFll)
    return GPTQ_ERR_SHAPE;
  if (tokens == 0) return GPTQ_OK;
  if (!x || !router || !up_qweight || !up_qzeros || !up_scales || !down_qweight || !down_qzeros || !down_scales ||
      !out || !workspace)
    return GPTQ_ERR_ARG;
  if (!aligned_to(x, 16) || !aligned_to(router, 16) || !aligned_to(up_qweight, 16) || !aligned_to(up_qzeros, 16) ||
      !aligned_to(up_scales, 16) || !aligned_to(down_qweight, 16) || !aligned_to(down_qzeros, 16) ||
      !aligned_to(down_scales, 16) || !aligned_to(out, 16) || !aligned_to(workspace, 16) || !aligned_to(ids, 4) ||
      !aligned_to(weights, 4))
    return GPTQ_ERR_ALIGN;
  if (workspace_bytes < gptq_moe_workspace_size(tokens, hidden, inter, experts, topk)) return GPTQ_ERR_WORKSPACE;
  gptq::MoeProblem p = {};
  const int rc = gptq::device_status_word(&p.status);
  if (rc) return rc;
  p.x = x; p.tokens = tokens; p.hidden = hidden; p.inter = inter; p.dtype = dtype;
  p.router = router; p.experts = experts; p.topk = topk; p.renormalize = renormalize;
  p.up = {up_qweight, up_qzeros, up_scales};
  p.down = {down_qweight, down_qzeros, down_scales};
  p.bits = bits;
  p.group_up = group == -1 ? hidden : group;
  p.group_down = group == -1 ? inter : group;
  p.zero_offset = fmt == GPTQ_FMT_V1 ? 1 : 0;
  p.out = out; p.ids = ids; p.weights = weights; p.workspace = workspace;
  return gptq::to_status(gptq::launch_moe(p, static_cast<cudaStream_t>(stream)));
}

extern "C" int gptq_sample(const void* logits, int batch, int vocab, long long row_stride, int dtype,
                           const float* uniform, const float* temperature, const int32_t* top_k, const float* top_p,
                           const float* min_p, int32_t* token, float* logprob, void* stream) {
  using gptq::aligned_to;
  if (dtype != GPTQ_F16 && dtype != GPTQ_BF16 && dtype != GPTQ_F32) return GPTQ_ERR_ARG;
  if (batch < 0 || vocab <= 0 || vocab > gptq::kMaxVocab || row_stride < vocab) return GPTQ_ERR_SHAPE;
  if (batch == 0) return GPTQ_OK;
  if (!logits || !uniform || !token) return GPTQ_ERR_ARG;
  if (!aligned_to(logits, dtype == GPTQ_F32 ? 4 : 2) || !aligned_to(uniform, 4) || !aligned_to(temperature, 4) ||
      !aligned_to(top_k, 4) || !aligned_to(top_p, 4) || !aligned_to(min_p, 4) || !aligned_to(token, 4) ||
      !aligned_to(logprob, 4))
    return GPTQ_ERR_ALIGN;
  gptq::SampleProblem p = {};
  const int rc = gptq::device_status_word(&p.status);
  if (rc) return rc;
  p.logits = logits; p.batch = batch; p.vocab = vocab; p.row_stride = row_stride; p.dtype = dtype;
  p.uniform = uniform; p.temperature = temperature; p.top_k = top_k; p.top_p = top_p; p.min_p = min_p;
  p.token = token; p.logprob = logprob;
  return gptq::to_status(gptq::launch_sample(p, static_cast<cudaStream_t>(stream)));
}
