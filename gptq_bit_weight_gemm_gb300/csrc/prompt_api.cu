// prompt_api.cu -- the C ABI of a prompt step's operators (include/gptq_prompt.h): host-side validation
// and dispatch, and the table of rotary frequencies (host).
#include <cuda_runtime.h>
#include <math.h>

#include "../../include/gptq_prompt.h"
#include "gptq_internal.h"
#include "prompt_internal.h"

namespace gptq {
namespace {

bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int to_status(cudaError_t e) { return e == cudaSuccess ? GPTQ_OK : GPTQ_ERR_CUDA; }

bool float_type(int dtype) { return dtype == GPTQ_F16 || dtype == GPTQ_BF16 || dtype == GPTQ_F32; }
size_t type_size(int dtype) { return dtype == GPTQ_F32 ? 4 : 2; }

bool head_dim_ok(int head_dim) { return head_dim > 0 && head_dim <= 256 && head_dim % 8 == 0; }

// Strides of a cache in elements, each a multiple of 8 where its dimension is stepped over (0 where it is
// not), and its last element within 2^35 of the first: rows are found by 32-bit offsets in 16-byte units.
int cache_strides(const long long* strides, int pages, int page_size, int kv_heads, int head_dim, long long* st) {
  const int steps[3] = {pages, page_size, kv_heads};
  __int128 last = head_dim;
  for (int i = 0; i < 3; ++i) {
    st[i] = steps[i] > 1 ? strides[i] : 0;
    if (st[i] < 0 || st[i] % 8) return GPTQ_ERR_ALIGN;
  }
  for (int i = 0; i < 3; ++i) {
    if (st[i] > (1ll << 40)) return GPTQ_ERR_SHAPE;
    last += static_cast<__int128>(steps[i] - 1) * st[i];
  }
  return last > (static_cast<__int128>(1) << 35) ? GPTQ_ERR_SHAPE : GPTQ_OK;
}

}  // namespace
}  // namespace gptq

extern "C" int gptq_page_plan(const int32_t* cached, const int32_t* added, int batch, int page_size, int32_t* block_table,
                              int table_width, int32_t* free_pages, int free_capacity, const int32_t* free_count,
                              int32_t* free_count_out, int32_t* seq_lens, int32_t* cu_tokens, int32_t* positions,
                              long long* slots, int max_tokens, void* stream) {
  using gptq::aligned_to;
  if (batch < 0 || batch > gptq::kMaxPlanBatch || page_size <= 0 || table_width <= 0 || free_capacity < 0 ||
      free_capacity > (1 << 30) || max_tokens < 0 || max_tokens > (1 << 30))
    return GPTQ_ERR_SHAPE;
  if (static_cast<long long>(table_width) * page_size > (1ll << 30)) return GPTQ_ERR_SHAPE;
  if (!free_count || !free_count_out || !cu_tokens) return GPTQ_ERR_ARG;
  if (batch > 0 && (!cached || !added || !block_table || !seq_lens)) return GPTQ_ERR_ARG;
  if ((free_capacity > 0 && !free_pages) || (max_tokens > 0 && (!positions || !slots))) return GPTQ_ERR_ARG;
  if (!aligned_to(cached, 4) || !aligned_to(added, 4) || !aligned_to(block_table, 4) || !aligned_to(free_pages, 4) ||
      !aligned_to(free_count, 4) || !aligned_to(free_count_out, 4) || !aligned_to(seq_lens, 4) ||
      !aligned_to(cu_tokens, 4) || !aligned_to(positions, 4) || !aligned_to(slots, 8))
    return GPTQ_ERR_ALIGN;
  gptq::PlanProblem p = {};
  const int rc = gptq::device_status_word(&p.status);
  if (rc) return rc;
  p.cached = cached; p.added = added; p.batch = batch; p.page_size = page_size;
  p.table = block_table; p.table_width = table_width;
  p.free_pages = free_pages; p.free_capacity = free_capacity;
  p.free_count = free_count; p.free_count_out = free_count_out;
  p.seq_lens = seq_lens; p.cu_tokens = cu_tokens; p.positions = positions; p.slots = slots; p.max_tokens = max_tokens;
  return gptq::to_status(gptq::launch_page_plan(p, static_cast<cudaStream_t>(stream)));
}

extern "C" int gptq_rms_norm(const void* x, int rows, int hidden, long long x_stride, int dtype, const void* residual,
                             long long residual_stride, int residual_dtype, void* residual_out,
                             long long residual_out_stride, const void* weight, int weight_dtype, float eps, void* out,
                             long long out_stride, int out_dtype, void* stream) {
  using gptq::aligned_to;
  using gptq::type_size;
  if (!gptq::float_type(dtype) || !gptq::float_type(out_dtype) || (weight && !gptq::float_type(weight_dtype)) ||
      (residual && !gptq::float_type(residual_dtype)))
    return GPTQ_ERR_ARG;
  if ((residual == nullptr) != (residual_out == nullptr)) return GPTQ_ERR_ARG;
  if (rows < 0 || hidden <= 0 || hidden > (1 << 20)) return GPTQ_ERR_SHAPE;
  // the stride of a single row is never stepped over
  if (rows > 1 && (x_stride < hidden || out_stride < hidden ||
                   (residual && (residual_stride < hidden || residual_out_stride < hidden))))
    return GPTQ_ERR_SHAPE;
  if (rows == 0) return GPTQ_OK;
  if (!x || !out) return GPTQ_ERR_ARG;
  if (!aligned_to(x, type_size(dtype)) || !aligned_to(out, type_size(out_dtype)) ||
      (weight && !aligned_to(weight, type_size(weight_dtype))) ||
      (residual && (!aligned_to(residual, type_size(residual_dtype)) || !aligned_to(residual_out, type_size(residual_dtype)))))
    return GPTQ_ERR_ALIGN;
  // a row is read whole before it is written only where both are the same bytes
  if (out == x && (out_dtype != dtype || (rows > 1 && out_stride != x_stride))) return GPTQ_ERR_ARG;
  if (residual && residual_out == residual && rows > 1 && residual_out_stride != residual_stride) return GPTQ_ERR_ARG;
  if (residual && (residual_out == x || residual_out == out || out == residual)) return GPTQ_ERR_ARG;
  gptq::NormProblem p = {};
  unsigned* status = nullptr;
  const int rc = gptq::device_status_word(&status);
  if (rc) return rc;
  p.x = x; p.rows = rows; p.hidden = hidden; p.x_stride = rows > 1 ? x_stride : hidden; p.dtype = dtype;
  p.residual = residual; p.residual_stride = rows > 1 ? residual_stride : hidden; p.residual_dtype = residual_dtype;
  p.residual_out = residual_out; p.residual_out_stride = rows > 1 ? residual_out_stride : hidden;
  p.weight = weight; p.weight_dtype = weight_dtype; p.eps = eps;
  p.out = out; p.out_stride = rows > 1 ? out_stride : hidden; p.out_dtype = out_dtype;
  return gptq::to_status(gptq::launch_rms_norm(p, static_cast<cudaStream_t>(stream)));
}

extern "C" int gptq_rotary_table(int rot_dim, double theta, int scaling, double factor, double original, double low,
                                 double high, unsigned long long* turns, double* amplitude) {
  if (rot_dim < 2 || rot_dim > 65536 || rot_dim % 2) return GPTQ_ERR_SHAPE;
  if (!turns || !amplitude || scaling < GPTQ_ROTARY_NONE || scaling > GPTQ_ROTARY_BANDS) return GPTQ_ERR_ARG;
  // (written so that a NaN is refused)
  if (!(theta > 1.0 && theta < 1e300)) return GPTQ_ERR_ARG;
  if (scaling != GPTQ_ROTARY_NONE && !(factor >= 1.0 && factor < 1e9)) return GPTQ_ERR_ARG;
  const bool limits = scaling == GPTQ_ROTARY_RAMP || scaling == GPTQ_ROTARY_BANDS;
  if (limits && !(original > 0.0 && original < 1e18 && low > 0.0 && high > low && high < 1e18)) return GPTQ_ERR_ARG;
  const double two_pi = 6.283185307179586476925;
  double base = theta;
  if (scaling == GPTQ_ROTARY_BASE && rot_dim > 2) base = theta * pow(factor, static_cast<double>(rot_dim) / (rot_dim - 2));
  double first = 0.0, last = 0.0;      // RAMP: the pairs that turn `high` and `low` times over `original`
  if (scaling == GPTQ_ROTARY_RAMP) {
    const double per = rot_dim / (2.0 * log(theta));
    first = fmax(floor(per * log(original / (high * two_pi))), 0.0);
    last = fmin(ceil(per * log(original / (low * two_pi))), rot_dim - 1.0);
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = pow(base, -2.0 * i / rot_dim);
    if (scaling == GPTQ_ROTARY_LINEAR) f /= factor;
    if (limits) {
      double keep;
      if (scaling == GPTQ_ROTARY_RAMP)
        keep = i >= last ? 0.0 : 1.0 - (i - first) / fmax(last - first, 0.001);   // (last may lie before the first pair)
      else
        keep = (original * f / two_pi - low) / (high - low);
      keep = fmin(fmax(keep, 0.0), 1.0);
      f = f / factor * (1.0 - keep) + f * keep;
    }
    turns[i] = static_cast<unsigned long long>(ldexp(f / two_pi, 64) + 0.5);   // f <= 1: below 2^62
  }
  *amplitude = scaling == GPTQ_ROTARY_RAMP ? 0.1 * log(factor) + 1.0 : 1.0;
  return GPTQ_OK;
}

extern "C" int gptq_rotary(const void* q, const void* k, const void* v, int tokens, int heads, int kv_heads, int head_dim,
                           int rot_dim, int interleaved, int dtype, const long long* strides, const int32_t* positions,
                           const unsigned long long* turns, float amplitude, void* q_out, void* k_out, void* k_cache,
                           void* v_cache, int pages, int page_size, const long long* slots, void* stream) {
  using gptq::aligned_to;
  if (dtype != GPTQ_F16 && dtype != GPTQ_BF16) return GPTQ_ERR_ARG;
  if ((interleaved != 0 && interleaved != 1) || !strides) return GPTQ_ERR_ARG;
  const bool append = k_cache != nullptr;
  if ((v_cache != nullptr) != append) return GPTQ_ERR_ARG;
  if (tokens < 0 || heads <= 0 || kv_heads <= 0 || heads > (1 << 16) || kv_heads > (1 << 16) || !gptq::head_dim_ok(head_dim) ||
      rot_dim < 2 || rot_dim % 2 || rot_dim > head_dim || (append && (pages <= 0 || page_size <= 0)))
    return GPTQ_ERR_SHAPE;
  if (tokens == 0) return GPTQ_OK;
  if (!q || !k || !positions || !turns || !q_out || (!k_out && !append) || (append && (!v || !slots))) return GPTQ_ERR_ARG;
  gptq::RotaryProblem p = {};
  long long st[5];
  const bool used[5] = {true, true, append, true, k_out != nullptr};
  const long long least[5] = {static_cast<long long>(heads) * head_dim, static_cast<long long>(kv_heads) * head_dim,
                              static_cast<long long>(kv_heads) * head_dim, static_cast<long long>(heads) * head_dim,
                              static_cast<long long>(kv_heads) * head_dim};
  for (int i = 0; i < 5; ++i) {
    st[i] = used[i] && tokens > 1 ? strides[i] : 0;
    if (st[i] < 0 || st[i] % 8) return GPTQ_ERR_ALIGN;
    // rows of an output that overlap would be written by several tokens
    if (i >= 3 && used[i] && tokens > 1 && st[i] < least[i]) return GPTQ_ERR_SHAPE;
  }
  if (append) {
    long long ks[3], vs[3];
    int rc = gptq::cache_strides(strides + 5, pages, page_size, kv_heads, head_dim, ks);
    if (rc == GPTQ_OK) rc = gptq::cache_strides(strides + 8, pages, page_size, kv_heads, head_dim, vs);
    if (rc) return rc;
    // rows of a cache that overlap would be written by several heads or tokens
    const int steps[3] = {pages, page_size, kv_heads};
    for (int i = 0; i < 3; ++i)
      if (steps[i] > 1 && (ks[i] < head_dim || vs[i] < head_dim)) return GPTQ_ERR_SHAPE;
    p.k_page = ks[0]; p.k_slot = ks[1]; p.k_head = ks[2];
    p.v_page = vs[0]; p.v_slot = vs[1]; p.v_head = vs[2];
  }
  // in place: a token's values are read before they are written only by the same place
  if ((q_out == q && tokens > 1 && st[3] != st[0]) || (k_out && k_out == k && tokens > 1 && st[4] != st[1])) return GPTQ_ERR_ARG;
  if (!aligned_to(q, 16) || !aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(q_out, 16) || !aligned_to(k_out, 16) ||
      !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) || !aligned_to(positions, 4) || !aligned_to(turns, 8) ||
      !aligned_to(slots, 8))
    return GPTQ_ERR_ALIGN;
  const int rc = gptq::device_status_word(&p.status);
  if (rc) return rc;
  p.q = q; p.k = k; p.v = append ? v : nullptr;
  p.tokens = tokens; p.heads = heads; p.kv_heads = kv_heads; p.head_dim = head_dim; p.rot_dim = rot_dim;
  p.interleaved = interleaved; p.dtype = dtype;
  p.q_token = st[0]; p.k_token = st[1]; p.v_token = st[2]; p.qo_token = st[3]; p.ko_token = st[4];
  p.positions = positions; p.turns = turns; p.amplitude = amplitude;
  p.q_out = q_out; p.k_out = k_out; p.k_cache = k_cache; p.v_cache = v_cache;
  p.pages = pages; p.page_size = page_size; p.slots = append ? slots : nullptr;
  return gptq::to_status(gptq::launch_rotary(p, static_cast<cudaStream_t>(stream)));
}

namespace {
thread_local unsigned chunk_wait_ns = gptq::kChunkWaitNs;
}

extern "C" int gptq_selftest_chunk_attention_wait(unsigned limit_ns) {
  if (limit_ns > 4000000000u) return GPTQ_ERR_ARG;
  chunk_wait_ns = limit_ns ? limit_ns : gptq::kChunkWaitNs;
  return GPTQ_OK;
}

extern "C" size_t gptq_chunk_attention_workspace_size(int heads, int kv_heads, int head_dim) {
  if (heads <= 0 || kv_heads <= 0 || heads % kv_heads || heads > (1 << 16) || !gptq::head_dim_ok(head_dim)) return 0;
  return gptq::chunk_attention_workspace_bytes(heads, kv_heads, head_dim);
}

extern "C" int gptq_chunk_attention(const void* q, int tokens, int heads, int dtype, const void* k_cache,
                                    const void* v_cache, int pages, int page_size, int kv_heads, int head_dim,
                                    const long long* strides, const int32_t* block_table, int table_width,
                                    const int32_t* seq_lens, const int32_t* cu_tokens, int batch, float scale, int window,
                                    void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  using gptq::aligned_to;
  if (dtype != GPTQ_F16 && dtype != GPTQ_BF16) return GPTQ_ERR_ARG;
  if (!strides) return GPTQ_ERR_ARG;
  if (tokens < 0 || batch < 0 || heads <= 0 || kv_heads <= 0 || heads % kv_heads || heads > (1 << 16) ||
      !gptq::head_dim_ok(head_dim) || pages <= 0 || page_size <= 0 || table_width <= 0 || window < 0)
    return GPTQ_ERR_SHAPE;
  // key positions and the count of rows are 32-bit
  if (static_cast<long long>(table_width) * page_size > (1ll << 30)) return GPTQ_ERR_SHAPE;
  if (static_cast<long long>(tokens) * heads > (1ll << 30) || static_cast<long long>(batch) * heads > (1ll << 30))
    return GPTQ_ERR_SHAPE;
  if (batch == 0 || tokens == 0) return GPTQ_OK;
  if (!q || !k_cache || !v_cache || !block_table || !seq_lens || !cu_tokens || !out || !workspace) return GPTQ_ERR_ARG;
  const long long q_token = tokens > 1 ? strides[0] : 0;
  if (q_token < 0 || q_token % 8) return GPTQ_ERR_ALIGN;
  long long ks[3], vs[3];
  int rc = gptq::cache_strides(strides + 1, pages, page_size, kv_heads, head_dim, ks);
  if (rc == GPTQ_OK) rc = gptq::cache_strides(strides + 4, pages, page_size, kv_heads, head_dim, vs);
  if (rc) return rc;
  if (!aligned_to(q, 16) || !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) || !aligned_to(out, 16) ||
      !aligned_to(workspace, 16) || !aligned_to(block_table, 4) || !aligned_to(seq_lens, 4) || !aligned_to(cu_tokens, 4) ||
      !aligned_to(lse, 4))
    return GPTQ_ERR_ALIGN;
  if (workspace_bytes < gptq_chunk_attention_workspace_size(heads, kv_heads, head_dim)) return GPTQ_ERR_WORKSPACE;
  gptq::ChunkProblem p = {};
  rc = gptq::device_status_word(&p.status);
  if (rc) return rc;
  p.q = q; p.tokens = tokens; p.heads = heads; p.dtype = dtype;
  p.k_cache = k_cache; p.v_cache = v_cache; p.pages = pages; p.page_size = page_size;
  p.kv_heads = kv_heads; p.head_dim = head_dim; p.q_token = q_token;
  p.k_page = ks[0]; p.k_slot = ks[1]; p.k_head = ks[2];
  p.v_page = vs[0]; p.v_slot = vs[1]; p.v_head = vs[2];
  p.table = block_table; p.table_width = table_width; p.lens = seq_lens; p.cu = cu_tokens; p.batch = batch;
  // (positions are below 2^30: a wider window hides nothing, and differences with it stay in 32 bits)
  p.scale = scale; p.window = window < (1 << 30) ? window : 1 << 30;
  p.out = out; p.lse = lse; p.workspace = workspace; p.wait_ns = chunk_wait_ns;
  return gptq::to_status(gptq::launch_chunk_attention(p, static_cast<cudaStream_t>(stream)));
}
