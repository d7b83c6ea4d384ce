/*
 * gptq_serving.h -- the operators a decode step of a quantised model needs beside the GEMMs of
 * gptq.h: attention of the new token over a paged key-value cache, the mixture-of-experts layer for
 * a few tokens, and the choice of the next token.
 *
 * Conventions are those of gptq.h: every buffer belongs to the caller; device entry points run
 * asynchronously on `stream` (a cudaStream_t; NULL = legacy default stream) on the current device
 * and return GPTQ_OK or a negative gptq_status, with nothing launched when validation fails; dtype
 * is GPTQ_F16, GPTQ_BF16 or (logits) GPTQ_F32; kernels never trap, and what only the device can see
 * sets a bit in the status word read by gptq_get_device_status().  Every input is read only after
 * the kernels issued before the call on `stream` have completed.
 *
 * Workspaces: one serves any number of calls of any shape that it is large enough for, one after the
 * other on one stream; calls that overlap on the GPU need workspaces of their own.  The workspace of
 * gptq_paged_attention starts with a control block that has to be zero before its first use
 * (cudaMemset once, or a zeroed allocation); every call that runs leaves it zero again.
 */
#ifndef GPTQ_SERVING_H
#define GPTQ_SERVING_H

#include "gptq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GPTQ_F32 2                    /* gptq_sample: fp32 logits */

/* Further bits of the device status word. */
#define GPTQ_DEV_PAGE_RANGE 0x20u     /* gptq_paged_attention: a live key's block-table entry was
                                         outside [0, pages); its page's keys were left out       */
#define GPTQ_DEV_SEQ_LEN 0x40u        /* gptq_paged_attention: a length was negative (taken as 0)
                                         or longer than the block table (cut to it, and its new
                                         token neither appended nor used)                        */
#define GPTQ_DEV_NO_TOKEN 0x80u       /* gptq_sample: a row held no logit above -inf; its token
                                         is -1                                                   */

/*
 * gptq_paged_attention -- attention of one new token of each sequence over its cached keys and
 * values:  out[b, h] = sum_j p_j v_j,  p = softmax_j(scale * q[b, h] . k_j),  over the keys j in
 * [max(0, n - window), n) of sequence b, n = seq_lens[b] (window 0: all n), k and v of head
 * h / (heads / kv_heads).  Key j of sequence b is slot j % page_size of page
 * block_table[b, j / page_size].  Sums, maxima and accumulators are fp32, the probabilities enter
 * the product with v in 15 (bf16) or 20 (fp16) significant bits, out is rounded once.
 * A sequence of length 0 gives zeros.  Nothing past a sequence's length (or before its window) is
 * used, whatever it holds: neither cache slots nor block-table entries.
 *
 * k_new, v_new [batch, kv_heads, head_dim] (both or neither): the new token's own key and value.
 * They are written to slot n - 1 of their sequence and used as key n - 1 (length 0: ignored); no
 * two sequences may share the page that holds slot n - 1 of one of them.  Without them the cache
 * already holds key n - 1.
 *
 *   q            [batch, heads, head_dim]: rows of a sequence contiguous, sequences q_stride apart
 *   k/v_cache    [pages, page_size, kv_heads, head_dim] in any order of the first three, each
 *                head_dim values contiguous
 *   strides      HOST array of 9 strides in elements, multiples of 8 (anything where the dimension
 *                is one): q batch, k_new batch, v_new batch, k page, k slot, k head, v page, v slot,
 *                v head
 *   block_table  [batch, table_width] int32, seq_lens [batch] int32 (4-byte aligned)
 *   out          [batch, heads, head_dim] contiguous
 *   lse          nullable [batch, heads] fp32: log sum_j exp(scale * q . k_j), -inf for length 0
 * Everything 16-bit is of `dtype` and 16-byte aligned.  head_dim: a multiple of 8 up to 256; heads a
 * multiple of kv_heads; a cache spans at most 2^35 elements (64 GiB; GPTQ_ERR_SHAPE).  workspace:
 * gptq_paged_attention_workspace_size() bytes, 16-byte aligned, control block zero (above).
 * batch == 0 is a no-op.
 */
size_t gptq_paged_attention_workspace_size(int heads, int kv_heads, int head_dim);
int gptq_paged_attention(const void* q, int batch, int heads, int dtype, void* k_cache, void* v_cache,
                         int pages, int page_size, int kv_heads, int head_dim, const long long* strides,
                         const int32_t* block_table, int table_width, const int32_t* seq_lens,
                         const void* k_new, const void* v_new, float scale, int window, void* out,
                         float* lse, void* workspace, size_t workspace_bytes, void* stream);

/*
 * gptq_moe -- the whole mixture-of-experts layer for up to 32 tokens on packed expert weights:
 *   p = softmax(router x),  S = the topk experts of largest p (equal p: the lower index first),
 *   w_e = p_e (renormalize: p_e / sum_{S} p),
 *   out = sum_{e in S} w_e * down_e( silu(gate_e x) * up_e x ).
 * Every weight of an expert that no token chose is left unread.  Products are of exact (q - zero)
 * and accumulate in fp32; the inner activation silu(g) * u is kept as fp16 times a power of two for
 * each row's run of 128 values, in 11 significant bits for bf16 and in 22 (a sum of two) for fp16;
 * out is rounded once.
 *   x        [tokens, hidden] of dtype          router [experts, hidden] of dtype
 *   up_*     packed as for gptq_gemm_grouped, K = hidden, N = 2 * inter: columns [0, inter) are the
 *            gate, [inter, 2 * inter) the up projection
 *   down_*   the same with K = inter, N = hidden
 *   out      [tokens, hidden] of dtype
 *   ids, weights   nullable [tokens, topk]: the chosen experts in order (int32) and their w (fp32)
 * hidden, inter: multiples of 32; group: -1 or a divisor of both; the groups are whole k-tiles (a
 * multiple of 128 / bits, 128 for 3-bit; with -1 so are hidden and inter), topk <= experts <= 1024,
 * topk <= 16, tokens <= 32; otherwise GPTQ_ERR_SHAPE.  A token whose router logits hold a NaN gets
 * NaN.  workspace: gptq_moe_workspace_size() bytes (0 for a shape outside the limits), 16-byte
 * aligned, holding anything.  tokens == 0 is a no-op.
 */
size_t gptq_moe_workspace_size(int tokens, int hidden, int inter, int experts, int topk);
int gptq_moe(const void* x, int tokens, int hidden, int inter, int dtype, const void* router, int experts,
             int topk, int renormalize, const int32_t* up_qweight, const int32_t* up_qzeros,
             const void* up_scales, const int32_t* down_qweight, const int32_t* down_qzeros,
             const void* down_scales, int bits, int group, int fmt, void* out, int32_t* ids,
             float* weights, void* workspace, size_t workspace_bytes, void* stream);

/*
 * gptq_sample -- one token for each row of logits, from a given uniform number:
 *   x = (l - max l) / temperature, w = exp(x), tokens ordered by l descending, equal l by index;
 *   kept: the first top_k; of these the shortest prefix whose mass reaches top_p of theirs (a token
 *   stays while the mass before it is < top_p * total); of these those with w >= min_p (the best
 *   token always stays);
 *   token = the first kept index, in index order, whose cumulated w exceeds uniform * (kept mass).
 * l is taken to fp32 and x and w are fp32; each w is rounded to a whole multiple of 2^-39 of the best
 * token's (vocab * 2^-40 of the total at most) and these are summed exactly, so that the result does
 * not depend on an order of summation.
 *   logits       [batch, vocab] of dtype (GPTQ_F16, GPTQ_BF16, GPTQ_F32), rows row_stride elements
 *                apart; aligned to the element
 *   uniform      [batch] fp32 in [0, 1) (below 0 or NaN: 0; 1 and above: the last kept token)
 *   temperature  nullable [batch] fp32: 1 where absent; 0, negative or NaN: the best token
 *   top_k        nullable [batch] int32: off where absent or <= 0
 *   top_p        nullable [batch] fp32: off where absent or >= 1; <= 0 or NaN: the best token
 *   min_p        nullable [batch] fp32: off where absent or <= 0; NaN: the best token
 *   token        [batch] int32
 *   logprob      nullable [batch] fp32: the token's log probability among the kept
 * A NaN logit is never chosen; +inf logits share the mass among themselves; a row without a logit
 * above -inf gives token -1, logprob NaN and GPTQ_DEV_NO_TOKEN.  vocab up to 2^22, batch == 0 is a
 * no-op.
 */
int gptq_sample(const void* logits, int batch, int vocab, long long row_stride, int dtype,
                const float* uniform, const float* temperature, const int32_t* top_k, const float* top_p,
                const float* min_p, int32_t* token, float* logprob, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GPTQ_SERVING_H */
