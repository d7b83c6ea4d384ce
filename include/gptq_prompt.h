/*
 * gptq_prompt.h -- the operators a step of a quantised model needs when its sequences bring chunks of
 * prompts: the plan of the step's pages and slots, the root-mean-square norm with the residual's
 * addition, the rotary embedding with the append to the paged cache, and the attention of each
 * sequence's new tokens over its cached keys and values.  The cache and its block table are those of
 * gptq_paged_attention (gptq_serving.h), which serves steps of one token a sequence.
 *
 * A step's rows: the new tokens of all sequences one after the other, those of sequence b in rows
 * [cu_tokens[b], cu_tokens[b + 1]).
 *
 * Conventions are those of gptq.h and gptq_serving.h: every buffer belongs to the caller; device entry
 * points run asynchronously on `stream` on the current device and return GPTQ_OK or a negative
 * gptq_status, with nothing launched when validation fails; kernels never trap, and what only the
 * device can see sets a bit in the status word read by gptq_get_device_status().  Every input is read
 * only after the kernels issued before the call on `stream` have completed.  Calls that overlap on the
 * GPU need outputs and workspaces of their own.
 */
#ifndef GPTQ_PROMPT_H
#define GPTQ_PROMPT_H

#include "gptq_serving.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further bits of the device status word (gptq_chunk_attention and gptq_page_plan also set
   GPTQ_DEV_PAGE_RANGE and GPTQ_DEV_SEQ_LEN). */
#define GPTQ_DEV_NO_PAGE 0x100u       /* gptq_page_plan: the free list had no page left for a sequence, or
                                         no room for one given back                             */
#define GPTQ_DEV_SLOT_RANGE 0x200u    /* gptq_rotary: a slot past the cache; its token was not written */
#define GPTQ_DEV_TOKEN_ROWS 0x400u    /* gptq_page_plan: more new tokens than max_tokens;
                                         gptq_chunk_attention: cu_tokens decreasing or outside
                                         [0, tokens], cut to it                                 */

/*
 * gptq_page_plan -- lengths, rows, positions and slots of a step, and the pages it takes and gives back.
 * Sequence b holds cached[b] tokens in ceil(cached / page_size) pages, the first entries of its row of
 * block_table, and gets added[b] more (negative: its last tokens are dropped; -cached: it ends).
 *   1. Pages that no longer hold a token go back to the free list, in the order of sequences and pages.
 *   2. Pages are taken from the end of the list, in the same order, and entered into block_table.
 *   free_pages   [free_capacity] int32, of which the first *free_count are free pages; entries past the
 *                new count are left as they are
 *   seq_lens     [batch] int32: cached + added
 *   cu_tokens    [batch + 1] int32: the rows of each sequence's new tokens
 *   positions    [max_tokens] int32: position of each row's token in its sequence
 *   slots        [max_tokens] int64: page * page_size + place in the page; rows behind the last
 *                sequence get position 0 and slot -1, so that a padded step writes nothing for them
 * seq_lens may be cached itself, and free_count_out free_count; other buffers must not overlap.
 * A sequence that would be longer than the block table (GPTQ_DEV_SEQ_LEN), or one from which on the list
 * has too few pages (GPTQ_DEV_NO_PAGE), keeps its length and pages; its rows stay, with slots -1: gptq_rotary
 * appends nothing for them, and what gptq_chunk_attention, which counts positions back from seq_lens, gives them
 * means nothing and is to be left out; the other sequences' rows are not touched by it.  cached
 * outside [0, table] and added below -cached are cut (GPTQ_DEV_SEQ_LEN); a page given back to a full list
 * is lost (GPTQ_DEV_NO_PAGE); rows past max_tokens are left out and cu_tokens is cut
 * (GPTQ_DEV_TOKEN_ROWS).  batch up to 8192, table_width * page_size, free_capacity and max_tokens up to 2^30;
 * otherwise GPTQ_ERR_SHAPE.
 * All 4-byte aligned, slots 8-byte.  batch == 0 writes cu_tokens[0] and the padding.
 */
int gptq_page_plan(const int32_t* cached, const int32_t* added, int batch, int page_size, int32_t* block_table,
                   int table_width, int32_t* free_pages, int free_capacity, const int32_t* free_count,
                   int32_t* free_count_out, int32_t* seq_lens, int32_t* cu_tokens, int32_t* positions,
                   long long* slots, int max_tokens, void* stream);

/*
 * gptq_rms_norm -- s = residual + x (x alone without a residual), residual_out = s,
 * out = s * weight / sqrt(mean(s^2) + eps), row by row; sums are fp32, each output is rounded once from
 * the unrounded s.
 *   x            [rows, hidden] of dtype (GPTQ_F16, GPTQ_BF16, GPTQ_F32), rows x_stride elements apart
 *   residual     nullable [rows, hidden] of residual_dtype; residual_out the same (both or neither; the
 *                same buffer with the same stride adds in place), rows residual_stride and
 *                residual_out_stride elements apart
 *   weight       nullable [hidden] of weight_dtype: ones where absent
 *   out          [rows, hidden] of out_dtype, rows out_stride elements apart (may be x, with its type
 *                and stride)
 * hidden up to 2^20.  Pointers aligned to their elements; where the rows of x, out and the residuals all start
 * on 16 bytes, or all as many elements behind such a place, they are read and written 16 bytes at a time, otherwise
 * one element at a time.  Buffers other than those named must not overlap.  rows == 0 is a no-op.
 */
int gptq_rms_norm(const void* x, int rows, int hidden, long long x_stride, int dtype, const void* residual,
                  long long residual_stride, int residual_dtype, void* residual_out,
                  long long residual_out_stride, const void* weight, int weight_dtype, float eps, void* out,
                  long long out_stride, int out_dtype, void* stream);

/*
 * gptq_rotary_table -- host: the frequencies of a rotary embedding of rot_dim dimensions, as gptq_rotary reads
 * them: turns[i] = f_i / (2 pi) * 2^64 for i < rot_dim / 2, with f_i = theta^(-2 i / rot_dim) and
 *   GPTQ_ROTARY_NONE    f_i
 *   GPTQ_ROTARY_LINEAR  f_i / factor
 *   GPTQ_ROTARY_BASE    theta * factor^(rot_dim / (rot_dim - 2)) in the place of theta
 *   GPTQ_ROTARY_RAMP    f_i where the pair turns `high` times and more over `original` positions, f_i / factor
 *                       where it turns `low` times and fewer, and between them a mixture, linear in i
 *                       between the two i (rounded outwards); *amplitude = 0.1 ln(factor) + 1
 *   GPTQ_ROTARY_BANDS   the same limits, the mixture linear in the turns; amplitude 1
 * rot_dim: even, 2 to 65536; theta > 1; factor >= 1, for RAMP and BANDS also original > 0 and 0 < low < high;
 * otherwise GPTQ_ERR_SHAPE (rot_dim) or GPTQ_ERR_ARG.
 */
#define GPTQ_ROTARY_NONE 0
#define GPTQ_ROTARY_LINEAR 1
#define GPTQ_ROTARY_BASE 2
#define GPTQ_ROTARY_RAMP 3
#define GPTQ_ROTARY_BANDS 4
int gptq_rotary_table(int rot_dim, double theta, int scaling, double factor, double original, double low,
                      double high, unsigned long long* turns, double* amplitude);

/*
 * gptq_rotary -- rotary embedding of the rows' queries and keys, and the append of keys and values to the
 * paged cache: each pair (a, b) of the first rot_dim dimensions of a head becomes
 *   amplitude * (a cos t - b sin t, a sin t + b cos t),  t = positions[row] * f_i,
 * pair i being dimensions (i, i + rot_dim / 2), or (2 i, 2 i + 1) with interleaved = 1; the others are
 * copied.  t is taken modulo a turn in whole numbers of 2^-64, exact for every position; products are
 * fp32, each output is rounded once.
 *   q, k, v      [tokens, heads or kv_heads, head_dim] of dtype (GPTQ_F16, GPTQ_BF16), heads of a token
 *                contiguous, tokens strides[0..2] elements apart
 *   q_out        [tokens, heads, head_dim], strides[3] apart; may be q with its stride
 *   k_out        nullable, [tokens, kv_heads, head_dim], strides[4] apart; may be k with its stride
 *   k/v_cache    nullable (both or neither, with v and slots): [pages, page_size, kv_heads, head_dim] in
 *                any order of the first three, strides[5..10] = k page, k slot, k head, v page, v slot,
 *                v head; row t's rotated key and its value go to slot slots[t] (int64: page * page_size +
 *                place), nowhere where that is negative; no two rows may have the same slot.  A cache whose
 *                rows overlap (a stride below head_dim) is refused with GPTQ_ERR_SHAPE
 *   positions    [tokens] int32          turns [rot_dim / 2], from gptq_rotary_table
 *   strides      HOST array of 11, in elements, multiples of 8 (anything where the dimension is one, or
 *                the tensor absent)
 * At least one of k_out and the caches is given.  16-bit data 16-byte aligned, slots and turns 8, positions
 * 4.  head_dim: a multiple of 8 up to 256; rot_dim: even, up to head_dim.  tokens == 0 is a no-op.
 */
int gptq_rotary(const void* q, const void* k, const void* v, int tokens, int heads, int kv_heads, int head_dim,
                int rot_dim, int interleaved, int dtype, const long long* strides, const int32_t* positions,
                const unsigned long long* turns, float amplitude, void* q_out, void* k_out, void* k_cache,
                void* v_cache, int pages, int page_size, const long long* slots, void* stream);

/*
 * gptq_chunk_attention -- causal attention of each sequence's new tokens over its cached keys and values,
 * their own among them (gptq_rotary has appended them):
 *   out[r, h] = sum_j p_j v_j,  p = softmax_j(scale * q[r, h] . k_j),
 * for row r = cu_tokens[b] + i, i < m = cu_tokens[b + 1] - cu_tokens[b], at position t = seq_lens[b] - m + i, over
 * the keys j in [max(0, t - window + 1), t] (window 0: [0, t]), k and v of head h / (heads / kv_heads).  Key j
 * is slot j % page_size of page block_table[b, j / page_size].  Sums, maxima and accumulators are
 * fp32, the probabilities enter the product with v in dtype, out is rounded once: its error is some 1.4 times that
 * of the one rounding (gptq_paged_attention, for steps of one token a sequence, carries the probabilities in two
 * parts and has the one rounding's).  Values of up to 2^89 in magnitude cannot overflow the sums.  A row whose position
 * is negative (seq_lens[b] < m) gives zeros.  Rows outside every sequence are left as they were; a row that
 * cu_tokens gives to two sequences (GPTQ_DEV_TOKEN_ROWS) gets the result of either.  What a row does
 * not see is not used for it, whatever it holds: cache slots, block-table entries past a sequence's
 * length, infinite or NaN values of later tokens.  An infinite or NaN value that a row sees reaches it, however
 * small its probability.
 *   q            [tokens, heads, head_dim]: heads of a token contiguous, tokens strides[0] apart
 *   k/v_cache    [pages, page_size, kv_heads, head_dim] in any order of the first three
 *   strides      HOST array of 7 strides in elements, multiples of 8 (anything where the dimension is
 *                one): q token, k page, k slot, k head, v page, v slot, v head
 *   block_table  [batch, table_width] int32, seq_lens [batch], cu_tokens [batch + 1] int32
 *   out          [tokens, heads, head_dim] contiguous
 *   lse          nullable [tokens, heads] fp32: log sum_j exp(scale * q . k_j), -inf without a key
 * Everything 16-bit is of `dtype` (GPTQ_F16, GPTQ_BF16) and 16-byte aligned.  head_dim: a multiple of 8 up to
 * 256; heads a multiple of kv_heads, up to 2^16; a cache spans at most 2^35 elements; tokens * heads and
 * batch * heads at most 2^30 (GPTQ_ERR_SHAPE).  workspace: gptq_chunk_attention_workspace_size() bytes, 16-byte
 * aligned, holding anything.  batch == 0 and tokens == 0 are no-ops.
 */
size_t gptq_chunk_attention_workspace_size(int heads, int kv_heads, int head_dim);
int gptq_chunk_attention(const void* q, int tokens, int heads, int dtype, const void* k_cache, const void* v_cache,
                         int pages, int page_size, int kv_heads, int head_dim, const long long* strides,
                         const int32_t* block_table, int table_width, const int32_t* seq_lens,
                         const int32_t* cu_tokens, int batch, float scale, int window, void* out, float* lse,
                         void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GPTQ_PROMPT_H */
