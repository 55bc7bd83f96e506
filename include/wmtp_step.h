/*
 * wmtp_step.h -- the work of a speculative decode step around its attention:
 * encoded queries and keys in the paged cache, page tables and slot maps on
 * the device, log probabilities, and which drafted tokens are accepted.
 *
 * The pages measure the attention alone and take these for granted ("Windowed-
 * MTP ...", arxivlens view, Abstract: the target verifies gamma+1 tokens and
 * accepts some of them).  With the calls below, the attention and the ring
 * calls of wmtp.h, a whole step stays on the GPU: lengths, page tables,
 * accepted counts and the ring's truncate_to are device arrays throughout, so
 * the step can be captured in one CUDA graph.
 *
 * The conventions of wmtp.h hold for every call here: device pointers owned by
 * the caller, nothing allocated, asynchronous on `stream` as a programmatic
 * dependent of the work before, host-detectable errors as a negative status
 * before anything is launched, device-detected ones as WMTP_DEV_* bits.  An
 * output overlaps no other buffer of its call, unless it is said below.
 * "Row" below is one distribution: `vocab` logits next to one another.  Calls of
 * the same sizes and alignment give the same bits.  A row's sums are split over more
 * CTAs where there are few rows, so its last bits depend on how many the call has.
 */
#ifndef WMTP_STEP_H_
#define WMTP_STEP_H_

#include <stddef.h>
#include <stdint.h>

#include "wmtp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of inputs that may have more than one. */
typedef enum { WMTP_BF16 = 0, WMTP_FP16 = 1, WMTP_FP32 = 2 } wmtp_dtype;

/* Further bits the kernels OR into *status_word. */
#define WMTP_DEV_POOL 0x40      /* free pages or slot-map rows ran out, or an
                                   inconsistent free count */
#define WMTP_DEV_LOGITS 0x80    /* a row that defines no distribution: NaN or +inf
                                   among its logits, or a bad temperature */
#define WMTP_DEV_TOKEN_OOB 0x100 /* a token id outside [0, vocab) */

/*
 * Rotary positions.  Pair i of a head (rotary_dim / 2 pairs) at position t is
 * turned by t * turn[i] / 2^64 full turns: turn[i] = f_i / (2 pi) * 2^64, f_i
 * the pair's angle per position in radians.  The product is taken modulo 2^64,
 * that is modulo whole turns, so far positions lose nothing.
 * Pair i holds elements i and i + rotary_dim/2 of the head, or 2i and 2i+1 if
 * interleaved.  Elements from rotary_dim on are not rotated.
 */
typedef struct {
  const uint64_t* turn; /* [rotary_dim / 2] device */
  int32_t rotary_dim;   /* even, 0 <= rotary_dim <= head_dim */
  int32_t interleaved;
  float factor;         /* cos and sin are multiplied by this (1: a rotation) */
} wmtp_rope;

/*
 * wmtp_qk_norm_rope -- encode a step's queries and keys: the RMS norm of each
 * head, the position rotation, and the write of K and V into the paged cache,
 * in one pass.  The attention calls take K "already encoded"; this encodes it.
 *
 * For token t and each query (and key) head row x of head_dim values:
 *   y = x * rsqrt(mean(x^2) + eps) * (weight + weight_offset)    (weight given)
 *   y = x                                                      (weight NULL)
 *   (a, b) -> factor * (a cos - b sin, b cos + a sin)   for each rotated pair
 * in fp32, rounded to bf16 once.  V is copied (rounded to bf16).
 *   tokens     : rows of q, k, v, positions, slots; token t is a row of any
 *                sequence (a verify block [batch][num_q] is batch * num_q rows)
 *   in_dtype   : of q, k, v: WMTP_BF16 or WMTP_FP32
 *   q, k, v    : [tokens][heads][head_dim] views, elements of a head next to
 *                one another, token and head strides in elements (cut from one
 *                packed projection, say).  16-byte aligned, strides too.
 *                q NULL: no queries (q_out NULL).  k NULL: no keys.
 *   positions  : [tokens] int32 rotary positions; a negative one marks a padding
 *                row, which is skipped: its rows of q_out and k_out and the
 *                cache stay as they were
 *   slots      : [tokens] int64 cache slots, page * page_size + row, or NULL to
 *                write no cache; -1 writes nothing for that token, any other
 *                slot outside the pool too, and sets WMTP_DEV_PAGE_OOB.  No
 *                two tokens have one slot (what it holds would be any mixture).
 *   kv         : with slots: k_pool, v_pool and num_pages are used
 *   v          : with slots, else NULL
 *   q_weight, k_weight : [head_dim] of weight_dtype (WMTP_BF16 or WMTP_FP32), or NULL
 *   q_out      : [tokens][num_heads_q][head_dim] bf16; may be q itself if q is
 *                contiguous bf16.  It is the attention calls' q.
 *   k_out      : [tokens][num_heads_kv][head_dim] bf16 or NULL: k_new of
 *                wmtp_ring_append and wmtp_verify_attn_append.  May be k itself
 *                if k is contiguous bf16.
 * Tokens are encoded in any order.  A q_out or k_out that lies over rows of q, k
 * or v in any other way, over the other one or over a pool is refused, and so are
 * pools that overlap.  q, k and v may be rows of the pools that no token's slot is.
 *   rope       : NULL: no rotation
 * head_dim is a multiple of 8 in 8..256.
 */
wmtp_status wmtp_qk_norm_rope(const wmtp_params* params, const wmtp_rope* rope, int32_t tokens, int32_t in_dtype,
                              const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k,
                              int64_t k_token_stride, int64_t k_head_stride, const void* v, int64_t v_token_stride,
                              int64_t v_head_stride, const int32_t* positions, const int64_t* slots,
                              const wmtp_paged_kv* kv, const void* q_weight, const void* k_weight,
                              int32_t weight_dtype, float weight_offset, float eps, void* q_out, void* k_out,
                              int32_t* status_word, void* stream);

/*
 * wmtp_pages_resize -- bring every sequence's pages to a new length, and map
 * its new tokens to cache slots.  The device counterpart of wmtp_pool_*: the
 * same free list over the page indices of one pool, kept in device memory.
 *
 * A sequence of n tokens holds ceil(n / page_size) pages, the first entries of
 * its page_table row.  Each sequence whose new_len is valid goes from kv_len[b]
 * to new_len[b]:
 *   1. pages above the new length return to the free list; their entries in
 *      page_table become -1 (new_len 0 ends a request).  An entry outside
 *      [0, num_pages) sets WMTP_DEV_PAGE_OOB and is returned as it is;
 *   2. missing pages are taken from the free list (those returned in step 1
 *      among them);
 *   3. kv_len[b] = new_len[b].
 * The free list is a stack.  Pages are taken for the lowest sequence and page
 * first and returned highest first, so taking back what was just grown leaves
 * the stack as it was.  Growing sequences are served in order while free pages
 * and rows of the slot map last: the first one that does not fit and every
 * growing one behind it keep their length and pages, and WMTP_DEV_POOL is set.
 *   page_table : [batch][max_pages] int32, in and out
 *   kv_len     : [batch] int32, in and out
 *   new_len    : [batch] int32; outside [0, max_pages * page_size]: the sequence
 *                is left as it was, WMTP_DEV_LEN_OOB
 *   free_pages : [num_pages] int32 stack, entries below *free_count are free;
 *   free_count : [1] int32.  A count that is negative or would pass num_pages
 *                sets WMTP_DEV_POOL; nothing is changed (the slot map is empty).
 *   The slot map of the tokens added (max_tokens 0: none, the three NULL):
 *   cu_tokens  : [batch + 1] int32, tokens added before sequence b
 *   positions  : [max_tokens] int32, slots : [max_tokens] int64: token
 *                cu_tokens[b] + i is at position (old kv_len[b]) + i, slot
 *                page * page_size + row; rows behind the last token are -1.
 *                Both are what wmtp_qk_norm_rope takes.  A token on a page
 *                outside [0, num_pages) has slot -1, WMTP_DEV_PAGE_OOB.
 *   workspace  : 256-byte aligned device scratch.  Call with workspace and
 *                free_pages NULL to get the size in *workspace_bytes; where it
 *                is 0 workspace may be NULL.
 * A page belongs to one sequence: a page that two rows of the table share would
 * be returned by each.  The buffers do not overlap.
 * page_size as wmtp.h; max_pages * page_size <= 2^30.
 */
wmtp_status wmtp_pages_resize(const wmtp_params* params, int32_t batch, int32_t* page_table, int32_t max_pages,
                              int32_t* kv_len, const int32_t* new_len, int32_t* free_pages, int32_t* free_count,
                              int32_t num_pages, int32_t* cu_tokens, int32_t* positions, int64_t* slots,
                              int32_t max_tokens, void* workspace, size_t* workspace_bytes, int32_t* status_word,
                              void* stream);

/*
 * wmtp_token_logprobs -- log probabilities of given tokens, with the entropy
 * and the most likely alternatives of each row.
 *
 * With y = (x - max x) / T and S = sum exp(y):
 *   logprob(token) = y[token] - ln S,   lse = max x / T + ln S,
 *   entropy = ln S - sum exp(y) y / S,
 *   top: the top_k largest logits, larger first, equal ones by lower id.
 *   logits      : [rows][vocab] of dtype, `row_stride` elements between rows;
 *                 what lies behind `vocab` is not read into any result
 *   temperature : [rows] fp32, or NULL for 1; finite, above 0, and log2(e) / T
 *                 finite in fp32 too, which it is from 4.25e-39 on
 *   tokens      : [rows][num_tokens] int32.  -1: no token (logprob -inf); any
 *                 other id outside [0, vocab) too, and WMTP_DEV_TOKEN_OOB
 *   logprobs_out: [rows][num_tokens]; entropy_out, lse_out: [rows] or NULL
 *   top_logprobs_out, top_ids_out: [rows][top_k], top_k in 0..64; places without
 *                 a token above -inf are (-inf, -1)
 * A logit of -inf is a masked token of probability 0.  A row of them alone has
 * lse = -inf, entropy 0 and no token.  A row with NaN or +inf, or with a bad
 * temperature, is NaN throughout, ids -1, and sets WMTP_DEV_LOGITS.
 * Sums are fp32, of terms that are good to 2^-22.
 */
wmtp_status wmtp_token_logprobs(int32_t rows, int32_t vocab, int32_t dtype, const void* logits, int64_t row_stride,
                                const float* temperature, const int32_t* tokens, int32_t num_tokens, int32_t top_k,
                                float* logprobs_out, float* entropy_out, float* lse_out, float* top_logprobs_out,
                                int32_t* top_ids_out, int32_t* status_word, void* stream);

/*
 * wmtp_accept_draft -- which of a step's drafted tokens the target accepts,
 * and the token that follows them.
 *
 * p_i is the target's distribution softmax(target[b][i] / T) that drafted
 * token d_i is checked against, q_i the draft's own, softmax(draft[b][i] / T),
 * or all of its weight on d_i if draft is NULL.  In order of i < num_draft[b]:
 *   T > 0 : d_i is accepted if u_i * q_i(d_i) < p_i(d_i); the first rejected
 *           one is replaced by a draw from max(p_i - q_i, 0) / its sum (from
 *           p_i where that is 0 everywhere), and behind num_draft[b] accepted
 *           ones follows a draw from p_{num_draft[b]}: the emitted tokens are
 *           distributed as the target's own.
 *   T == 0: d_i is accepted if it is the lowest id with the largest logit, and
 *           the token that follows is that id of its row.
 * A draw is the lowest id whose cumulated weight is above u * (their sum), with
 * u = uniforms[b][num_q - 1].
 *   target    : [batch][num_q][vocab] of dtype, strides in elements
 *   draft     : [batch][num_q - 1][vocab] of dtype, or NULL
 *   draft_tokens : [batch][num_q - 1] int32 (NULL if num_q is 1); an id outside
 *               [0, vocab) is rejected and sets WMTP_DEV_TOKEN_OOB
 *   uniforms  : [batch][num_q] fp32 in [0, 1)
 *   num_draft : [batch] int32 in [0, num_q - 1], or NULL for num_q - 1 (outside:
 *               WMTP_DEV_LEN_OOB, the sequence emits nothing)
 *   temperature : [batch] fp32, 0 or as for wmtp_token_logprobs, or NULL for 1
 *   tokens_out: [batch][num_q] int32, the emitted tokens, -1 behind them
 *   count_out : [batch] int32, how many: accepted + 1
 *   logprobs_out : [batch][num_q] fp32 or NULL: ln p_i of each emitted token (of
 *               T = 1 for a greedy sequence), 0 behind them
 * Once a row that is needed defines no distribution (NaN, +inf, -inf alone, a
 * bad temperature) the sequence ends there: WMTP_DEV_LOGITS, and count_out is
 * the tokens before it.
 *   workspace : as in wmtp_draft_attn_full (NULL: size query)
 * num_q in 1..32.  Masked tokens (top-k, top-p, a grammar) are -inf logits.
 * p_i(d_i), q_i(d_i), their comparison and the log probabilities are fp32, from
 * sums as in wmtp_token_logprobs: a u_i next to the border, within fp32's rounding
 * of it, may fall on either side.  The draw's weights and sums are 64-bit.
 */
wmtp_status wmtp_accept_draft(int32_t batch, int32_t num_q, int32_t vocab, int32_t dtype, const void* target,
                              int64_t target_batch_stride, int64_t target_row_stride, const void* draft,
                              int64_t draft_batch_stride, int64_t draft_row_stride, const int32_t* draft_tokens,
                              const float* uniforms, const int32_t* num_draft, const float* temperature,
                              int32_t* tokens_out, int32_t* count_out, float* logprobs_out, void* workspace,
                              size_t* workspace_bytes, int32_t* status_word, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* WMTP_STEP_H_ */
