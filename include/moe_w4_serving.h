/*
 * moe_w4_serving.h -- C ABI of the operators around the sparse-MoE layer in a
 * decode step: the paged key-value cache (append), the attention of one new
 * token per sequence over it (attend), dropping cached tokens by accumulated
 * attention weight (evict), and the log probabilities of given tokens with
 * entropy and the top alternatives (logprobs).  Part of libmoe_w4.so; the
 * conventions of moe_w4.h hold here too: device pointers, caller-owned buffers,
 * no allocation and no synchronisation, one stream per call, 0 or a negative
 * MOE_W4_ERR_* code, nothing enqueued on an argument error, deterministic
 * results (identical inputs give identical bytes), graph-capturable calls.
 *
 * Workspace.  Every call takes a workspace, 256-byte aligned, that is cleared
 * once, as a whole, with moe_w4_workspace_init.  Its first MOE_W4_CTRL_BYTES are
 * the control header of moe_w4.h: the int32 at moe_w4_status_offset() is the
 * sticky device status.
 *   MOE_W4_STATUS_BAD_INDEX: a sequence, slot, page, length or token index read
 *     from device memory was out of range; what it would have touched is left
 *     out, nothing out of range is accessed.
 *   MOE_W4_STATUS_WAIT_TIMEOUT: in moe_w4_attend_decode a wait for another CTA's
 *     part of a sequence ran out (2 s), as when the lengths change while it
 *     runs; its output is not valid.  Clear the workspace before its next use.
 * The attention and the eviction keep counters behind the header that are zero
 * between calls.  A workspace serves one stream at a time; the operators of this
 * header may share one, but not with a call of moe_w4.h.
 */
#ifndef MOE_W4_SERVING_H
#define MOE_W4_SERVING_H

#include "moe_w4.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { MOE_W4_TYPE_BF16 = 0, MOE_W4_TYPE_FP16 = 1, MOE_W4_TYPE_FP32 = 2 };

#define MOE_W4_CTRL_BYTES 256
#define MOE_W4_MAX_SEQS 4096        /* sequences of one cache               */
#define MOE_W4_MAX_TOP 32           /* alternatives of moe_w4_token_logprobs */
#define MOE_W4_MAX_VOCAB (1 << 20)  /* logits of a row                       */

/* A paged key-value cache.  The keys of page p, head h, slot s (0 <= s <
 * page_size) start at k + p * page_stride + h * head_stride + s * slot_stride
 * elements and are head_dim contiguous elements; v alike.  Both orders,
 * [page][head][slot][dim] and [page][slot][head][dim], are strides of this.
 * Token t of sequence b lies in page block_table[b * table_stride + t /
 * page_size], slot t % page_size; entries past the sequence's last page are
 * not read.
 * Supported: dtype bf16 or fp16; head_dim 64, 128 or 256; 1 <= n_kv_heads <=
 * 1024; page_size >= 1; 1 <= n_seqs <= MOE_W4_MAX_SEQS (0: every call returns
 * at once); strides non-negative multiples of 8 below 2^35, k and v 16-byte aligned;
 * pages_per_seq * page_size <= 2^30.
 * Sequences may share pages that calls only read (a common prefix); a page
 * that append or evict writes must belong to one sequence. */
typedef struct {
    int dtype;                        /* MOE_W4_TYPE_BF16 or MOE_W4_TYPE_FP16     */
    int n_kv_heads, head_dim, page_size, num_pages;
    int64_t page_stride, head_stride, slot_stride;   /* elements                 */
    void *k, *v;
    int n_seqs, pages_per_seq;
    int64_t table_stride;             /* int32 entries between sequences         */
    const int32_t* block_table;
    const int32_t* seq_lens;          /* [n_seqs] tokens held, the new one included */
} moe_w4_kv_cache;

/* What is kept beside the cache for eviction, per sequence, kv head and slot
 * (entry b * seq_stride + h * head_stride + token): the attention weight that
 * the token has drawn so far, and its position in the sequence as it was fed.
 * After an eviction the heads of a sequence hold different tokens, in no
 * particular order; `pos` says which (NULL where nothing is evicted). */
typedef struct {
    float* weight;
    int32_t* pos;
    int64_t seq_stride, head_stride;
    int slots;                        /* entries per sequence and head           */
} moe_w4_kv_track;

/* Writes n tokens' keys and values into the cache.
 *   k, v   [n][n_kv_heads][head_dim] of the cache's type; token i starts at
 *          i * k_stride (v_stride) elements, multiples of 8, so both may be
 *          views of one projection's output; 16-byte aligned
 *   seq    int32 [n] sequence of each token, or NULL: token i belongs to
 *          sequence i (then n == n_seqs)
 *   slot   int32 [n] token index within the sequence, or NULL: its last one,
 *          seq_lens[seq] - 1 (a sequence of length 0 then gets nothing)
 *   track  NULL, or the arrays to start for the new tokens in every head:
 *          weight 0, pos pos[i] (pos NULL: the token index)
 * Two tokens of one call must not share a place.  seq_lens is read only where
 * slot is NULL, and never changed. */
int moe_w4_kv_append(const moe_w4_kv_cache* c, const moe_w4_kv_track* track, int n, const void* k, int64_t k_stride,
                     const void* v, int64_t v_stride, const int32_t* seq, const int32_t* slot, const int32_t* pos,
                     void* workspace, size_t ws_bytes, cudaStream_t stream);

/* Attention of one new token per sequence over its seq_lens[b] cached tokens:
 *   s_t = scale * q . k_t,  p = softmax(s),  out = sum_t p_t v_t,
 *   lse = log sum_t exp(s_t)
 * CTAs that share a sequence wait for one another, with a limit, so the launch is
 * cooperative; moe_w4_test_skip_publish on its workspace makes those waits run out.
 * Query heads h * group .. h * group + group - 1 (group = n_q_heads /
 * n_kv_heads, at most 128) share kv head h.  Scores, maxima and sums are fp32;
 * probabilities are two 16-bit terms of the cache's type in the product with v:
 * off by at most 2^-17 (bf16), or 2^-21 and 2^-38 of the row's largest (fp16);
 * out is rounded once.
 *   q, out [n_seqs][n_q_heads][head_dim] of the cache's type, sequences
 *          q_stride (out_stride) elements apart, multiples of 8; 16-byte
 *          aligned
 *   lse    fp32 [n_seqs][n_q_heads], or NULL
 *   max_len  an upper bound of the lengths, <= pages_per_seq * page_size (a
 *          longer length sets MOE_W4_STATUS_BAD_INDEX and is cut)
 *   track, weight_out  both NULL, or: weight_out[t] = track->weight[t] + the sum
 *          of p_t over the kv head's query heads, for t < seq_lens[b] (fp32, the
 *          strides of track; may be track->weight).  track->pos is not used.
 * A sequence of length 0, or whose scores are all -inf, gives zeros and lse
 * -inf.  Tokens on pages outside the cache take no part, as if they scored -inf
 * (and set MOE_W4_STATUS_BAD_INDEX).  Cache slots past the length are not read as numbers: they may hold
 * anything, NaN included.  MOE_W4_ERR_UNSUPPORTED where n_seqs * n_kv_heads *
 * (tiles of 64 tokens up to max_len + 1) * (blocks of 24 query heads of a kv
 * head, 16 at head_dim 256) passes 2^31. */
size_t moe_w4_attend_workspace_size(const moe_w4_kv_cache* c, int n_q_heads, int max_len, int with_track);
int moe_w4_attend_decode(const moe_w4_kv_cache* c, int n_q_heads, const void* q, int64_t q_stride, float scale,
                         int max_len, void* out, int64_t out_stride, float* lse, const moe_w4_kv_track* track,
                         float* weight_out, void* workspace, size_t ws_bytes, cudaStream_t stream);

/* Cuts every sequence of more than `budget` tokens to `budget`, head by head.
 * Kept are, in this order of preference: tokens with pos < sink or pos >=
 * seen[b] - recent; then the larger weight (NaN below every number, -0 equal
 * to 0); of equals the lower token index.  Tokens kept in place stay there;
 * the kept tokens at indexes >= budget move, in ascending order, into the
 * places below budget that were dropped, in ascending order (a move from or to a
 * page outside the cache is left out: the place keeps its token, and
 * MOE_W4_STATUS_BAD_INDEX is set): keys and values inside the cache, and
 *   lens_out[b]       = min(seq_lens[b], budget)
 *   weight_out, pos_out (strides of track) the weights and positions of the
 *                     tokens now at 0 .. lens_out[b] - 1
 * The outputs may be the inputs (lens_out == seq_lens, weight_out ==
 * track->weight, pos_out == track->pos) or separate arrays.  1 <= budget,
 * sink, recent >= 0, sink + recent <= budget; max_len as above, <=
 * track->slots; n_seqs * n_kv_heads <= 65535. */
size_t moe_w4_evict_workspace_size(const moe_w4_kv_cache* c, int budget, int max_len);
int moe_w4_kv_evict(const moe_w4_kv_cache* c, const moe_w4_kv_track* track, const int32_t* seen, int budget, int sink,
                    int recent, int max_len, int32_t* lens_out, float* weight_out, int32_t* pos_out, void* workspace,
                    size_t ws_bytes, cudaStream_t stream);

/* Log probabilities of given tokens under softmax(logits), natural logarithms:
 *   logits  [n][vocab] fp32, bf16 or fp16, rows row_stride (>= vocab) elements
 *           apart; any alignment of the element
 *   targets int32 [n] and logprob fp32 [n], or both NULL: logprob[i] =
 *           logits[i][targets[i]] - lse_i.  A target of -1 asks for nothing
 *           (logprob 0); others outside 0..vocab-1 give NaN and set
 *           MOE_W4_STATUS_BAD_INDEX
 *   entropy fp32 [n] or NULL: -sum p log p (tokens of probability 0 add 0)
 *   top     0..min(MOE_W4_MAX_TOP, vocab) alternatives per row into top_index
 *           int32 [n][top] and top_logprob fp32 [n][top], best first, of equal
 *           logits the lower index first (-0 equal to 0, NaN after every number)
 * Sums are fp32.  -inf logits are masked tokens: probability 0.  A row with a
 * NaN or +inf logit, or with nothing but -inf, has no softmax: logprob, entropy
 * and top_logprob are NaN there, top_index stands. */
int moe_w4_token_logprobs(int dtype, int n, int vocab, const void* logits, int64_t row_stride, const int32_t* targets,
                          int top, float* logprob, float* entropy, int32_t* top_index, float* top_logprob,
                          void* workspace, size_t ws_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_W4_SERVING_H */
