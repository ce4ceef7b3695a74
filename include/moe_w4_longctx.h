/*
 * moe_w4_longctx.h -- C ABI of the operators for long contexts in a decode step:
 * norms of queries and keys with the position rotation, a paged key-value cache
 * of 8-bit codes (append, read back, attention of one new token per sequence),
 * and that attention with a sliding window.  Part of libmoe_w4.so; the
 * conventions of moe_w4.h and moe_w4_serving.h hold: device pointers,
 * caller-owned buffers, no allocation and no synchronisation, one stream per
 * call, 0 or a negative MOE_W4_ERR_* code, nothing enqueued on an argument
 * error, deterministic results, graph-capturable calls, the workspace of
 * moe_w4_serving.h with its sticky status.  Calls of many arguments
 * take them as a struct, which is read during the call only.
 */
#ifndef MOE_W4_LONGCTX_H
#define MOE_W4_LONGCTX_H

#include "moe_w4_serving.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The rotation: pair i (0 <= i < pairs) of a head turns by the angle
 * 2 pi * frac(positions[axis[i]] * turns[i] / 2^64), that is turns[i] holds the
 * pair's frequency in turns per position, mod 1, as a 64-bit fraction; exact for
 * positions of any size.  The first 2 * pairs dimensions of a head turn: pair i is
 * dimensions i and pairs + i, or with `interleaved` 2 i and 2 i + 1.  Cosine and
 * sine are multiplied by `scale`. */
typedef struct {
    const uint64_t* turns;            /* [pairs]                                 */
    const int32_t* axis;              /* [pairs] 0..axes-1 (others count as the nearest), or NULL: 0 */
    int pairs;                        /* a multiple of 8, 2 * pairs <= head_dim  */
    int axes;                         /* 1..8 rows of positions                  */
    int interleaved;
    float scale;
} moe_w4_rope;

/* Per head of n tokens, queries and keys alike:
 *   y = x * rsqrt(mean(x^2) + eps) * w      (w + 1 with unit_offset)
 * and then the rotation of y; all in fp32 (cosines and sines are off by at most 2^-22),
 * rounded once.
 *   dtype     bf16 or fp16, of q, k, outputs and weights; head_dim 64, 128 or 256
 *   q, q_out  [n][n_q_heads][head_dim], tokens q_stride (qo_stride) elements
 *             apart, multiples of 8; 16-byte aligned; k alike, n_k_heads may be 0
 *   q_weight, k_weight  [head_dim], 16-byte aligned, or NULL: no norm
 *   rope      or NULL: no rotation
 *   positions int32 [rope->axes][n], axes pos_stride apart
 * q_out may be q and k_out k (in place, equal strides); they must not overlap
 * otherwise.  n * (n_q_heads + n_k_heads) < 2^30. */
typedef struct {
    int dtype, n, head_dim, n_q_heads, n_k_heads, unit_offset;
    float eps;
    const void* q;
    void* q_out;
    const void* k;
    void* k_out;
    int64_t q_stride, qo_stride, k_stride, ko_stride;
    const void *q_weight, *k_weight;
    const moe_w4_rope* rope;
    const int32_t* positions;
    int64_t pos_stride;
} moe_w4_qk_call;
int moe_w4_qk_norm_rope(const moe_w4_qk_call* a, cudaStream_t stream);

/* A cache of 8-bit codes: value = code * scale, codes E4M3 (1-4-3 bits, largest
 * 448, NaN, no infinity), an fp32 scale for each block of `block` tokens of a
 * head, keys and values apart.  `c` describes it as in moe_w4_serving.h, but c.k
 * and c.v hold one-byte codes (strides multiples of 16) and c.dtype is the type of
 * the tokens that are written and read and of queries and outputs.
 * The scale of page p, head h, slot s is k_scale[p * scale_page_stride + h *
 * scale_head_stride + s / block].  block: a power of two, 1..128, that divides
 * page_size. */
typedef struct {
    moe_w4_kv_cache c;
    float *k_scale, *v_scale;
    int64_t scale_page_stride, scale_head_stride;
    int block;
} moe_w4_kv8_cache;

/* n tokens of a cache, in memory [n][n_kv_heads][head_dim] of its type: token i at
 * i * k_stride (v_stride) elements of k (v), multiples of 8, 16-byte aligned; seq and
 * slot as in moe_w4_kv_append. */
typedef struct {
    int n;
    void *k, *v;
    int64_t k_stride, v_stride;
    const int32_t *seq, *slot;
    void* workspace;
    size_t ws_bytes;
} moe_w4_kv_tokens;

/* Writes tokens.  The tokens of one block have to be consecutive rows with
 * consecutive indexes (unlike rows of moe_w4_kv_append, which may have any order), and
 * no token may be named twice: several rows of a block apart from one another each set
 * its scale, and which one stays is not defined.  The debug build refuses such a call on the
 * device: MOE_W4_STATUS_BAD_INDEX, nothing is written.
 * A block's scale is the smallest power of two, 2^-100 to 2^119, that brings the
 * largest finite magnitude of its tokens to 448 or below; codes are the nearest
 * (ties to even), infinities become +-448, NaN stays NaN.  Powers of two lose no
 * bits: codes are floating point, and those of a block already begun can follow a
 * larger scale exactly, down to their smallest steps.  A call that writes the
 * first token of a block begins it: other tokens in it that the call does not
 * write have no meaning afterwards.  Otherwise the block's scale only grows, and
 * the codes of its other tokens are brought to it.  (A scale set by the caller that
 * is no power of two is rounded up to one, one outside that range brought into it,
 * and one that is not positive and finite counts as 2^-100.) */
int moe_w4_kv8_append(const moe_w4_kv8_cache* c, const moe_w4_kv_tokens* t, cudaStream_t stream);

/* Reads tokens back, rounded once from code * scale; they may be named in any order
 * and more than once.  A token that the cache does not have is zeros (and sets
 * MOE_W4_STATUS_BAD_INDEX, unless it is the last one of a sequence of length 0);
 * a cache of 0 sequences has none.
 * moe_w4_kv_read does the same for a cache of 16-bit values. */
int moe_w4_kv8_read(const moe_w4_kv8_cache* c, const moe_w4_kv_tokens* t, cudaStream_t stream);
int moe_w4_kv_read(const moe_w4_kv_cache* c, const moe_w4_kv_tokens* t, cudaStream_t stream);

/* moe_w4_attend_decode over a cache of 8-bit codes, and over one of 16-bit values
 * with a window (no weights are added up).  window 0: every token is seen (sink is
 * 0 then); otherwise token t of a sequence of n is seen where t < sink or
 * t >= n - window.  Tokens that are not seen are not read, their pages may be
 * anything.  Scales of tokens that are seen are finite and not negative.  Sums are fp32:
 * of bf16 codes, values are below 2^80 in magnitude, and so is `scale` times a head's
 * largest query times a key's scale.
 * Over codes, queries enter the product as fp16, scaled by a power of two per head so that
 * the largest is 2^14 to 2^15: exact, but for those below 2^-29 of the largest,
 * which are off by at most 2^-39 of it.  Probabilities times the values' scales are two fp16
 * terms, off by at most 2^-21, or 2^-49 of the row's largest such product (2^-157 where scales
 * lie below 2^-100).  Probabilities below 2^-125 of the row's largest count as 0.
 * The workspace of moe_w4_attend_window is moe_w4_attend_workspace_size(..., 0)
 * bytes.  Members as the arguments of
 * moe_w4_attend_decode. */
typedef struct {
    int n_q_heads, max_len, window, sink;
    float scale;
    const void* q;
    void* out;
    int64_t q_stride, out_stride;
    float* lse;
    void* workspace;
    size_t ws_bytes;
} moe_w4_attend_call;
size_t moe_w4_kv8_attend_workspace_size(const moe_w4_kv8_cache* c, int n_q_heads, int max_len);
int moe_w4_kv8_attend(const moe_w4_kv8_cache* c, const moe_w4_attend_call* a, cudaStream_t stream);
int moe_w4_attend_window(const moe_w4_kv_cache* c, const moe_w4_attend_call* a, cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_W4_LONGCTX_H */
