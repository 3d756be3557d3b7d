/*
 * libred_decode.h -- the reductions of a decoding step of drafted tokens:
 * norms of query and key heads with the rotary position rotation, a paged
 * key/value cache that is quantised as it is written, attention of drafted
 * tokens over that cache, and the verification of the drafted tokens against
 * the target's probabilities.
 *
 * The conventions of libred.h hold: device pointers, calls asynchronous on
 * `stream`, argument errors reported as RED_ERR_INVALID_ARG before any HIP
 * call and with nothing enqueued, deterministic results, nothing thrown.
 * Arguments come in structs that the call reads before it returns. Strides
 * count elements of the tensor they belong to; the last dimension (`dim` or
 * the vocabulary) is always contiguous. Every pointer is aligned to its
 * element. Inputs must not overlap outputs, from their first element to their
 * last, unless a call says otherwise.
 *
 * Scratch: the backward pass of the norms, attention (max_len above 32) and the
 * verification keep partials in the stream's scratch buffer (the one of the
 * column reductions): grown on demand, kept until the process exits. While
 * the stream is being captured into a graph a call whose scratch is missing or
 * too small returns RED_ERR_CAPTURE before it touches the stream; an earlier
 * call on the stream provides it, of the same types, kv heads and dim, and of no
 * fewer sequences, tokens, nodes, query heads, drafts and vocabulary.
 */
#ifndef LIBRED_DECODE_H_
#define LIBRED_DECODE_H_

#include "libred.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. RED_E4M3: 8-bit floats with 4 exponent and 3 mantissa bits
 * (largest value 448, no infinity). */
enum { RED_F32 = 0, RED_F16 = 1, RED_BF16 = 2, RED_I8 = 3, RED_E4M3 = 4 };

/* Heads of a batch of tokens: element (t, h, d) lies at
 * data + t * token_stride + h * head_stride + d. Strides of 0 or more. */
typedef struct red_heads {
    void *data;
    int64_t heads;
    int64_t token_stride;
    int64_t head_stride;
} red_heads;

#define RED_HEAD_MAX_DIM 256

/*
 * RMS norm of every head of q and k, its weight, and the rotary rotation of
 * the result's first `rot` elements, in one pass:
 *
 *   y = x * rsqrt(mean(x^2) + eps) * w
 *   (y_a, y_b) -> (y_a cos - y_b sin, y_a sin + y_b cos),  angle pos[t] * freq[i]
 *
 * with i = 0 .. rot/2 - 1 and the pair (a, b) = (i, i + rot/2), or (2i, 2i + 1)
 * where `interleaved` is not 0. Elements from `rot` on are not rotated.
 * type: RED_F32, RED_F16 or RED_BF16 of x, the weights and y; arithmetic in
 * float32, angles in float64, one rounding at the end. 1 <= dim <= 256,
 * rot even, 0 <= rot <= dim. weights: `dim` elements, NULL for ones. freq:
 * rot/2 floats. q.heads or k.heads may be 0. q_out and k_out have q's and k's
 * shape, strides of their own, and may be q and k themselves (same strides):
 * the norm is then done in place. tokens == 0 does nothing.
 */
typedef struct red_qk_norm_rope_args {
    int type;
    int interleaved;
    size_t tokens;
    size_t dim;
    size_t rot;
    float eps;
    red_heads q, k;         /* in */
    red_heads q_out, k_out; /* out */
    const void *q_weight;
    const void *k_weight;
    const int64_t *pos; /* tokens */
    const float *freq;
} red_qk_norm_rope_args;

red_status red_qk_norm_rope(const red_qk_norm_rope_args *a, hipStream_t stream);

/*
 * Its backward pass: from the gradients of the outputs, those of q, k and of
 * both weights (float32, summed over tokens and heads in a fixed order; NULL
 * where not wanted). a->q and a->k are the inputs of the forward pass,
 * a->q_out and a->k_out receive the gradients of q and k, dq and dk hold the
 * gradients of the outputs. tokens == 0 stores zeros in the weight gradients.
 */
red_status red_qk_norm_rope_backward(const red_qk_norm_rope_args *a, const red_heads *dq, const red_heads *dk,
                                     float *dq_weight, float *dk_weight, hipStream_t stream);

/*
 * A paged cache of keys and values. Row (page p, head h, place s) starts at
 * p * page_stride + h * head_stride + s * place_stride in k and in v, and
 * holds `dim` elements. type RED_F16 / RED_BF16: the values themselves, the
 * scales NULL. RED_I8 / RED_E4M3: value = element * scale, one float32 scale
 * a row, at p * scale_page_stride + h * scale_head_stride + s *
 * scale_place_stride in k_scales and v_scales.
 */
typedef struct red_paged_cache {
    void *k;
    void *v;
    float *k_scales;
    float *v_scales;
    int type;
    size_t pages;
    size_t heads;
    size_t places; /* tokens a page holds */
    size_t dim;
    int64_t page_stride, head_stride, place_stride;
    int64_t scale_page_stride, scale_head_stride, scale_place_stride;
} red_paged_cache;

/*
 * Write the keys and values of `tokens` tokens into the cache: token t goes
 * to slot slots[t] = page * places + place. A slot outside [0, pages *
 * places) is skipped (padding). Two tokens of one call must not share a slot.
 * type: RED_F16 or RED_BF16, and the cache's own type where that has 16 bits.
 * 8-bit caches: with top = max|x| of the row, the scale is top / 127 (RED_I8)
 * or top / 448 (RED_E4M3) and an element is x * (127 or 448) / top rounded to
 * nearest, ties to even; a row of zeros has scale 0. A row that holds an
 * infinity or a NaN is stored as zeros with that scale, and reads back as NaN.
 * k and v must have the cache's heads; dim 1 .. 256.
 */
red_status red_cache_write(const red_paged_cache *cache, int type, const red_heads *k, const red_heads *v,
                           const int64_t *slots, size_t tokens, hipStream_t stream);

/*
 * Read tokens back in 16 bits (8-bit caches: element * scale in float32, then
 * rounded to 16 bits). A slot outside the cache reads as zeros. k and v are
 * written.
 */
red_status red_cache_read(const red_paged_cache *cache, int type, const red_heads *k, const red_heads *v,
                          const int64_t *slots, size_t tokens, hipStream_t stream);

#define RED_TREE_MAX_NODES 64

/*
 * Attention of drafted tokens over a paged cache. Sequence b holds lens[b]
 * tokens and then the `nodes` drafted ones, whose keys and values are in the
 * cache too: token t lies at place t % places of page table[b * table_stride
 * + t / places]. Node i sees every token below lens[b], and of the nodes
 * those whose bit is set in tree_mask[b * nodes + i] (bit j: node j; itself
 * among them where it is to be seen), or, where tree_mask is NULL, nodes 0 ..
 * i. Only the first node_count[b] nodes exist (NULL: all).
 *
 *   s = scale * q . k,  out = softmax(s) v,  lse = log sum exp(s)
 *
 * Query head h reads kv head h / (q_heads / cache heads). A row that sees
 * nothing, and every row of a node that does not exist, gets out = 0 and
 * lse = -inf; what lies in the cache behind a mask, infinities and NaN
 * included, does not reach a result. A value row of an 8-bit cache whose scale
 * is no number makes the outputs of the rows that see it NaN, not their lse.
 *
 * type: RED_F16 or RED_BF16 of q and out, and of a 16-bit cache. q and out:
 * (batch, nodes, q_heads, dim) with strides of their own, rows on 16-byte
 * boundaries, the rows of out in that order; lse: batch * nodes * q_heads
 * floats. The cache's dim is a multiple of 16 up to 256, its rows start on
 * 16-byte boundaries, those of one head within 64 GiB of each other; the
 * strides of its scales are below 2^32. nodes <= 64, batch and q_heads <=
 * 65535, max_len <= 2^30, and batch * kv heads * (max_len / 32) * (rows of a kv
 * head / 64), each rounded up, below 2^31 (where it is not the call may return
 * RED_ERR_INVALID_ARG). max_len is the
 * largest number of tokens, nodes included, that a sequence may have: it
 * shapes the launch, and tokens from it on (or beyond table_cols pages) are
 * not looked at. A page number outside the cache is not followed: its tokens
 * read as zeros. Scales of an 8-bit cache are not negative; a scale below
 * 2^-100 counts as that for values; calls that meet one outside 2^-50 .. 2^10,
 * zeros apart, take up to three times as long. Scores and sums are held in float32; in
 * the product with V their exponentials are rounded to `type` (to float16
 * with an 8-bit cache).
 */
typedef struct red_tree_attention_args {
    int type;
    float scale;
    size_t batch, nodes, q_heads;
    size_t max_len;
    const void *q;
    void *out;
    float *lse;
    int64_t q_batch_stride, q_node_stride, q_head_stride;
    int64_t out_batch_stride, out_node_stride, out_head_stride;
    red_paged_cache cache;
    const int32_t *table;
    size_t table_cols;
    int64_t table_stride;
    const int32_t *lens;
    const int64_t *tree_mask;
    const int32_t *node_count;
} red_tree_attention_args;

red_status red_tree_attention(const red_tree_attention_args *a, hipStream_t stream);

/*
 * Verification of drafted tokens by given random numbers. p: (batch, drafts +
 * 1, vocab), the target's probabilities after each prefix; q: (batch, drafts,
 * vocab), the draft's, or NULL where its tokens were certain (q = 1 for the
 * drafted token). Draft i of draft_count[b] (NULL: all) is accepted while
 *
 *   u[b][i] * q[b][i][d_i] < p[b][i][d_i],  d_i = drafted[b][i]
 *
 * (in float64; a token outside the vocabulary is refused), and accepted[b] = n
 * counts those before the first refusal. tokens[b] (drafts + 1 of them) holds
 * the n accepted tokens, then one drawn from the weights w by r[b] (0 <= r <
 * 1), then -1. w = max(p[b][n] - q[b][n], 0) after a refusal, or p[b][n] where
 * that is 0 everywhere or nothing was refused; the token is the first whose
 * running sum of w (float64) exceeds r times the sum. -1 stands for it where
 * w has no positive element or the sum is NaN; with r of 1 or more it is the
 * last of positive weight. type: RED_F32, RED_F16 or RED_BF16 of p and q.
 * drafted, u and tokens are contiguous. drafts may be 0.
 */
typedef struct red_verify_drafts_args {
    int type;
    size_t batch, drafts, vocab;
    const void *p;
    int64_t p_batch_stride, p_step_stride;
    const void *q;
    int64_t q_batch_stride, q_step_stride;
    const int64_t *drafted;
    const float *u;
    const float *r;
    const int32_t *draft_count;
    int32_t *accepted;
    int64_t *tokens;
} red_verify_drafts_args;

red_status red_verify_drafts(const red_verify_drafts_args *a, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBRED_DECODE_H_ */
