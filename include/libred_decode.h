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
 * element. Inputs must not overlap outputs unless a call says otherwise.
 *
 * Scratch: the backward pass of the norms, attention over long caches and the
 * verification keep partials in the stream's scratch buffer (the one of the
 * column reductions): grown on demand, kept until the process exits. While
 * the stream is being captured into a graph a call whose scratch is missing or
 * too small returns RED_ERR_CAPTURE before it touches the stream; an earlier
 * call of the same or a larger shape on the stream provides it.
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
 * Read tokens back in 16 bits (8-bit caches: element * scale, rounded once).
 * A slot outside the cache reads as zeros. k and v are written.
 */
red_status red_cache_read(const red_paged_cache *cache, int type, const red_heads *k, const red_heads *v,
                          const int64_t *slots, size_t tokens, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBRED_DECODE_H_ */
