/*
 * libred_serve.h -- what a serving step needs around the calls of
 * libred_decode.h: where the next tokens of every sequence go in the paged
 * cache, attention over the pages that a cheap score selects, and sampling
 * from filtered probabilities.
 *
 * The conventions of libred_decode.h hold: device pointers, argument structs
 * that the call reads before it returns, strides in elements with a contiguous
 * last dimension, inputs that do not overlap outputs, refusals before any HIP
 * call, deterministic results. Scratch: every call here but the bounds of pages
 * and the sampling of up to 8192 tokens keeps intermediate results in the
 * stream's scratch buffer, under the rule of libred_decode.h: while a stream is
 * captured, an earlier call on it of the same types, kv heads, dim and places,
 * and no less of the rest, must have provided it, else the call returns
 * RED_ERR_CAPTURE.
 */
#ifndef LIBRED_SERVE_H_
#define LIBRED_SERVE_H_

#include "libred_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Pages and slots for the next tokens of `batch` sequences. Sequence b holds
 * lens[b] tokens and takes counts[b] more (numbers below 0 count as 0). Row b
 * of `table` lists its pages, held[b] of them; free_pages is a stack of
 * free_count[0] pages, `pages` at most, whose entries behind that are -1.
 *
 *  - Rows with done[b] != 0 (NULL: none) are given back first: their pages are
 *    pushed, rows in order and the pages of a row in order, and held[b] counts
 *    as 0. lens[b] is that of the sequence that has the row now.
 *  - Sequence b wants max(0, ceil((lens[b] + counts[b]) / places) - held[b])
 *    pages, none where counts[b] is 0. It is refused where its tokens are more
 *    than table_cols pages hold or their numbers pass `tokens`, and wants none
 *    then.
 *  - Going through the sequences in order, pages are handed out as long as
 *    there are enough; from the first sequence that does not get its pages on,
 *    every one that wants any is refused. The pages taken are the topmost of
 *    the stack, lowest first, and their entries become -1.
 *
 * Token i of sequence b is number starts[b] + i, starts[b] being the running
 * sum of the counts before b, at most `tokens`; starts has batch + 1 numbers.
 * pos[number] = lens[b] + i, and slots[number] = table[b][pos / places] *
 * places + pos % places, or -1 where b was refused. Numbers from
 * starts[batch] on have slot -1 and position 0. granted[b] is counts[b], or 0
 * where refused. table, held, free_pages and free_count are updated; entries
 * of the table from held[b] on are left as they were.
 *
 * A page must be listed once, in a row or on the stack. Page numbers are not
 * looked at: one outside the cache gives slots outside of it. held[b] counts
 * as at least 0 and at most table_cols, free_count[0] as at most `pages`; pages
 * that the stack has no room for are dropped. batch <= 65535, tokens and pages
 * below 2^31, table_cols <= 2^30, places <= 2^20, and batch * table_cols below
 * 2^31. slots and pos are `tokens` numbers each.
 */
typedef struct red_plan_slots_args {
    size_t batch, tokens, places, pages;
    const int32_t *lens;
    const int32_t *counts;
    const int32_t *done;
    int32_t *table;
    size_t table_cols;
    int64_t table_stride;
    int32_t *held;
    int32_t *free_pages;
    int32_t *free_count;
    int64_t *slots;
    int64_t *pos;
    int32_t *starts;
    int32_t *granted;
} red_plan_slots_args;

red_status red_plan_slots(const red_plan_slots_args *a, hipStream_t stream);

/*
 * The least and the largest element of the keys of whole pages:
 *
 *   lo[page][h][d] = min over the page's tokens of k[d], hi = max
 *
 * for the pages of sequence b that hold tokens from first[b] (NULL: 0) to
 * lens[b] - 1, all their tokens below lens[b] counted; at most `most` pages of
 * a sequence, the first of them (it shapes the launch). A NaN is passed over;
 * where there is nothing else lo is inf and hi -inf. type RED_F16 or RED_BF16
 * of lo and hi, and the cache's own type where that has 16 bits; with an 8-bit
 * cache element * scale in float32, rounded to `type`. lo and hi: element
 * (p, h, d) at p * bound_page_stride + h * bound_head_stride + d, pages and
 * heads those of the cache. (Rounded to nearest, as red_cache_read does: a key
 * in float32 may lie outside its page's bounds by half a step of `type`, the key
 * that is read back in `type` does not.) The cache's v and v_scales are not read and may be
 * NULL. Page numbers outside the cache are skipped. Two sequences may share
 * pages that both fill. batch <= 65535.
 */
typedef struct red_page_bounds_args {
    int type;
    size_t batch, most;
    red_paged_cache cache;
    const int32_t *table;
    size_t table_cols;
    int64_t table_stride;
    const int32_t *lens;
    const int32_t *first;
    void *lo;
    void *hi;
    int64_t bound_page_stride, bound_head_stride;
} red_page_bounds_args;

red_status red_page_bounds(const red_page_bounds_args *a, hipStream_t stream);

/*
 * The pages that are worth reading for the queries of every sequence, chosen
 * for each kv head. Sequence b has lens[b] tokens and then its nodes
 * (node_count[b] of them, NULL: all), whose keys may be in the cache or not
 * yet; P = ceil((lens[b] + nodes) / places). With q (batch, nodes, q_heads,
 * dim), of which heads h * group .. read kv head h, a page's score is the sum
 * over these heads and the nodes of the largest q . k that a key between the
 * page's bounds could have:
 *
 *   score = sum max(q_d lo_d, q_d hi_d) = sum_d (U_d hi_d + D_d lo_d),
 *   U_d = sum max(q_d, 0),  D_d = sum min(q_d, 0)
 *
 * in float64, a product of 0 and an infinite bound being 0. Selected are
 * min(P, budget) pages: the first `first`, those from floor(lens[b] / places) -
 * last on, and of the others those of the largest scores, ties to the lower
 * page; a score that is NaN is below all others. selected[b][h][i] (int32, batch x kv heads x budget) are their page
 * numbers in the order of the sequence, then -1. selected_lens[b] = lens[b] -
 * places * (pages left out): lens of the sequence that has the selected pages
 * alone. A sequence without nodes has no pages selected and length 0.
 *
 * The score is of q . k: for an attention whose scale is below 0, -q is given.
 *
 * type RED_F16 or RED_BF16 of q, lo and hi (as red_page_bounds leaves them;
 * pages behind floor(lens / places) - last are not looked at). max_len: the
 * most tokens of a sequence, nodes included; it shapes the launch, and tokens
 * from it on, or beyond table_cols pages, do not count. Page numbers outside
 * [0, pages) have score NaN. budget >= first + last + 1 + ceil(nodes /
 * places). nodes <= 64, batch and q_heads <= 65535, q_heads a multiple of the kv
 * heads and not 0, dim 1 .. 256, max_len <= 2^30, batch * kv heads * ceil(max_len / places) below 2^31.
 */
typedef struct red_select_pages_args {
    int type;
    size_t batch, nodes, q_heads, kv_heads, dim;
    size_t pages, places;
    size_t budget, first, last;
    size_t max_len;
    const void *q;
    int64_t q_batch_stride, q_node_stride, q_head_stride;
    const void *lo;
    const void *hi;
    int64_t bound_page_stride, bound_head_stride;
    const int32_t *table;
    size_t table_cols;
    int64_t table_stride;
    const int32_t *lens;
    const int32_t *node_count;
    int32_t *selected;
    int32_t *selected_lens;
} red_select_pages_args;

red_status red_select_pages(const red_select_pages_args *a, hipStream_t stream);

/*
 * red_tree_attention with a table for each kv head: token t of sequence b lies,
 * for kv head h, in page table[b * table_stride + h * table_head_stride + t /
 * places]. With what red_select_pages leaves (table_head_stride = budget,
 * table_stride = kv heads * budget, lens = selected_lens) it attends over the
 * selected pages alone. table_head_stride 0: red_tree_attention.
 */
red_status red_sparse_attention(const red_tree_attention_args *a, int64_t table_head_stride, hipStream_t stream);

/*
 * Sampling. logits: (batch, steps, vocab); settings are those of a sequence,
 * r, tokens and probs those of each step. With x a row of logits, T its
 * temperature, and the tokens in order of falling x, ties by their numbers:
 *
 *   w_i = exp((x_i - max x) / T)
 *   top_k: the first top_k of the order are kept
 *   top_p: of those, the ones before which the sum of w is below top_p times
 *          their whole sum
 *   min_p: of those, the ones of w >= min_p
 *   probs_i = w_i / sum of kept w, 0 where not kept
 *   token: the first whose running sum of kept w exceeds r times that sum
 *
 * The first of the order is always kept. A setting that is NULL, top_k below
 * 1 or from vocab on, top_p or min_p that is NaN, top_p from 1 on and min_p
 * down from 0 filter nothing; min_p above 1 counts as 1, top_p below 0 as 0.
 * T NULL is 1; a T of 0, below, or NaN keeps the first of the order alone. A
 * NaN counts as -inf; -inf has w = 0; where x holds +inf, those have w = 1 and
 * all others 0. A row of -inf has probabilities 0 and token -1. With r of 1 or
 * more, or NaN, the token is the last that may be drawn.
 *
 * Weights are float64; in sums each counts as a whole number of units, so they
 * do not depend on any order. A unit is 2^(ceil(log2 vocab) - 62), 2^-51 at the
 * least. A weight below half a unit has its probability, but is not drawn. Rows
 * of more than 8192 tokens are added up by bins of equal ratios of the weight,
 * in which a weight counts to within 2^-35 of itself, those below half a unit
 * too; where all kept tokens have the largest logit the sums are exact. A border
 * or token whose target lies closer to a running sum than that may be the
 * neighbouring one, the same one every time.
 *
 * type: RED_F32, RED_F16 or RED_BF16 of the logits; probs_type the same of
 * probs. tokens (with r) or probs may be NULL: not wanted. tokens and r are
 * contiguous. batch <= 65535, steps <= 65535, batch * steps below 2^22,
 * 1 <= vocab <= 2^20. Rows of probs lie apart from each other.
 */
typedef struct red_sample_args {
    int type;
    int probs_type;
    size_t batch, steps, vocab;
    const void *logits;
    int64_t batch_stride, step_stride;
    const float *temperature; /* batch */
    const int32_t *top_k;
    const float *top_p;
    const float *min_p;
    const float *r;  /* batch * steps */
    int64_t *tokens; /* batch * steps */
    void *probs;
    int64_t probs_batch_stride, probs_step_stride;
} red_sample_args;

red_status red_sample(const red_sample_args *a, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBRED_SERVE_H_ */
