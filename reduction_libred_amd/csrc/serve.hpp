// serve.hpp -- internal interface between the C entry points of libred_serve.h
// (serve.cpp) and their kernels. Every launcher enqueues on `stream` and
// returns the hipError_t of the launch.
#pragma once

#include "decode.hpp"
#include "libred_serve.h"

namespace libred {

// Bytes up to the highest that is not 0. (Written with compares: from "v ? 64 -
// __clzll(v) : 0" as a shift's distance the compiler drops the case of 0.)
__host__ __device__ inline int bytes_of(uint64_t v) {
    int n = 0;
    for (int i = 0; i < 8; ++i)
        if (v >> (8 * i)) n = i + 1;
    return n;
}

// Slots of a step's tokens.
struct PlanSlots {
    const int32_t *lens, *counts, *done;  // done null: none
    int32_t* table;
    int64_t table_stride;
    int32_t *held, *stack, *height;
    int64_t *slots, *pos;
    int32_t *starts, *granted;
    int batch, tokens, cols, places, pages;
    // Of a sequence, in the scratch: pages it has, of those taken the ones before
    // its, of those given back the ones before its.
    int32_t *have, *before, *back;
    int32_t* sums;   // 4: stack's height before, with the pages given back, and behind the step
    int32_t* fresh;  // the pages taken
};
// blocks 0: one launch of one block; else two, or three unless `few` pages are moved.
hipError_t launch_plan_slots(const PlanSlots& a, int blocks, bool few, hipStream_t stream);

// Bounds of the keys of pages.
struct PageBounds {
    PagedCache cache;
    const int32_t* table;
    int64_t table_stride;
    const int32_t *lens, *first;
    void *lo, *hi;
    int64_t bound_page, bound_head;
    int cols, most;
};
constexpr int kBoundsWaves = 4;  // waves a block, a (page, head) each
hipError_t launch_page_bounds(int type, int cache_type, int vec, int lanes, const PageBounds& a, unsigned int blocks,
                              unsigned int batch, hipStream_t stream);

// Selection of pages.
struct SelectPages {
    const void* q;
    int64_t q_batch, q_node, q_head;
    const void *lo, *hi;
    int64_t bound_page, bound_head;
    const int32_t* table;
    int64_t table_stride;
    const int32_t *lens, *count;
    int32_t *selected, *selected_lens;
    uint64_t* keys;  // batch * heads * most: of pages, larger for those that are rather selected
    int64_t pages;
    int batch, nodes, heads, group, dim, places, budget, first, last;
    int most;   // pages of a sequence
    int share;  // of them that a block scores
    int max_len;
};
constexpr int kSelectPages = 64;  // a multiple of this many pages has a block that scores them
hipError_t launch_select_pages(int type, int vec, int lanes, const SelectPages& a, hipStream_t stream);

// Sampling. A row goes through one block, or is cut into chunks. The list holds the
// codes near a border, 1000 of 131072 as a rule; flat rows have more (see
// sample_split.hip).
constexpr int kSampleChunk = 8192, kSampleGrid = 512, kSampleList = 16384;
// Rows of up to so many logits are held by one block. (Microseconds of 1 / 192 / 1900
// float32 rows, top-p, replayed: 4000 logits 10.4 / 11.6 / 74 by a block, 22 / 24 / 120
// by chunks; 8000 logits 15.0 / 16.7 / 117 and 23 / 26 / 145; 12000 logits, for which a
// block's registers are too few, 29 / 39 / 286 and 24 / 29 / 139.)
constexpr int kSampleRow = 8192;
struct SampleHead {  // of a chunk
    uint64_t first;  // the first code of the order
    int count;       // logits above -inf, where top-k asks for it
};
enum { kRowNone = 0, kRowOne = 1, kRowWhole = 2, kRowCut = 3 };  // empty, one token kept, by a block alone, by its chunks
struct SamplePlan {  // of a row
    uint64_t first, cut, k_rest, k_before, p_before, all;
    uint64_t largest;  // relative units of the largest weight
    double norm;  // of a bin's relative sum to units, at bin 0
    float from[2], upto[2];  // logits that are gathered
    int state, ranges, low, high;
    int use_k, use_p;
    unsigned int held;  // how many are
    uint64_t border;  // the last code that is kept
    double share;     // of a weight in the probabilities
};
struct Sample {
    const void* x;
    int64_t batch_stride, step_stride;
    const float* temperature;
    const int32_t* top_k;
    const float *top_p, *min_p, *r;
    int64_t* tokens;
    void* probs;
    int64_t probs_batch, probs_step;
    int steps, vocab;
    int shift;  // weights are counted in units of 2^-shift
    int first_row;
    int chunks;    // of a row; 0: none
    int filtered;  // top-k, top-p or min-p may leave something out
    SampleHead* heads;         // rows * chunks
    unsigned long long* bins;  // rows * chunks * kSampleGrid
    unsigned long long* list;  // rows * kSampleList
    SamplePlan* plans;         // rows
};
hipError_t launch_sample_split(int type, int probs_type, const Sample& a, unsigned int rows, hipStream_t stream);
hipError_t launch_sample(int type, int probs_type, const Sample& a, unsigned int rows, hipStream_t stream);

}  // namespace libred
