// decode.hpp -- internal interface between the C entry points of
// libred_decode.h (decode.cpp) and their kernels. Every launcher enqueues on
// `stream` and returns the hipError_t of the launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

#include "libred_decode.h"

namespace libred {

// Heads of a batch of tokens as a kernel sees them.
struct Heads {
    void* p;
    int64_t ts, hs;  // elements from one token / head to the next
};

// Row norms of heads with the rotation. A row is reduced by `lanes` lanes
// holding `vec` neighbouring elements each (lanes 64 and vec 1: up to 4
// elements a lane, 64 apart).
struct QkNorm {
    Heads q, k, q_out, k_out, dq, dk;  // dq, dk: backward only
    const void *q_weight, *k_weight;   // null: ones
    const int64_t* pos;
    const float* freq;
    float* partials;  // backward: 2 * dim floats a block
    int64_t tokens;
    int q_heads, k_heads, dim, rot, interleaved;
    int parts;  // waves that share a token's heads; above 1 only where tokens * parts is below 2^31
    float eps;
};

constexpr int kQkNormWaves = 4;  // waves a block

hipError_t launch_qk_norm_f32(int vec, int lanes, const QkNorm& a, bool back, int blocks, hipStream_t stream);
hipError_t launch_qk_norm_f16(int vec, int lanes, const QkNorm& a, bool back, int blocks, hipStream_t stream);
hipError_t launch_qk_norm_bf16(int vec, int lanes, const QkNorm& a, bool back, int blocks, hipStream_t stream);
// dw[c] = sum over blocks of partials[b * 2 * dim + c]; c < dim: q, from dim on: k.
hipError_t launch_qk_norm_weights(const float* partials, int blocks, int dim, float* dq_weight, float* dk_weight,
                                  hipStream_t stream);

// Rows of a paged cache of 16-bit or 8-bit elements, as a kernel sees them:
// strides in elements.
struct PagedCache {
    void *k, *v;
    float *k_scales, *v_scales;
    int64_t page_stride, head_stride, place_stride;
    int64_t scale_page_stride, scale_head_stride, scale_place_stride;
    int64_t pages;
    int heads, places, dim;
};

struct CacheRows {
    PagedCache cache;
    Heads k, v;  // the tokens' rows: read by a write into the cache, written by a read
    const int64_t* slots;
    int64_t tokens;
    int parts;  // blocks that share the heads of a group of tokens
};

// `vec` 8: rows on 16-byte (16-bit elements) and 8-byte (8-bit ones)
// boundaries, dim a multiple of 8; 1: any. lanes: of a row.
constexpr int kCacheWaves = 4;  // waves a block, each with 64 / lanes tokens
hipError_t launch_cache_write(int type, int cache_type, int vec, int lanes, const CacheRows& a, unsigned int groups,
                              hipStream_t stream);
hipError_t launch_cache_read(int type, int cache_type, int vec, int lanes, const CacheRows& a, unsigned int groups,
                             hipStream_t stream);

// Attention of drafted tokens. Rows of one kv head are numbered node * group +
// query head of the group; a block takes `rows` of them (the shape's) at a
// time. Sequence, kv head and block of rows make a segment; the tiles of all
// segments, one after the other, are shared out evenly over `blocks` blocks.
struct TreeAttention {
    const void* q;
    void* out;
    float* lse;
    int64_t q_batch, q_node, q_head, out_batch, out_node, out_head;  // strides
    PagedCache cache;
    const int32_t* table;
    int64_t table_stride;
    const int32_t* lens;
    const int64_t* mask;   // null: a chain
    const int32_t* count;  // null: all nodes
    int batch, nodes, group, max_tokens, row_blocks;
    int blocks;  // 0: one block a segment, whatever its tiles, that writes the output
    float scale;  // magnitude, times log2(e)
    uint32_t page16, place16;  // strides of the cache's pages and places in units of 16 bytes
    // Token t < 2^30 is in page (4 t factor >> 32) >> shift of its sequence:
    // shift = ceil(log2 places), factor = 2^(30 + shift) / places cut, plus 1.
    uint32_t places_factor;
    int places_shift;
    unsigned int flip;  // 0x80008000 where the scale is negative: the sign of q
    unsigned int keep;  // 0 where the scale is 0 (q is then, and scale is that of 1)
    // The sums of a segment's piece in block w are number w + segment, `rows`
    // rows of `dim` floats, and a maximum and a sum a row.
    float* part_o;
    float2* part_ml;
    int* plan;  // batch + 2: tiles of a segment before sequence b (block 0 writes it), tiles a block
};

// How waves share a block: `waves_m` groups of `wave_rows` rows times
// `waves_t` parts of the tokens, `step` tokens a wave at a time.
struct AttentionShape {
    int wave_rows, waves_m, waves_t, step;
    constexpr int rows() const { return wave_rows * waves_m; }
    constexpr int tokens() const { return waves_t * step; }
    constexpr bool is(const AttentionShape& o) const {
        return wave_rows == o.wave_rows && waves_m == o.waves_m && waves_t == o.waves_t && step == o.step;
    }
};
constexpr AttentionShape kFewestRows = {16, 1, 4, 32}, kFewRows = {32, 1, 4, 32}, kHalfRows = {16, 4, 1, 32},
                         kManyRows = {32, 4, 1, 64};
constexpr int kNarrowHeads = 128, kNarrowPairs = 96;
// The shape for `rows` rows of a kv head of `dim` elements, cached in `bytes`
// each. Few rows share the queries and split the tokens among a block's waves,
// many rows split the rows and share the tokens; 16 rows a wave read every
// tile of LDS twice as often, 32 rows need twice the registers: they spill
// from 97 elements of 16 bits (17 to 32 rows), and do not fit beyond 128.
// Microseconds of 8 sequences of 3000 to 8000 tokens, 4 kv heads:
//   rows, heads, cache     kFewRows  kHalfRows  kManyRows
//   32,    64, bf16          16.3      19.7
//   32,    96, bf16          20.9      22.8
//   32,   128, bf16          33.4      23.9       31.5
//   64,    64, bf16 / e4m3             19.4 / 24.6   22.4 / 25.5
//   64,   128, bf16 / e4m3             26.0 / 27.3   32.0 / 32.2
//   128,   64, bf16                    29.5       24.7
//   128,  128, bf16                    39.5       36.4
// 32 sequences of 1500 to 16384 tokens, 8 kv heads of 128 in int8, 32 rows:
// kFewRows 115.5, kHalfRows 234.
constexpr AttentionShape attention_shape(int rows, int dim, int bytes) {
    return rows <= kFewestRows.rows()                                    ? kFewestRows
           : dim > kNarrowHeads                                          ? kHalfRows
           : rows <= kFewRows.rows() && (bytes == 1 || dim <= kNarrowPairs) ? kFewRows
           : rows <= kHalfRows.rows()                                    ? kHalfRows
                                                                         : kManyRows;
}
// The fewest tokens of a tile that so many rows, or fewer, are given.
constexpr int attention_least_tokens(int rows, int dim, int bytes) {
    int least = attention_shape(rows, dim, bytes).tokens();
    for (const int fewer : {kFewestRows.rows(), kFewRows.rows(), kHalfRows.rows()})
        if (fewer < rows && attention_shape(fewer, dim, bytes).tokens() < least) least = attention_shape(fewer, dim, bytes).tokens();
    return least;
}
// Blocks that a compute unit holds at once.
constexpr int attention_blocks(int rows, int dim) { return rows <= kFewestRows.rows() && dim > kNarrowHeads ? 1 : 2; }
// How many of `all` tiles (below 2^31) each of `blocks` blocks takes, and the
// first that is block `share`'s.
__host__ __device__ inline int share_size(int all, int blocks) { return all / blocks + (all % blocks != 0); }
__host__ __device__ inline int share_begin(int all, int per, int share) {
    const int64_t at = (int64_t)per * share;
    return (int)(at < all ? at : all);
}
// Joins the pieces of every row into the output (rows_a_block: the shape's).
hipError_t launch_attention_combine(int type, const TreeAttention& a, int rows_a_block, hipStream_t stream);
hipError_t launch_tree_attention(int type, int cache_type, const TreeAttention& a, hipStream_t stream);
hipError_t launch_attention_f16_16(const TreeAttention& a, hipStream_t stream);
hipError_t launch_attention_f16_i8(const TreeAttention& a, hipStream_t stream);
hipError_t launch_attention_f16_e4m3(const TreeAttention& a, hipStream_t stream);
hipError_t launch_attention_bf16_16(const TreeAttention& a, hipStream_t stream);
hipError_t launch_attention_bf16_i8(const TreeAttention& a, hipStream_t stream);
hipError_t launch_attention_bf16_e4m3(const TreeAttention& a, hipStream_t stream);

// Verification of drafted tokens: a sequence's row is cut into `segs` segments
// of `seg` tokens.
struct Verify {
    const void *p, *q;  // q null: the draft's tokens were certain
    int64_t p_batch, p_step, q_batch, q_step;
    const int64_t* drafted;
    const float *u, *r;
    const int32_t* count;
    int32_t* accepted;
    int64_t* tokens;
    double* sums;  // batch * segs
    int64_t vocab, seg;
    int batch, drafts, segs;
    int blocks;  // a sequence, of 4 waves that take segments in turn; 0: one launch, a block a sequence
};
constexpr int kVerifyMaxSegs = 256;
hipError_t launch_verify(int type, const Verify& a, hipStream_t stream);

}  // namespace libred
