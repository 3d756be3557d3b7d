// decode.hpp -- internal interface between the C entry points of
// libred_decode.h (decode.cpp) and their kernels. Every launcher enqueues on
// `stream` and returns the hipError_t of the launch.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

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
    int parts;  // waves that share a token's heads
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

}  // namespace libred
