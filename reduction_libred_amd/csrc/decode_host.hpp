// decode_host.hpp -- what the C entry points of libred_decode.h and
// libred_serve.h share on the host: spans and checks of strided and paged
// tensors, and how many blocks a launch may have.
#pragma once

#include "decode.hpp"
#include "host.hpp"

namespace libred {

inline size_t type_bytes(int type) { return type == RED_F32 ? 4 : type == RED_F16 || type == RED_BF16 ? 2 : 1; }

// Largest element offset a strided tensor may reach (the byte offset of an
// 8-byte element still fits 63 bits).
constexpr int64_t kMaxSpan = (int64_t)1 << 59;

// Elements spanned by tokens x heads x dim at these strides; -1 if a stride
// is negative or the span is out of range.
inline int64_t span_of(const red_heads& h, size_t tokens, size_t dim) {
    if (h.heads < 0 || h.token_stride < 0 || h.head_stride < 0) return -1;
    if (h.heads == 0 || tokens == 0) return 0;
    int64_t a, b, s;
    if (__builtin_mul_overflow((int64_t)(tokens - 1), h.token_stride, &a) ||
        __builtin_mul_overflow(h.heads - 1, h.head_stride, &b) || __builtin_add_overflow(a, b, &s) ||
        __builtin_add_overflow(s, (int64_t)dim, &s) || s > kMaxSpan)
        return -1;
    return s;
}

// Rows of an output must lie apart from each other.
inline bool rows_apart(const red_heads& h, size_t tokens, size_t dim) {
    const int64_t d = (int64_t)dim, t = (int64_t)tokens;
    if (h.heads == 0 || t == 0) return true;
    if (h.heads > 1 && h.head_stride < d) return false;
    if (t > 1 && h.token_stride < d) return false;
    if (h.heads == 1 || t == 1) return true;
    return h.token_stride >= (h.heads - 1) * h.head_stride + d || h.head_stride >= (t - 1) * h.token_stride + d;
}

// Elements (or scales) spanned by a paged tensor of these strides, -1 if
// negative or out of range.
inline int64_t paged_span(const red_paged_cache& c, int64_t page, int64_t head, int64_t place, size_t dim) {
    if (page < 0 || head < 0 || place < 0) return -1;
    int64_t a, b, d, s;
    if (__builtin_mul_overflow((int64_t)c.pages - 1, page, &a) || __builtin_mul_overflow((int64_t)c.heads - 1, head, &b) ||
        __builtin_mul_overflow((int64_t)c.places - 1, place, &d) || __builtin_add_overflow(a, b, &s) ||
        __builtin_add_overflow(s, d, &s) || __builtin_add_overflow(s, (int64_t)dim, &s) || s > kMaxSpan)
        return -1;
    return s;
}

// A cache with at least one page, or one that holds nothing (pages 0).
inline bool cache_valid(const red_paged_cache* c) {
    if (c == nullptr) return false;
    if (c->type != RED_F16 && c->type != RED_BF16 && c->type != RED_I8 && c->type != RED_E4M3) return false;
    if (c->heads < 1 || c->heads > 1 << 20 || c->places < 1 || c->places > 1 << 20 || c->dim < 1 ||
        c->dim > RED_HEAD_MAX_DIM || c->pages > (size_t)1 << 40)
        return false;
    if (c->pages == 0) return true;
    const bool scaled = c->type == RED_I8 || c->type == RED_E4M3;
    const size_t es = type_bytes(c->type);
    if (c->k == nullptr || c->v == nullptr || !is_aligned(c->k, es) || !is_aligned(c->v, es)) return false;
    if (paged_span(*c, c->page_stride, c->head_stride, c->place_stride, c->dim) < 0) return false;
    if (!scaled) return c->k_scales == nullptr && c->v_scales == nullptr;
    if (c->k_scales == nullptr || c->v_scales == nullptr || !is_aligned(c->k_scales, 4) || !is_aligned(c->v_scales, 4))
        return false;
    return paged_span(*c, c->scale_page_stride, c->scale_head_stride, c->scale_place_stride, 1) >= 0;
}

inline PagedCache to_cache(const red_paged_cache& c) {
    return PagedCache{c.k, c.v, c.k_scales, c.v_scales, c.page_stride,
                      c.head_stride, c.place_stride, c.scale_page_stride, c.scale_head_stride, c.scale_place_stride,
                      (int64_t)c.pages, (int)c.heads, (int)c.places, (int)c.dim};
}

// Whether the cache's rows start on `bytes` boundaries.
inline bool cache_rows_on(const red_paged_cache& c, size_t bytes) {
    const int64_t es = (int64_t)type_bytes(c.type), b = (int64_t)bytes;
    return is_aligned(c.k, bytes) && is_aligned(c.v, bytes) && (c.pages <= 1 || c.page_stride * es % b == 0) &&
           (c.heads == 1 || c.head_stride * es % b == 0) && (c.places == 1 || c.place_stride * es % b == 0);
}

// A launch has fewer than 2^32 threads: most blocks of 256 that one may have.
// Calls of more go in several launches, one after the other.
constexpr size_t kMaxBlocks = ((size_t)1 << 24) - 1;

}  // namespace libred
