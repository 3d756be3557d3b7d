// Rows of keys and values into a paged cache, quantised on the way to 8 bits,
// and back.
//
// Write, for a row x: top = max|x|, scale = top / M, element = round(x M / top),
// M = 127 (int8) or 448 (e4m3). Read: element * scale. Both move each row once;
// nothing but memory bounds them (32768 tokens x 8 heads of 128, bf16 and e4m3,
// 204 MB a call: write 44.7 us, 4.6 TB/s; read 36.0 us, 5.7 TB/s; a cache of
// bf16, 268 MB a call: 48.4 and 52.6 us, 5.5 and 5.1 TB/s; 20 tokens in int8 3.7
// and 3.2 us). G lanes hold a row, 8 neighbouring elements
// each (one 16-byte load), so the maximum takes log2(G) lane moves. A wave
// takes 64 / G neighbouring tokens and goes through their (key or value, head)
// pairs: a token's page and place are worked out once, rows of neighbouring
// slots lie side by side in the cache, and their scales share one store. All
// pairs of 4 * 64 / G tokens belong to one block, so that a cache line of
// scales is filled through one XCD's L2.
#include "decode_common.hpp"

namespace libred {

struct Whole {  // 16-bit cache: the values themselves
    using bits = uint16_t;
    static constexpr bool kScaled = false;
};
struct I8 {
    using bits = uint8_t;
    static constexpr bool kScaled = true;
    static constexpr float kTop = 127.f;
    // Adding 1.5 * 2^23 rounds to a whole number (to nearest, ties to even)
    // and leaves its two's complement in the low bits. The sum must not be
    // fused with the product before it: that would round x M / top once
    // instead of twice, and differ at halves.
    static __device__ __forceinline__ uint32_t code(float y) {
#pragma clang fp contract(off)
        return __builtin_bit_cast(uint32_t, y + 12582912.f) & 0xFFu;
    }
    static __device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
        return code(a) | code(b) << 8 | code(c) << 16 | code(d) << 24;
    }
    static __device__ __forceinline__ void unpack4(uint32_t w, float* f) {
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = (float)(int8_t)(w >> (8 * j));
    }
};
struct E4M3 {
    using bits = uint8_t;
    static constexpr bool kScaled = true;
    static constexpr float kTop = 448.f;
    static __device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
        int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
    }
    static __device__ __forceinline__ void unpack4(uint32_t w, float* f) {
        f[0] = __builtin_amdgcn_cvt_f32_fp8((int)w, 0);
        f[1] = __builtin_amdgcn_cvt_f32_fp8((int)w, 1);
        f[2] = __builtin_amdgcn_cvt_f32_fp8((int)w, 2);
        f[3] = __builtin_amdgcn_cvt_f32_fp8((int)w, 3);
    }
};

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Element offset of the row (slot, head 0) and of its scale; false where the
// slot lies outside the cache.
__device__ __forceinline__ bool place_of(const PagedCache& c, int64_t slot, int64_t* row, int64_t* scale) {
    if (slot < 0 || slot >= c.pages * c.places) return false;
    int64_t page, place;
    if (slot <= 0xFFFFFFFFll) {
        const uint32_t q = (uint32_t)slot / (uint32_t)c.places;
        page = q;
        place = (uint32_t)slot - q * (uint32_t)c.places;
    } else {
        page = slot / c.places;
        place = slot - page * c.places;
    }
    *row = page * c.page_stride + place * c.place_stride;
    *scale = page * c.scale_page_stride + place * c.scale_place_stride;
    return true;
}

// The elements of a lane: VEC neighbours (NV 1), or NV of them G apart.
template <class T, class C, int VEC, int G, int NV>
__global__ __launch_bounds__(kCacheWaves* kWave) void cache_write_kernel(CacheRows a) {
    using V = typename Vec<T, VEC>::type;
    constexpr int R = kWave / G;
    // Rows a group has in flight (8: 46.7 us where 4 take 43.5). Stores stay in
    // the caches, for the attention that reads them next: past them the write
    // took 45.8 us and a read after it 39.8 instead of 35.6.
    constexpr int U = NV == 1 ? 4 : 1;
    const int lane = threadIdx.x % G;
    const int64_t t = (int64_t)blockIdx.x * (kCacheWaves * R) + threadIdx.x / G;
    if (t >= a.tokens) return;  // whole groups leave
    const PagedCache& c = a.cache;
    int64_t row, scale;
    if (!place_of(c, a.slots[t], &row, &scale)) return;
    const int pairs = 2 * c.heads, per = (pairs + a.parts - 1) / a.parts;
    const int first = blockIdx.y * per, last = min(pairs, first + per);
    for (int p0 = first; p0 < last; p0 += U) {
        V x[U][NV];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int p = min(p0 + u, last - 1);
            const bool isk = p < c.heads;
            const Heads& s = isk ? a.k : a.v;
            const V* src = reinterpret_cast<const V*>(static_cast<const typename T::bits*>(s.p) + t * s.ts +
                                                      (isk ? p : p - c.heads) * s.hs);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int at = lane + v * G;
                x[u][v] = load_vec<true>(src + (at * VEC < c.dim ? at : 0));
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int p = p0 + u;
            if (p >= last) break;
            const bool isk = p < c.heads;
            const int h = isk ? p : p - c.heads;
            typename C::bits* dst = static_cast<typename C::bits*>(isk ? c.k : c.v) + row + h * c.head_stride;
            if constexpr (!C::kScaled) {
#pragma unroll
                for (int v = 0; v < NV; ++v)
                    if ((lane + v * G) * VEC < c.dim) reinterpret_cast<V*>(dst)[lane + v * G] = x[u][v];
            } else {
                float f[NV][VEC];
                // The largest magnitude by its bits, so that a NaN counts as
                // larger than an infinity and both reach the scale.
                uint32_t top = 0;
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    // Lanes beyond the row hold its first elements again.
                    widen_vec<T, VEC>(x[u][v], f[v]);
#pragma unroll
                    for (int j = 0; j < VEC; ++j)
                        top = max(top, __builtin_bit_cast(uint32_t, f[v][j]) & 0x7FFFFFFFu);
                }
                top = group_combine<G>(top, [](uint32_t m, uint32_t n) { return max(m, n); });
                const float tf = __builtin_bit_cast(float, top);
                // Rows below 2^-100: M / top would leave the range, so the
                // row is scaled up first, exactly.
                const bool tiny = tf < 0x1p-100f;
                const float pre = tiny ? 0x1p100f : 1.f;
                float inv = top != 0 ? C::kTop / (tf * pre) : 0.f;
                const bool finite = top < 0x7F800000u;
                float y[NV][VEC];
#pragma unroll
                for (int v = 0; v < NV; ++v)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) y[v][j] = finite ? f[v][j] * pre * inv : 0.f;
                if constexpr (VEC == 8) {
                    u32x2 w = {C::pack4(y[0][0], y[0][1], y[0][2], y[0][3]), C::pack4(y[0][4], y[0][5], y[0][6], y[0][7])};
                    if (lane * VEC < c.dim) reinterpret_cast<u32x2*>(dst)[lane] = w;
                } else {
#pragma unroll
                    for (int v = 0; v < NV; ++v)
                        if (lane + v * G < c.dim) dst[lane + v * G] = (uint8_t)C::pack4(y[v][0], 0.f, 0.f, 0.f);
                }
                if (lane == 0) (isk ? c.k_scales : c.v_scales)[scale + h * c.scale_head_stride] = tf / C::kTop;
            }
        }
    }
}

// A product rounded to float32. A float16 conversion right behind it would be
// made one rounding with it, but not for vectors of 8, and a cache would read
// differently by how its rows are aligned: the empty asm keeps them apart.
__device__ __forceinline__ float product(float a, float b) {
    float p = a * b;
    asm("" : "+v"(p));
    return p;
}

template <class T, class C, int VEC, int G, int NV>
__global__ __launch_bounds__(kCacheWaves* kWave) void cache_read_kernel(CacheRows a) {
    using V = typename Vec<T, VEC>::type;
    constexpr int R = kWave / G;
    constexpr int U = NV == 1 ? 4 : 1;
    const int lane = threadIdx.x % G;
    const int64_t t = (int64_t)blockIdx.x * (kCacheWaves * R) + threadIdx.x / G;
    if (t >= a.tokens) return;
    const PagedCache& c = a.cache;
    int64_t row = 0, scale = 0;
    const bool inside = place_of(c, a.slots[t], &row, &scale);
    const int pairs = 2 * c.heads, per = (pairs + a.parts - 1) / a.parts;
    const int first = blockIdx.y * per, last = min(pairs, first + per);
    for (int p0 = first; p0 < last; p0 += U) {
        V x[U][NV];
        u32x2 w[U];
        uint8_t b[U][NV];
        float s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int p = min(p0 + u, last - 1);
            const bool isk = p < c.heads;
            const int h = isk ? p : p - c.heads;
            const typename C::bits* src = static_cast<const typename C::bits*>(isk ? c.k : c.v) + row + h * c.head_stride;
            if constexpr (C::kScaled) s[u] = (isk ? c.k_scales : c.v_scales)[scale + h * c.scale_head_stride];
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int at = (lane + v * G) * VEC < c.dim ? lane + v * G : 0;
                if constexpr (!C::kScaled) x[u][v] = reinterpret_cast<const V*>(src)[at];
                else if constexpr (VEC == 8) w[u] = reinterpret_cast<const u32x2*>(src)[at];
                else b[u][v] = src[at];
            }
        }
        if (!inside) {  // the loads were of the cache's first row: zeros instead
#pragma unroll
            for (int u = 0; u < U; ++u) {
                s[u] = 0.f;
                w[u] = u32x2{0, 0};
#pragma unroll
                for (int v = 0; v < NV; ++v) x[u][v] = V{}, b[u][v] = 0;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int p = p0 + u;
            if (p >= last) break;
            const bool isk = p < c.heads;
            const Heads& o = isk ? a.k : a.v;
            V* dst = reinterpret_cast<V*>(static_cast<typename T::bits*>(o.p) + t * o.ts + (isk ? p : p - c.heads) * o.hs);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if ((lane + v * G) * VEC >= c.dim) continue;
                if constexpr (!C::kScaled) {
                    store_vec<true>(dst + lane + v * G, x[u][v]);
                } else if constexpr (VEC == 8) {
                    float f[8];
                    C::unpack4(w[u][0], f);
                    C::unpack4(w[u][1], f + 4);
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] *= s[u];
                    store_vec<true>(dst + lane, narrow_vec<T, 8>(f));
                } else {
                    float f[4];
                    C::unpack4(b[u][v], f);
                    dst[lane + v * G] = T::narrow(product(f[0], s[u]));
                }
            }
        }
    }
}

namespace {

template <class T, class C, int VEC, int G, int NV>
hipError_t launch_shape(const CacheRows& a, bool write, unsigned int groups, hipStream_t stream) {
    const dim3 grid(groups, (unsigned int)a.parts);
    if (write)
        cache_write_kernel<T, C, VEC, G, NV><<<grid, kCacheWaves * kWave, 0, stream>>>(a);
    else
        cache_read_kernel<T, C, VEC, G, NV><<<grid, kCacheWaves * kWave, 0, stream>>>(a);
    return hipGetLastError();
}

template <class T, class C>
hipError_t launch_types(int vec, int lanes, const CacheRows& a, bool write, unsigned int groups, hipStream_t stream) {
    if (vec == 1) return launch_shape<T, C, 1, 64, 4>(a, write, groups, stream);
    switch (lanes) {
        case 8: return launch_shape<T, C, 8, 8, 1>(a, write, groups, stream);
        case 16: return launch_shape<T, C, 8, 16, 1>(a, write, groups, stream);
        case 32: return launch_shape<T, C, 8, 32, 1>(a, write, groups, stream);
        default: return hipErrorInvalidValue;
    }
}

template <class T>
hipError_t launch_cache(int cache_type, int vec, int lanes, const CacheRows& a, bool write, unsigned int groups,
                        hipStream_t stream) {
    if (cache_type == RED_I8) return launch_types<T, I8>(vec, lanes, a, write, groups, stream);
    if (cache_type == RED_E4M3) return launch_types<T, E4M3>(vec, lanes, a, write, groups, stream);
    return launch_types<T, Whole>(vec, lanes, a, write, groups, stream);
}

}  // namespace

hipError_t launch_cache_write(int type, int cache_type, int vec, int lanes, const CacheRows& a, unsigned int groups,
                              hipStream_t stream) {
    return type == RED_F16 ? launch_cache<F16>(cache_type, vec, lanes, a, true, groups, stream)
                           : launch_cache<BF16>(cache_type, vec, lanes, a, true, groups, stream);
}

hipError_t launch_cache_read(int type, int cache_type, int vec, int lanes, const CacheRows& a, unsigned int groups,
                             hipStream_t stream) {
    return type == RED_F16 ? launch_cache<F16>(cache_type, vec, lanes, a, false, groups, stream)
                           : launch_cache<BF16>(cache_type, vec, lanes, a, false, groups, stream);
}

}  // namespace libred
