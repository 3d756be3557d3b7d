// The least and the largest elements of the keys of pages:
//
//     lo[d] = min over the page's tokens of k[d],  hi[d] = max.
//
// A wave has a (page, head): G lanes hold a row, one 16-byte load each, so 64 / G
// rows are read at once, four times over, and joined by lane moves at the end.
// Minima and maxima are of float32 values, and rounding them to 16 bits is the same
// as rounding the elements, since rounding keeps the order.
//
// 8 sequences of 7001 to 16384 tokens, 8 heads of 128 in pages of 64, int8 (105 MB with
// scales and bounds): 21.4 us, 4.9 TB/s of the 7.2 that a read reaches, e4m3 the same,
// bfloat16 (204 MB) 32, 6.4 TB/s; a decoding step's page or two of
// 32 sequences 3.3 us, a launch. What is left is the chain of each wave (length, page
// number, keys) at 4 waves a SIMD: 2 or 8 loads in flight, or 6 waves, take 21 to 23.
// Joined by 96 moves through the LDS instead of 28 lane swaps: 25.4.
#include "decode_common.hpp"
#include "serve.hpp"

namespace libred {

namespace {

struct Plain {  // 16-bit cache
    using bits = uint16_t;
    static constexpr bool kScaled = false;
};
struct CodeI8 {
    using bits = uint8_t;
    static constexpr bool kScaled = true;
    static __device__ __forceinline__ void widen4(uint32_t w, float* f) {
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = (float)(int8_t)(w >> (8 * j));
    }
};
struct CodeE4M3 {
    using bits = uint8_t;
    static constexpr bool kScaled = true;
    static __device__ __forceinline__ void widen4(uint32_t w, float* f) {
        f[0] = __builtin_amdgcn_cvt_f32_fp8((int)w, 0);
        f[1] = __builtin_amdgcn_cvt_f32_fp8((int)w, 1);
        f[2] = __builtin_amdgcn_cvt_f32_fp8((int)w, 2);
        f[3] = __builtin_amdgcn_cvt_f32_fp8((int)w, 3);
    }
};

// Joins the N elements that each lane has of the 64 / G rows that a wave read. At
// every step two lanes hand each other half of what they have left, so each ends
// with N * G / 64 elements of all rows, those from (bit 5 of the lane) * N / 2 +
// (bit 4) * N / 4 + (bit 3) * N / 8 on, and all lanes write.
template <int N, int G, class F>
__device__ __forceinline__ void join_rows(float (&v)[N], F op) {
    auto bits = [](float x) { return __builtin_bit_cast(uint32_t, x); };
    auto number = [](uint32_t x) { return __builtin_bit_cast(float, x); };
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const auto s = __builtin_amdgcn_permlane32_swap(bits(v[i]), bits(v[i + N / 2]), false, false);
        v[i] = op(number(s[0]), number(s[1]));
    }
    if constexpr (G <= 16)
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const auto s = __builtin_amdgcn_permlane16_swap(bits(v[i]), bits(v[i + N / 4]), false, false);
            v[i] = op(number(s[0]), number(s[1]));
        }
    if constexpr (G <= 8) {
        const bool upper = threadIdx.x >> 3 & 1;
#pragma unroll
        for (int i = 0; i < N / 8; ++i) {
            const float own = upper ? v[i + N / 8] : v[i], other = upper ? v[i] : v[i + N / 8];
            v[i] = op(own, dpp_move<0x128, 0xF>(other, other));  // 8 lanes on, in rows of 16
        }
    }
}

// VEC elements a lane: those of a 16-byte load, G lanes a row; VEC 1 (any
// alignment): 64 lanes, up to 4 elements each, 64 apart.
template <class T, class C, int VEC, int G>
__global__ __launch_bounds__(kBoundsWaves* kWave) void page_bounds_kernel(PageBounds a) {
    constexpr int N = VEC == 1 ? 4 : VEC, R = kWave / G;
    // Groups of R rows on their way at once.
    constexpr int U = VEC == 1 ? 1 : 4;
    const PagedCache& c = a.cache;
    const int b = blockIdx.y, lane = threadIdx.x % kWave, in = lane % G, row = lane / G;
    const int64_t item = (int64_t)blockIdx.x * kBoundsWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t nth = item / c.heads;
    const int h = (int)(item - nth * c.heads);
    const int len = max(a.lens[b], 0), from = a.first ? max(a.first[b], 0) : 0;
    const int64_t j = from / c.places + nth;  // page of the sequence
    if (nth >= a.most || j >= a.cols || from >= len || j * c.places >= len) return;
    const int page = a.table[b * a.table_stride + j];
    if (page < 0 || page >= c.pages) return;
    const int tokens = (int)min((int64_t)c.places, len - j * c.places);
    const typename C::bits* k = static_cast<const typename C::bits*>(c.k) + page * c.page_stride + h * c.head_stride;
    const float* scales = C::kScaled ? c.k_scales + page * c.scale_page_stride + h * c.scale_head_stride : nullptr;
    float lo[N], hi[N];
#pragma unroll
    for (int i = 0; i < N; ++i) lo[i] = __builtin_inff(), hi[i] = -__builtin_inff();
    const bool there = VEC == 1 || in * VEC < c.dim;
    for (int t0 = 0; t0 < tokens; t0 += R * U) {
        u32x4 x[U];
        float s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // Rows behind the last are the last again.
            const int t = min(t0 + u * R + row, tokens - 1);
            if constexpr (VEC > 1) x[u] = reinterpret_cast<const u32x4*>(k + t * c.place_stride)[there ? in : 0];
            s[u] = C::kScaled ? scales[t * c.scale_place_stride] : 1.f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float f[N];
            if constexpr (VEC == 1) {
                const typename C::bits* r = k + min(t0 + row, tokens - 1) * c.place_stride;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int d = in + i * kWave < c.dim ? in + i * kWave : 0;
                    if constexpr (C::kScaled) {
                        float w[4];
                        C::widen4(r[d], w);
                        f[i] = w[0];
                    } else {
                        f[i] = T::widen(r[d]);
                    }
                }
            } else if constexpr (C::kScaled) {
#pragma unroll
                for (int w = 0; w < 4; ++w) C::widen4(x[u][w], f + 4 * w);
            } else {
                widen_vec<T, 8>(__builtin_bit_cast(typename Vec<T, 8>::type, x[u]), f);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                // fmin and fmax pass over a quiet NaN, but of a signalling one the hardware
                // makes a quiet one in place of what came before it. A product is quiet.
                float v;
                if constexpr (C::kScaled) v = f[i] * s[u];
                else v = __builtin_canonicalizef(f[i]);
                lo[i] = fminf(lo[i], v);
                hi[i] = fmaxf(hi[i], v);
            }
        }
    }
    const int64_t at = page * a.bound_page + h * a.bound_head;
    typename T::bits *to_lo = static_cast<typename T::bits*>(a.lo) + at, *to_hi = static_cast<typename T::bits*>(a.hi) + at;
    if constexpr (VEC > 1) {
        constexpr int L = N / R;
        typedef typename T::bits Out __attribute__((ext_vector_type(L)));
        join_rows<N, G>(lo, [](float m, float n) { return fminf(m, n); });
        join_rows<N, G>(hi, [](float m, float n) { return fmaxf(m, n); });
        if (there) {
            Out l, m;
#pragma unroll
            for (int i = 0; i < L; ++i) l[i] = T::narrow(lo[i]), m[i] = T::narrow(hi[i]);
            const int e = in * N + (lane >> 5 & 1) * (N / 2) + (G <= 16 ? (lane >> 4 & 1) * (N / 4) : 0) + (G <= 8 ? (lane >> 3 & 1) * (N / 8) : 0);
            *reinterpret_cast<Out*>(to_lo + e) = l;
            *reinterpret_cast<Out*>(to_hi + e) = m;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (in + i * kWave < c.dim) {
                to_lo[in + i * kWave] = T::narrow(lo[i]);
                to_hi[in + i * kWave] = T::narrow(hi[i]);
            }
    }
}

template <class T, class C>
hipError_t launch_types(int vec, int lanes, const PageBounds& a, dim3 grid, hipStream_t stream) {
    constexpr int threads = kBoundsWaves * kWave, V = C::kScaled ? 16 : 8;
    if (vec == 1) page_bounds_kernel<T, C, 1, 64><<<grid, threads, 0, stream>>>(a);
    else if (lanes == 8) page_bounds_kernel<T, C, V, 8><<<grid, threads, 0, stream>>>(a);
    else if (lanes == 16) page_bounds_kernel<T, C, V, 16><<<grid, threads, 0, stream>>>(a);
    else if constexpr (!C::kScaled) page_bounds_kernel<T, C, V, 32><<<grid, threads, 0, stream>>>(a);
    return hipGetLastError();
}

template <class T>
hipError_t launch_cache(int cache_type, int vec, int lanes, const PageBounds& a, dim3 grid, hipStream_t stream) {
    if (cache_type == RED_I8) return launch_types<T, CodeI8>(vec, lanes, a, grid, stream);
    if (cache_type == RED_E4M3) return launch_types<T, CodeE4M3>(vec, lanes, a, grid, stream);
    return launch_types<T, Plain>(vec, lanes, a, grid, stream);
}

}  // namespace

hipError_t launch_page_bounds(int type, int cache_type, int vec, int lanes, const PageBounds& a, unsigned int blocks,
                              unsigned int batch, hipStream_t stream) {
    const dim3 grid(blocks, batch);
    return type == RED_F16 ? launch_cache<F16>(cache_type, vec, lanes, a, grid, stream)
                           : launch_cache<BF16>(cache_type, vec, lanes, a, grid, stream);
}

}  // namespace libred
