// decode_common.hpp -- element types, vectors of them and sums over lane groups,
// shared by the kernels of the decoding step.
#pragma once

#include "decode.hpp"
#include "device_common.hpp"

namespace libred {

struct F32 {
    using bits = uint32_t;
    static __device__ __forceinline__ float widen(bits b) { return __builtin_bit_cast(float, b); }
    static __device__ __forceinline__ bits narrow(float v) { return __builtin_bit_cast(bits, v); }
};
struct F16 {
    using bits = uint16_t;
    static __device__ __forceinline__ float widen(bits b) { return (float)__builtin_bit_cast(_Float16, b); }
    static __device__ __forceinline__ bits narrow(float v) { return __builtin_bit_cast(bits, (_Float16)v); }
};
struct BF16 {
    using bits = uint16_t;
    static __device__ __forceinline__ float widen(bits b) { return __builtin_bit_cast(float, (uint32_t)b << 16); }
    static __device__ __forceinline__ bits narrow(float v) { return __builtin_bit_cast(bits, (__bf16)v); }
};

template <class T, int VEC>
struct Vec {
    typedef typename T::bits type __attribute__((ext_vector_type(VEC)));
};
template <class T>
struct Vec<T, 1> {
    typedef typename T::bits type;
};

template <class T, int VEC>
__device__ __forceinline__ void widen_vec(typename Vec<T, VEC>::type v, float (&f)[VEC]) {
    if constexpr (VEC == 1) {
        f[0] = T::widen(v);
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) f[j] = T::widen(v[j]);
    }
}
template <class T, int VEC>
__device__ __forceinline__ typename Vec<T, VEC>::type narrow_vec(const float (&f)[VEC]) {
    if constexpr (VEC == 1) {
        return T::narrow(f[0]);
    } else {
        typename Vec<T, VEC>::type v;
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] = T::narrow(f[j]);
        return v;
    }
}

// Combine over the G lanes of a group with `op`; every lane gets the result.
template <int G, class V, class F>
__device__ __forceinline__ V group_combine(V v, F op) {
    if constexpr (G >= 2) v = op(v, dpp_move<0xB1, 0xF>(v, v));   // neighbours
    if constexpr (G >= 4) v = op(v, dpp_move<0x4E, 0xF>(v, v));   // pairs of a quad
    if constexpr (G >= 8) v = op(v, dpp_move<0x141, 0xF>(v, v));  // quads of a half row
    if constexpr (G >= 16) v = op(v, dpp_move<0x140, 0xF>(v, v)); // half rows of a row
    if constexpr (G >= 32) v = op(v, __shfl_xor(v, 16));
    if constexpr (G >= 64) v = op(v, __shfl_xor(v, 32));
    return v;
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
    return group_combine<G>(v, [](float a, float b) { return a + b; });
}

// A wave's LDS writes are seen by its own later reads (the LDS serves a wave
// in order); this keeps the compiler from moving them past each other.
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Tokens of sequence b, nodes included, and how many nodes it has.
__device__ __forceinline__ int sequence_tokens(const TreeAttention& a, int b, int* nodes) {
    const int count = a.count ? min(max(a.count[b], 0), a.nodes) : a.nodes;
    *nodes = count;
    return (int)min((int64_t)max(a.lens[b], 0) + count, (int64_t)a.max_tokens);
}

}  // namespace libred
