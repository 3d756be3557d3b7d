// qk_norm.hpp -- RMS norm of every query and key head with the rotary rotation
// in the same pass, and its backward pass.
//
// Forward, for a head x of `dim` elements at position p:
//     r = 1 / sqrt(mean(x^2) + eps),  y = x r w,
//     (y_a, y_b) -> (y_a c - y_b s, y_a s + y_b c),  c, s = cos, sin(p freq_i).
// Backward: g is dy rotated the other way, h = g w,
//     dx = r (h - x r^2 mean(h x)),  dw = sum over rows of g x r.
//
// A wave takes one token (or one of `parts` shares of its heads) and goes
// through the heads, 64 / G rows at a time: G lanes hold a row, VEC
// neighbouring elements each, loaded with one 16-byte load. Cosines, sines and
// weights depend on the column alone, so a lane loads them once a token and
// keeps them in registers. The angles of a token are computed once, one pair a
// lane: the product and its reduction to an eighth of a turn in float64 (a
// position of 2^20 leaves a float32 angle no correct digit behind the point),
// then the Taylor sums of sine and cosine.
#pragma once

#include "decode_common.hpp"

namespace libred {

// cos and sin of 2 pi t from t in turns. Quarter turns come off exactly, the
// rest is at most an eighth of a turn, where the Taylor sums to the 14th power
// are off by less than 1e-15.
__device__ __forceinline__ float2 cos_sin_turns(double t) {
    const double q = rint(4.0 * t);
    const double x = (t - 0.25 * q) * 6.283185307179586476925;
    const double z = x * x;
    double s = 1.0 / 6227020800.0, c = -1.0 / 87178291200.0;
    s = fma(s, z, -1.0 / 39916800.0);
    s = fma(s, z, 1.0 / 362880.0);
    s = fma(s, z, -1.0 / 5040.0);
    s = fma(s, z, 1.0 / 120.0);
    s = fma(s, z, -1.0 / 6.0);
    s = fma(s * z, x, x);
    c = fma(c, z, 1.0 / 479001600.0);
    c = fma(c, z, -1.0 / 3628800.0);
    c = fma(c, z, 1.0 / 40320.0);
    c = fma(c, z, -1.0 / 720.0);
    c = fma(c, z, 1.0 / 24.0);
    c = fma(c, z, -0.5);
    c = fma(c, z, 1.0);
    const int n = (int)(q - 4.0 * floor(q * 0.25));
    const double a = n & 1 ? s : c, b = n & 1 ? c : s;
    return make_float2((float)(n == 1 || n == 2 ? -a : a), (float)(n >= 2 ? -b : b));
}

constexpr int kHeadMax = RED_HEAD_MAX_DIM;
// LDS of a wave: cosines and sines of a token, or the rows that change halves.
constexpr int kWaveFloats = 64 * 8;

// How the two elements of a pair meet.
enum { kTurnNone = 0, kTurnInside = 1, kTurnVectors = 2, kTurnElements = 3 };

template <int VEC>
__device__ __forceinline__ int turn_mode(int rot, int interleaved) {
    if (rot == 0) return kTurnNone;
    if (interleaved) return VEC > 1 ? kTurnInside : kTurnElements;
    return (rot / 2) % VEC == 0 && VEC > 1 ? kTurnVectors : kTurnElements;
}

// f <- f c + partner g for the elements of this lane; `row` is the row's part
// of the wave's LDS (dim floats), u0 this lane's first element.
template <int VEC, int G, int NV>
__device__ __forceinline__ void turn(float (&f)[NV][VEC], const float (&c)[NV][VEC], const float (&g)[NV][VEC],
                                     int mode, int interleaved, int lane, int dim, int rot, float* row) {
    if (mode == kTurnNone) return;
    if constexpr (VEC > 1) {
        if (mode == kTurnInside) {
#pragma unroll
            for (int j = 0; j < VEC; j += 2) {
                const float a = f[0][j], b = f[0][j + 1];
                f[0][j] = a * c[0][j] + b * g[0][j];
                f[0][j + 1] = b * c[0][j + 1] + a * g[0][j + 1];
            }
            return;
        }
    }
    const int half = rot / 2;
    wave_lds_fence();
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int d = (lane + v * G) * VEC;
        if (d >= rot) continue;
        if constexpr (VEC >= 4) {
#pragma unroll
            for (int j = 0; j < VEC; j += 4)
                *reinterpret_cast<f32x4*>(row + d + j) = f32x4{f[v][j], f[v][j + 1], f[v][j + 2], f[v][j + 3]};
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) row[d + j] = f[v][j];
        }
    }
    wave_lds_fence();
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int d = (lane + v * G) * VEC;
        if (d >= rot) continue;
        if (VEC > 1 && mode == kTurnVectors) {
            const f32x4* o = reinterpret_cast<const f32x4*>(row + (d < half ? d + half : d - half));
#pragma unroll
            for (int j = 0; j < VEC; ++j) f[v][j] = f[v][j] * c[v][j] + o[j / 4][j % 4] * g[v][j];
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const int e = d + j;
                const int o = interleaved ? e ^ 1 : (e < half ? e + half : e - half);
                if (e < rot) f[v][j] = f[v][j] * c[v][j] + row[o] * g[v][j];
            }
        }
    }
}

// Cosines and signed sines of this lane's columns for token position `p`.
// back: the rotation the other way.
template <int VEC, int G, int NV, bool BACK>
__device__ __forceinline__ void token_turns(float (&c)[NV][VEC], float (&g)[NV][VEC], int64_t p, const float* freq,
                                            int rot, int interleaved, int lane, float2* table) {
    const int half = rot / 2;
    wave_lds_fence();
    for (int i = threadIdx.x % kWave; i < half; i += kWave) {
        const double a = (double)p * (double)freq[i] * 0.15915494309189533577;  // turns
        table[i] = cos_sin_turns(a - rint(a));
    }
    wave_lds_fence();
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const int d = (lane + v * G) * VEC + j;
            float2 cs = make_float2(1.f, 0.f);
            bool first = true;
            if (d < rot) {
                first = interleaved ? !(d & 1) : d < half;
                cs = table[interleaved ? d >> 1 : (first ? d : d - half)];
            }
            c[v][j] = cs.x;
            g[v][j] = first != BACK ? -cs.y : cs.y;
        }
    }
    wave_lds_fence();
}

template <class T, int VEC, int G, int NV>
__device__ __forceinline__ void load_weight(float (&w)[NV][VEC], const void* p, int dim, int lane) {
    using V = typename Vec<T, VEC>::type;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int u = lane + v * G;
        if (p != nullptr && u * VEC < dim) {
            widen_vec<T, VEC>(static_cast<const V*>(p)[u], w[v]);
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) w[v][j] = 1.f;
        }
    }
}

// Address of row r (queries first, then keys) of token t.
template <class T>
__device__ __forceinline__ typename T::bits* row_of(const Heads& q, const Heads& k, int q_heads, int64_t t, int r) {
    const bool isq = r < q_heads;
    typename T::bits* p = static_cast<typename T::bits*>(isq ? q.p : k.p);
    return p + t * (isq ? q.ts : k.ts) + (isq ? r : r - q_heads) * (isq ? q.hs : k.hs);
}

template <class T, int VEC, int G, int NV>
__global__ __launch_bounds__(kQkNormWaves* kWave) void qk_norm_kernel(QkNorm a) {
    using V = typename Vec<T, VEC>::type;
    constexpr int R = kWave / G;  // rows at a time
    constexpr int U = NV == 1 ? 4 : 1;  // of which loads are in flight
    __shared__ __align__(16) float lds[kQkNormWaves][kWaveFloats];
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % G, group = (threadIdx.x % kWave) / G;
    const int64_t id = (int64_t)blockIdx.x * kQkNormWaves + wave;
    const int64_t t = id / a.parts;
    if (t >= a.tokens) return;
    const int part = (int)(id - t * a.parts), rows = a.q_heads + a.k_heads;
    const int passes = (rows + R - 1) / R, per = (passes + a.parts - 1) / a.parts;
    const int first = part * per, last = min(passes, first + per);
    float wq[NV][VEC], wk[NV][VEC], c[NV][VEC], g[NV][VEC];
    load_weight<T, VEC, G, NV>(wq, a.q_weight, a.dim, lane);
    load_weight<T, VEC, G, NV>(wk, a.k_weight, a.dim, lane);
    const int mode = turn_mode<VEC>(a.rot, a.interleaved);
    token_turns<VEC, G, NV, false>(c, g, a.pos[t], a.freq, a.rot, a.interleaved, lane,
                                   reinterpret_cast<float2*>(lds[wave]));
    float* row = lds[wave] + group * (G * VEC * NV);
    const float inv = 1.f / (float)a.dim;
    for (int p0 = first; p0 < last; p0 += U) {
        V x[U][NV];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = (p0 + u) * R + group;
            const V* src = reinterpret_cast<const V*>(row_of<T>(a.q, a.k, a.q_heads, t, r < rows ? r : 0));
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                x[u][v] = V{};
                if (p0 + u < last && r < rows && (lane + v * G) * VEC < a.dim) x[u][v] = src[lane + v * G];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (p0 + u >= last) break;
            const int r = (p0 + u) * R + group;
            float y[NV][VEC], sum = 0.f;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                widen_vec<T, VEC>(x[u][v], y[v]);
#pragma unroll
                for (int j = 0; j < VEC; ++j) sum += y[v][j] * y[v][j];
            }
            const float rn = rsqrtf(group_sum<G>(sum) * inv + a.eps);
            const bool isq = r < a.q_heads;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int j = 0; j < VEC; ++j) y[v][j] *= rn * (isq ? wq[v][j] : wk[v][j]);
            turn<VEC, G, NV>(y, c, g, mode, a.interleaved, lane, a.dim, a.rot, row);
            if (r < rows) {
                V* dst = reinterpret_cast<V*>(row_of<T>(a.q_out, a.k_out, a.q_heads, t, r));
#pragma unroll
                for (int v = 0; v < NV; ++v)
                    if ((lane + v * G) * VEC < a.dim) dst[lane + v * G] = narrow_vec<T, VEC>(y[v]);
            }
        }
    }
}

// The backward pass. Waves go through tokens with a stride, so that a lane can
// add up the weight gradients of its columns in registers; they are added over
// the wave's groups, then over the block's waves, and one row of 2 dim
// partials a block goes to memory (qk_norm_weights_kernel adds those).
template <class T, int VEC, int G, int NV>
__global__ __launch_bounds__(kQkNormWaves* kWave) void qk_norm_backward_kernel(QkNorm a) {
    using V = typename Vec<T, VEC>::type;
    constexpr int R = kWave / G;
    constexpr int U = NV == 1 ? 2 : 1;
    __shared__ __align__(16) float lds[kQkNormWaves][kWaveFloats];
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % G, group = (threadIdx.x % kWave) / G;
    const int rows = a.q_heads + a.k_heads;
    const int passes = (rows + R - 1) / R, per = (passes + a.parts - 1) / a.parts;
    float wq[NV][VEC], wk[NV][VEC], c[NV][VEC], g[NV][VEC], aq[NV][VEC], ak[NV][VEC];
    load_weight<T, VEC, G, NV>(wq, a.q_weight, a.dim, lane);
    load_weight<T, VEC, G, NV>(wk, a.k_weight, a.dim, lane);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < VEC; ++j) aq[v][j] = ak[v][j] = 0.f;
    const int mode = turn_mode<VEC>(a.rot, a.interleaved);
    float* row = lds[wave] + group * (G * VEC * NV);
    const float inv = 1.f / (float)a.dim;
    const int64_t items = a.tokens * a.parts;
    for (int64_t id = (int64_t)blockIdx.x * kQkNormWaves + wave; id < items; id += (int64_t)gridDim.x * kQkNormWaves) {
        const int64_t t = id / a.parts;
        const int part = (int)(id - t * a.parts);
        const int first = part * per, last = min(passes, first + per);
        token_turns<VEC, G, NV, true>(c, g, a.pos[t], a.freq, a.rot, a.interleaved, lane,
                                      reinterpret_cast<float2*>(lds[wave]));
        for (int p0 = first; p0 < last; p0 += U) {
            V x[U][NV], e[U][NV];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = (p0 + u) * R + group, rr = r < rows ? r : 0;
                const V* sx = reinterpret_cast<const V*>(row_of<T>(a.q, a.k, a.q_heads, t, rr));
                const V* se = reinterpret_cast<const V*>(row_of<T>(a.dq, a.dk, a.q_heads, t, rr));
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    x[u][v] = e[u][v] = V{};
                    if (p0 + u < last && r < rows && (lane + v * G) * VEC < a.dim) {
                        x[u][v] = sx[lane + v * G];
                        e[u][v] = se[lane + v * G];
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (p0 + u >= last) break;
                const int r = (p0 + u) * R + group;
                float f[NV][VEC], d[NV][VEC], xx = 0.f, hx = 0.f;
                const bool isq = r < a.q_heads;
#pragma unroll
                for (int v = 0; v < NV; ++v) widen_vec<T, VEC>(e[u][v], d[v]);
                turn<VEC, G, NV>(d, c, g, mode, a.interleaved, lane, a.dim, a.rot, row);
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    widen_vec<T, VEC>(x[u][v], f[v]);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        xx += f[v][j] * f[v][j];
                        hx += d[v][j] * (isq ? wq[v][j] : wk[v][j]) * f[v][j];
                    }
                }
                const float rn = rsqrtf(group_sum<G>(xx) * inv + a.eps);
                const float m = rn * rn * (group_sum<G>(hx) * inv);
                if (r < rows) {
                    V* dst = reinterpret_cast<V*>(row_of<T>(a.q_out, a.k_out, a.q_heads, t, r));
#pragma unroll
                    for (int v = 0; v < NV; ++v) {
                        float o[VEC];
#pragma unroll
                        for (int j = 0; j < VEC; ++j) {
                            o[j] = rn * (d[v][j] * (isq ? wq[v][j] : wk[v][j]) - f[v][j] * m);
                            const float dw = d[v][j] * f[v][j] * rn;
                            if (isq) aq[v][j] += dw;
                            else ak[v][j] += dw;
                        }
                        if ((lane + v * G) * VEC < a.dim) dst[lane + v * G] = narrow_vec<T, VEC>(o);
                    }
                }
            }
        }
    }
    // Partials: groups of the wave, then waves of the block, in a fixed order.
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                float s = which ? ak[v][j] : aq[v][j];
                for (int o = G; o < kWave; o <<= 1) s += __shfl_xor(s, o);
                const int col = (lane + v * G) * VEC + j;
                if (group == 0 && col < a.dim) lds[wave][col] = s;
            }
        __syncthreads();
        for (int col = threadIdx.x; col < a.dim; col += kQkNormWaves * kWave) {
            float s = 0.f;
            for (int w = 0; w < kQkNormWaves; ++w) s += lds[w][col];
            a.partials[((size_t)blockIdx.x * 2 + which) * a.dim + col] = s;
        }
    }
}

template <class T, int VEC, int G, int NV>
hipError_t launch_qk_norm_shape(const QkNorm& a, bool back, int blocks, hipStream_t stream) {
    if (back)
        qk_norm_backward_kernel<T, VEC, G, NV><<<blocks, kQkNormWaves * kWave, 0, stream>>>(a);
    else
        qk_norm_kernel<T, VEC, G, NV><<<blocks, kQkNormWaves * kWave, 0, stream>>>(a);
    return hipGetLastError();
}

template <class T, int VEC>
hipError_t launch_qk_norm_vec(int lanes, const QkNorm& a, bool back, int blocks, hipStream_t stream) {
    switch (lanes) {
        case 4: return launch_qk_norm_shape<T, VEC, 4, 1>(a, back, blocks, stream);
        case 8: return launch_qk_norm_shape<T, VEC, 8, 1>(a, back, blocks, stream);
        case 16: return launch_qk_norm_shape<T, VEC, 16, 1>(a, back, blocks, stream);
        case 32: return launch_qk_norm_shape<T, VEC, 32, 1>(a, back, blocks, stream);
        case 64: return launch_qk_norm_shape<T, VEC, 64, 1>(a, back, blocks, stream);
        default: return hipErrorInvalidValue;
    }
}

template <class T>
hipError_t launch_qk_norm_type(int vec, int lanes, const QkNorm& a, bool back, int blocks, hipStream_t stream) {
    if (vec == 1) return launch_qk_norm_shape<T, 1, 64, 4>(a, back, blocks, stream);
    if (vec == 4) return launch_qk_norm_vec<T, 4>(lanes, a, back, blocks, stream);
    if constexpr (sizeof(typename T::bits) == 2)
        if (vec == 8) return launch_qk_norm_vec<T, 8>(lanes, a, back, blocks, stream);
    return hipErrorInvalidValue;
}

}  // namespace libred
