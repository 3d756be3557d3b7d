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

// Cosines and signed sines of this lane's columns for token t. BACK: the
// rotation the other way.
template <int VEC, int G, int NV, bool BACK>
__device__ __forceinline__ void token_turns(float (&c)[NV][VEC], float (&g)[NV][VEC], const int64_t* pos, int64_t t,
                                            const float* freq, int rot, int interleaved, int lane, float2* table) {
    if (rot == 0) return;
    const int half = rot / 2;
    const int64_t p = pos[t];
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

// A token's rows are taken in passes of R heads, those of q first; a pass is of
// q or of k, so that which weight to use is the same for the whole wave.
template <class T, int R>
struct Passes {
    const QkNorm& a;
    int64_t t;
    int group;
    __device__ int of_q() const { return (a.q_heads + R - 1) / R; }
    __device__ int all() const { return of_q() + (a.k_heads + R - 1) / R; }
    __device__ bool is_q(int p) const { return p < of_q(); }
    __device__ int head(int p) const { return (is_q(p) ? p : p - of_q()) * R + group; }
    __device__ bool there(int p) const { return head(p) < (is_q(p) ? a.q_heads : a.k_heads); }
    // Row of this group in pass p, in the tensors of q or k.
    __device__ typename T::bits* row(int p, const Heads& q, const Heads& k) const {
        const Heads& h = is_q(p) ? q : k;
        return static_cast<typename T::bits*>(h.p) + t * h.ts + (there(p) ? head(p) : 0) * h.hs;
    }
};

// Loads are made without a branch (around one the compiler would not know how
// many are on their way, and would wait for all of them at each use): lanes
// beyond the row read its first elements, and keep() drops them.
template <class T, int VEC, int G, int NV>
__device__ __forceinline__ void load_row(typename Vec<T, VEC>::type (&x)[NV], const typename T::bits* p, int dim, int lane) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int u = lane + v * G;
        x[v] = reinterpret_cast<const typename Vec<T, VEC>::type*>(p)[u * VEC < dim ? u : 0];
    }
}
template <int VEC, int G, int NV>
__device__ __forceinline__ void keep(float (&f)[NV][VEC], bool there, int dim, int lane) {
    if (__all(there) && dim == G * VEC * NV) return;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < VEC; ++j) f[v][j] = there && (lane + v * G) * VEC < dim ? f[v][j] : 0.f;
}
template <class T, int VEC, int G, int NV>
__device__ __forceinline__ void store_row(typename T::bits* p, const float (&y)[NV][VEC], bool there, int dim, int lane) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
        if (there && (lane + v * G) * VEC < dim)
            reinterpret_cast<typename Vec<T, VEC>::type*>(p)[lane + v * G] = narrow_vec<T, VEC>(y[v]);
}

template <class T, int VEC, int G, int NV>
__global__ __launch_bounds__(kQkNormWaves* kWave) void qk_norm_kernel(QkNorm a) {
    using V = typename Vec<T, VEC>::type;
    constexpr int R = kWave / G;        // rows at a time
    constexpr int U = NV == 1 ? 4 : 1;  // passes whose loads are in flight
    __shared__ __align__(16) float lds[kQkNormWaves][kWaveFloats];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % G;
    const int group = (threadIdx.x % kWave) / G;
    const int64_t id = (int64_t)blockIdx.x * kQkNormWaves + wave;
    const int64_t t = a.parts == 1 ? id : id / a.parts;
    if (t >= a.tokens) return;
    const Passes<T, R> rows = {a, t, group};
    const int part = (int)(id - t * a.parts), per = (rows.all() + a.parts - 1) / a.parts;
    const int first = part * per, last = min(rows.all(), first + per);
    V x[U][NV];
    auto load = [&](int p0) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            load_row<T, VEC, G, NV>(x[u], rows.row(min(p0 + u, last - 1), a.q, a.k), a.dim, lane);
    };
    if (first >= last) return;
    load(first);  // before the angles, which take as long
    float wq[NV][VEC], wk[NV][VEC], c[NV][VEC], g[NV][VEC];
    load_weight<T, VEC, G, NV>(wq, a.q_weight, a.dim, lane);
    load_weight<T, VEC, G, NV>(wk, a.k_weight, a.dim, lane);
    const int mode = turn_mode<VEC>(a.rot, a.interleaved);
    token_turns<VEC, G, NV, false>(c, g, a.pos, t, a.freq, a.rot, a.interleaved, lane, reinterpret_cast<float2*>(lds[wave]));
    float* row = lds[wave] + group * (G * VEC * NV);
    const float inv = 1.f / (float)a.dim;
    auto norm = [&](const V(&in)[NV], const float(&w)[NV][VEC], int p) {
        float y[NV][VEC], sum = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) widen_vec<T, VEC>(in[v], y[v]);
        keep<VEC, G, NV>(y, rows.there(p), a.dim, lane);
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < VEC; ++j) sum += y[v][j] * y[v][j];
        const float rn = rsqrtf(group_sum<G>(sum) * inv + a.eps);
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < VEC; ++j) y[v][j] *= rn * w[v][j];
        turn<VEC, G, NV>(y, c, g, mode, a.interleaved, lane, a.dim, a.rot, row);
        store_row<T, VEC, G, NV>(rows.row(p, a.q_out, a.k_out), y, rows.there(p), a.dim, lane);
    };
    for (int p0 = first; p0 < last; p0 += U) {
        if (p0 > first) load(p0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (p0 + u >= last) break;
            if (rows.is_q(p0 + u)) norm(x[u], wq, p0 + u);
            else norm(x[u], wk, p0 + u);
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
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % G;
    const int group = (threadIdx.x % kWave) / G;
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
        const int64_t t = a.parts == 1 ? id : id / a.parts;
        const Passes<T, R> rows = {a, t, group};
        const int part = (int)(id - t * a.parts), per = (rows.all() + a.parts - 1) / a.parts;
        const int first = part * per, last = min(rows.all(), first + per);
        V x[2][U][NV], e[2][U][NV];  // the rows at hand, and those on their way
        auto load = [&](int p0, V(&x)[U][NV], V(&e)[U][NV]) {
#pragma unroll
            for (int u = 0; u < U; ++u)
            {
                const int p = min(p0 + u, last - 1);
                load_row<T, VEC, G, NV>(x[u], rows.row(p, a.q, a.k), a.dim, lane);
                load_row<T, VEC, G, NV>(e[u], rows.row(p, a.dq, a.dk), a.dim, lane);
            }
        };
        if (first >= last) continue;
        load(first, x[0], e[0]);
        token_turns<VEC, G, NV, true>(c, g, a.pos, t, a.freq, a.rot, a.interleaved, lane, reinterpret_cast<float2*>(lds[wave]));
        auto back = [&](const V(&in)[NV], const V(&dy)[NV], const float(&w)[NV][VEC], float(&dw)[NV][VEC], int p) {
            float f[NV][VEC], d[NV][VEC], o[NV][VEC], xx = 0.f, hx = 0.f;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                widen_vec<T, VEC>(dy[v], d[v]);
                widen_vec<T, VEC>(in[v], f[v]);
            }
            const bool there = rows.there(p);
            keep<VEC, G, NV>(d, there, a.dim, lane);
            keep<VEC, G, NV>(f, there, a.dim, lane);
            turn<VEC, G, NV>(d, c, g, mode, a.interleaved, lane, a.dim, a.rot, row);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    xx += f[v][j] * f[v][j];
                    o[v][j] = d[v][j] * w[v][j];
                    hx += o[v][j] * f[v][j];
                }
            }
            const float rn = rsqrtf(group_sum<G>(xx) * inv + a.eps);
            const float m = rn * rn * (group_sum<G>(hx) * inv);
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    o[v][j] = rn * (o[v][j] - f[v][j] * m);
                    // A row that is not there is zeros, but eps may be 0.
                    dw[v][j] += there ? d[v][j] * (f[v][j] * rn) : 0.f;
                }
            store_row<T, VEC, G, NV>(rows.row(p, a.q_out, a.k_out), o, there, a.dim, lane);
        };
        auto some = [&](int p0, const V(&x)[U][NV], const V(&e)[U][NV]) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (p0 + u >= last) break;
                if (rows.is_q(p0 + u)) back(x[u], e[u], wq, aq, p0 + u);
                else back(x[u], e[u], wk, ak, p0 + u);
            }
        };
        for (int p0 = first; p0 < last; p0 += 2 * U) {
            load(p0 + U, x[1], e[1]);
            some(p0, x[0], e[0]);
            load(p0 + 2 * U, x[0], e[0]);
            some(p0 + U, x[1], e[1]);
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
