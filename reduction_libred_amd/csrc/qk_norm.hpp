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
//
// Memory bounds both passes. 16384 tokens of 32 + 8 heads of 128 in bf16:
// forward 336 MB in 62.1 us (5.4 TB/s; a copy of that size reaches 6.15),
// backward 503 MB in 91.7 us (5.5 TB/s) and 4.8 us for the sum of the weights'
// partials. 12 tokens take 4.4 us, one trip to memory after another.
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

// How the two elements of a pair meet: in a lane's own vector (neighbours as
// pairs), as whole vectors of two lanes (halves, at vector boundaries), or
// element by element (anything, nothing turned included). The kernels are
// built for each: chosen at run time, the branches alone doubled their
// instructions.
enum { kTurnInside = 0, kTurnVectors = 1, kTurnElements = 2 };

inline int turn_mode(int vec, int rot, int interleaved) {
    if (vec == 1 || rot == 0 || rot % vec != 0) return kTurnElements;
    return interleaved ? kTurnInside : rot / 2 % vec == 0 ? kTurnVectors : kTurnElements;
}

template <class T, int VEC>
using RowVec = typename Vec<T, VEC>::type;

// The element that shares a pair with element d.
__device__ __forceinline__ int partner_of(int d, int rot, int interleaved) {
    if (d >= rot) return d;
    const int half = rot / 2;
    return interleaved ? d ^ 1 : (d < half ? d + half : d - half);
}

// The partners of this lane's elements, through the wave's LDS as they are;
// `row` is the row's part of it (rot elements). 0 where nothing turns.
template <class T, int VEC, int G, int NV, int MODE>
__device__ __forceinline__ void partners(float (&f)[NV][VEC], const RowVec<T, VEC> (&x)[NV], int interleaved, int lane,
                                         int rot, typename T::bits* row) {
    using V = RowVec<T, VEC>;
    if constexpr (MODE == kTurnInside) {
        float y[VEC];
        widen_vec<T, VEC>(x[0], y);
        const bool turns = lane * VEC < rot;
#pragma unroll
        for (int j = 0; j < VEC; ++j) f[0][j] = turns ? y[j ^ 1] : 0.f;
    } else {
        wave_lds_fence();
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int u = lane + v * G;
            if (u * VEC < rot) reinterpret_cast<V*>(row)[u] = x[v];
        }
        wave_lds_fence();
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int d = (lane + v * G) * VEC;
            if constexpr (MODE == kTurnVectors) {
                V y = V{};
                if (d < rot) y = *reinterpret_cast<const V*>(row + (d < rot / 2 ? d + rot / 2 : d - rot / 2));
                widen_vec<T, VEC>(y, f[v]);
            } else {
#pragma unroll
                for (int j = 0; j < VEC; ++j) f[v][j] = d + j < rot ? T::widen(row[partner_of(d + j, rot, interleaved)]) : 0.f;
            }
        }
    }
}

// The angles of token t as cosines and sines in the wave's LDS.
__device__ __forceinline__ void token_angles(const int64_t* pos, int64_t t, const float* freq, int rot, float* cosines,
                                             float* sines) {
    if (rot == 0) return;
    const int64_t p = pos[t];
    wave_lds_fence();
    for (int i = threadIdx.x % kWave; i < rot / 2; i += kWave) {
        const double a = (double)p * (double)freq[i] * 0.15915494309189533577;  // turns
        const float2 cs = cos_sin_turns(a - rint(a));
        cosines[i] = cs.x;
        sines[i] = cs.y;
    }
    wave_lds_fence();
}

// Cosines and signed sines of this lane's columns: (x, partner) -> x c +
// partner g; c = 1, g = 0 beyond the rotated part. BACK: the rotation the
// other way.
template <int VEC, int G, int NV, int MODE, bool BACK>
__device__ __forceinline__ void lane_turns(float (&c)[NV][VEC], float (&g)[NV][VEC], int rot, int interleaved, int lane,
                                           const float* cosines, const float* sines) {
    const int half = rot / 2;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int d = (lane + v * G) * VEC;
        if constexpr (MODE == kTurnVectors) {
            const bool turns = d < rot, first = d < half;
            const int i = turns ? (first ? d : d - half) : 0;
#pragma unroll
            for (int j = 0; j < VEC; j += 4) {
                const f32x4 cs = *reinterpret_cast<const f32x4*>(cosines + i + j), sn = *reinterpret_cast<const f32x4*>(sines + i + j);
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    c[v][j + y] = turns ? cs[y] : 1.f;
                    g[v][j + y] = turns ? (first != BACK ? -sn[y] : sn[y]) : 0.f;
                }
            }
        } else if constexpr (MODE == kTurnInside) {
            const bool turns = d < rot;
#pragma unroll
            for (int j = 0; j < VEC; j += 2) {
                const float cs = cosines[turns ? (d + j) / 2 : 0], sn = sines[turns ? (d + j) / 2 : 0];
                c[v][j] = c[v][j + 1] = turns ? cs : 1.f;
                g[v][j] = turns ? (BACK ? sn : -sn) : 0.f;
                g[v][j + 1] = -g[v][j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const int e = d + j;
                const bool turns = e < rot, first = interleaved ? !(e & 1) : e < half;
                const int i = interleaved ? e >> 1 : (first ? e : e - half);
                c[v][j] = turns ? cosines[i] : 1.f;
                g[v][j] = turns ? (first != BACK ? -sines[i] : sines[i]) : 0.f;
            }
        }
    }
    wave_lds_fence();
}

// A weight at this lane's columns, or at their partners (0 where nothing turns:
// there the partner has no part in the result, whatever its weight is).
template <class T, int VEC, int G, int NV>
__device__ __forceinline__ void load_weight(float (&w)[NV][VEC], const void* p, int dim, int lane) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int u = lane + v * G;
        if (p != nullptr) {
            widen_vec<T, VEC>(static_cast<const RowVec<T, VEC>*>(p)[u * VEC < dim ? u : 0], w[v]);
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) w[v][j] = 1.f;
        }
    }
}
template <class T, int VEC, int G, int NV, int MODE>
__device__ __forceinline__ void load_partner_weight(float (&w)[NV][VEC], const float (&own)[NV][VEC], const void* p, int rot,
                                                    int interleaved, int lane) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int d = (lane + v * G) * VEC;
        if constexpr (MODE == kTurnInside) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) w[v][j] = d < rot ? own[v][j ^ 1] : 0.f;
        } else if (p == nullptr) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) w[v][j] = d + j < rot ? 1.f : 0.f;
        } else if constexpr (MODE == kTurnVectors) {
            const int o = d < rot ? (d < rot / 2 ? d + rot / 2 : d - rot / 2) : 0;
            widen_vec<T, VEC>(*reinterpret_cast<const RowVec<T, VEC>*>(static_cast<const typename T::bits*>(p) + o), w[v]);
#pragma unroll
            for (int j = 0; j < VEC; ++j) w[v][j] = d < rot ? w[v][j] : 0.f;
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                w[v][j] = d + j < rot ? T::widen(static_cast<const typename T::bits*>(p)[partner_of(d + j, rot, interleaved)]) : 0.f;
        }
    }
}

// A token's rows are taken in passes of R heads, those of q first; a pass is of
// q or of k, so that which weight to use is the same for the whole wave. A row
// is found as an address that is the wave's and an offset below 4 GiB that is
// the lane's (the entry point sees to that), which costs one instruction.
template <class T, int R, int VEC>
struct Passes {
    const QkNorm& a;
    int group, lane;
    __device__ int of_q() const { return (a.q_heads + R - 1) / R; }
    __device__ int all() const { return of_q() + (a.k_heads + R - 1) / R; }
    __device__ bool is_q(int p) const { return p < of_q(); }
    __device__ int head0(int p) const { return (is_q(p) ? p : p - of_q()) * R; }
    __device__ bool there(int p) const { return head0(p) + group < (is_q(p) ? a.q_heads : a.k_heads); }
    // Of this lane's group in a tensor of heads, in bytes.
    __device__ uint32_t offset(const Heads& h) const { return (uint32_t)group * (uint32_t)h.hs * (uint32_t)sizeof(typename T::bits); }
    __device__ char* base(int p, int64_t t, const Heads& h) const {
        return static_cast<char*>(h.p) + (t * h.ts + head0(p) * h.hs) * (int64_t)sizeof(typename T::bits);
    }
};

// Loads are made without a branch (around one the compiler would not know how
// many are on their way, and would wait for all of them at each use): lanes
// beyond the row read its first elements, and keep() drops them.
template <class T, int VEC, int G, int NV>
__device__ __forceinline__ void load_row(RowVec<T, VEC> (&x)[NV], const char* base, uint32_t offset, int dim, int lane) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int u = lane + v * G;
        x[v] = load_vec<true>(reinterpret_cast<const RowVec<T, VEC>*>(base + (uint32_t)(offset + (u * VEC < dim ? u : 0) * (uint32_t)sizeof(RowVec<T, VEC>))));
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
__device__ __forceinline__ void store_row(char* base, uint32_t offset, const float (&y)[NV][VEC], bool there, int dim,
                                          int lane) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int u = lane + v * G;
        if (there && u * VEC < dim)
            store_vec<false>(reinterpret_cast<RowVec<T, VEC>*>(base + (uint32_t)(offset + u * (uint32_t)sizeof(RowVec<T, VEC>))), narrow_vec<T, VEC>(y[v]));
    }
}

// One argument of every 64-byte line, so that all lines are asked for at once.
__device__ __forceinline__ void ask_for_arguments(const QkNorm& a) {
    asm volatile("" ::"s"(a.q.p), "s"(a.k_out.p), "s"(a.q_weight), "s"(a.tokens));
}

// With the weight folded into cosine and sine, an element of the result is
//     r (x (w c) + partner (w_partner g)),
// so the exchange of partners does not wait for the row's sum.
template <class T, int VEC, int G, int NV, int MODE>
__global__ __launch_bounds__(kQkNormWaves* kWave) void qk_norm_kernel(QkNorm a) {
    using V = RowVec<T, VEC>;
    constexpr int R = kWave / G;        // rows at a time
    constexpr int U = NV == 1 ? 5 : 1;  // passes whose loads are in flight
    __shared__ __align__(16) float lds[kQkNormWaves][kWaveFloats];
    ask_for_arguments(a);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % G;
    const int group = (threadIdx.x % kWave) / G;
    const int64_t id = (int64_t)blockIdx.x * kQkNormWaves + wave;
    const int64_t t = a.parts == 1 ? id : (uint32_t)id / (uint32_t)a.parts;
    if (t >= a.tokens) return;
    const Passes<T, R, VEC> rows = {a, group, lane};
    const int part = (int)(id - t * a.parts), per = (rows.all() + a.parts - 1) / a.parts;
    const int first = part * per, last = min(rows.all(), first + per);
    if (first >= last) return;
    const uint32_t in_q = rows.offset(a.q), in_k = rows.offset(a.k), out_q = rows.offset(a.q_out), out_k = rows.offset(a.k_out);
    V x[U][NV];
    auto load = [&](int p0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int p = min(p0 + u, last - 1);
            const bool q = rows.is_q(p);
            load_row<T, VEC, G, NV>(x[u], rows.base(p, t, q ? a.q : a.k), rows.there(p) ? (q ? in_q : in_k) : 0, a.dim, lane);
        }
    };
    load(first);  // before the angles, which take as long
    float aq[NV][VEC], bq[NV][VEC], ak[NV][VEC], bk[NV][VEC];
    {
        float c[NV][VEC], g[NV][VEC];
        load_weight<T, VEC, G, NV>(aq, a.q_weight, a.dim, lane);
        load_weight<T, VEC, G, NV>(ak, a.k_weight, a.dim, lane);
        load_partner_weight<T, VEC, G, NV, MODE>(bq, aq, a.q_weight, a.rot, a.interleaved, lane);
        load_partner_weight<T, VEC, G, NV, MODE>(bk, ak, a.k_weight, a.rot, a.interleaved, lane);
        token_angles(a.pos, t, a.freq, a.rot, lds[wave], lds[wave] + kHeadMax / 2);
        lane_turns<VEC, G, NV, MODE, false>(c, g, a.rot, a.interleaved, lane, lds[wave], lds[wave] + kHeadMax / 2);
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                aq[v][j] *= c[v][j], ak[v][j] *= c[v][j];
                bq[v][j] *= g[v][j], bk[v][j] *= g[v][j];
            }
    }
    typename T::bits* row = reinterpret_cast<typename T::bits*>(lds[wave]) + group * (G * VEC * NV);
    const float inv = 1.f / (float)a.dim;
    auto norm = [&](const V(&in)[NV], const float(&wc)[NV][VEC], const float(&wg)[NV][VEC], int p, const Heads& to, uint32_t at) {
        float y[NV][VEC], o[NV][VEC], sum = 0.f;
        partners<T, VEC, G, NV, MODE>(o, in, a.interleaved, lane, a.rot, row);
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
            for (int j = 0; j < VEC; ++j) y[v][j] = rn * (y[v][j] * wc[v][j] + o[v][j] * wg[v][j]);
        store_row<T, VEC, G, NV>(rows.base(p, t, to), at, y, rows.there(p), a.dim, lane);
    };
    for (int p0 = first; p0 < last; p0 += U) {
        if (p0 > first) load(p0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (p0 + u >= last) break;
            if (rows.is_q(p0 + u)) norm(x[u], aq, bq, p0 + u, a.q_out, out_q);
            else norm(x[u], ak, bk, p0 + u, a.k_out, out_k);
        }
    }
}

// The backward pass. Waves go through tokens with a stride, so that a lane can
// add up the weight gradients of its columns in registers; they are added over
// the wave's groups, then over the block's waves, and one row of 2 dim
// partials a block goes to memory (qk_norm_weights_kernel adds those).
template <class T, int VEC, int G, int NV, int MODE>
__global__ __launch_bounds__(kQkNormWaves* kWave) void qk_norm_backward_kernel(QkNorm a) {
    using V = RowVec<T, VEC>;
    constexpr int R = kWave / G;
    constexpr int U = NV == 1 ? 2 : 1;
    __shared__ __align__(16) float lds[kQkNormWaves][kWaveFloats];
    ask_for_arguments(a);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % G;
    const int group = (threadIdx.x % kWave) / G;
    float wq[NV][VEC], wk[NV][VEC], c[NV][VEC], g[NV][VEC], aq[NV][VEC], ak[NV][VEC];
    load_weight<T, VEC, G, NV>(wq, a.q_weight, a.dim, lane);
    load_weight<T, VEC, G, NV>(wk, a.k_weight, a.dim, lane);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < VEC; ++j) aq[v][j] = ak[v][j] = 0.f;
    typename T::bits* row = reinterpret_cast<typename T::bits*>(lds[wave]) + group * (G * VEC * NV);
    const float inv = 1.f / (float)a.dim;
    const Passes<T, R, VEC> rows = {a, group, lane};
    const uint32_t x_q = rows.offset(a.q), x_k = rows.offset(a.k), d_q = rows.offset(a.dq), d_k = rows.offset(a.dk);
    const uint32_t out_q = rows.offset(a.q_out), out_k = rows.offset(a.k_out);
    const int64_t items = a.tokens * a.parts;
    for (int64_t id = (int64_t)blockIdx.x * kQkNormWaves + wave; id < items; id += (int64_t)gridDim.x * kQkNormWaves) {
        const int64_t t = a.parts == 1 ? id : (uint32_t)id / (uint32_t)a.parts;
        const int part = (int)(id - t * a.parts), per = (rows.all() + a.parts - 1) / a.parts;
        const int first = part * per, last = min(rows.all(), first + per);
        if (first >= last) continue;
        V x[2][U][NV], e[2][U][NV];  // the rows at hand, and those on their way
        auto load = [&](int p0, V(&x)[U][NV], V(&e)[U][NV]) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // Past the last pass, the first rows of all: those are in the
                // caches. (This token's last rows again, past their use: a
                // fifth more bytes from memory, 97 us / 91.)
                const bool over = p0 + u >= last;
                const int p = over ? 0 : p0 + u;
                const int64_t of = over ? 0 : t;
                const bool q = rows.is_q(p), there = rows.there(p);
                load_row<T, VEC, G, NV>(x[u], rows.base(p, of, q ? a.q : a.k), there ? (q ? x_q : x_k) : 0, a.dim, lane);
                load_row<T, VEC, G, NV>(e[u], rows.base(p, of, q ? a.dq : a.dk), there ? (q ? d_q : d_k) : 0, a.dim, lane);
            }
        };
        load(first, x[0], e[0]);
        token_angles(a.pos, t, a.freq, a.rot, lds[wave], lds[wave] + kHeadMax / 2);
        lane_turns<VEC, G, NV, MODE, true>(c, g, a.rot, a.interleaved, lane, lds[wave], lds[wave] + kHeadMax / 2);
        auto back = [&](const V(&in)[NV], const V(&dy)[NV], const float(&w)[NV][VEC], float(&dw)[NV][VEC], int p, const Heads& to, uint32_t at) {
            float f[NV][VEC], d[NV][VEC], o[NV][VEC], xx = 0.f, hx = 0.f;
            partners<T, VEC, G, NV, MODE>(o, dy, a.interleaved, lane, a.rot, row);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                widen_vec<T, VEC>(dy[v], d[v]);
                widen_vec<T, VEC>(in[v], f[v]);
#pragma unroll
                for (int j = 0; j < VEC; ++j) d[v][j] = d[v][j] * c[v][j] + o[v][j] * g[v][j];
            }
            const bool there = rows.there(p);
            keep<VEC, G, NV>(d, there, a.dim, lane);
            keep<VEC, G, NV>(f, there, a.dim, lane);
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    xx += f[v][j] * f[v][j];
                    o[v][j] = d[v][j] * w[v][j];
                    hx += o[v][j] * f[v][j];
                }
            // The root of a row that is not there may be infinite.
            const float rn = there ? rsqrtf(group_sum<G>(xx) * inv + a.eps) : 0.f;
            const float m = rn * rn * (group_sum<G>(hx) * inv);
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    o[v][j] = rn * (o[v][j] - f[v][j] * m);
                    dw[v][j] += d[v][j] * (f[v][j] * rn);
                }
            store_row<T, VEC, G, NV>(rows.base(p, t, to), at, o, there, a.dim, lane);
        };
        auto some = [&](int p0, const V(&x)[U][NV], const V(&e)[U][NV]) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (p0 + u >= last) break;
                if (rows.is_q(p0 + u)) back(x[u], e[u], wq, aq, p0 + u, a.q_out, out_q);
                else back(x[u], e[u], wk, ak, p0 + u, a.k_out, out_k);
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

template <class T, int VEC, int G, int NV, int MODE>
hipError_t launch_qk_norm_mode(const QkNorm& a, bool back, int blocks, hipStream_t stream) {
    if (back)
        qk_norm_backward_kernel<T, VEC, G, NV, MODE><<<blocks, kQkNormWaves * kWave, 0, stream>>>(a);
    else
        qk_norm_kernel<T, VEC, G, NV, MODE><<<blocks, kQkNormWaves * kWave, 0, stream>>>(a);
    return hipGetLastError();
}

template <class T, int VEC, int G>
hipError_t launch_qk_norm_lanes(const QkNorm& a, bool back, int blocks, hipStream_t stream) {
    switch (turn_mode(VEC, a.rot, a.interleaved)) {
        case kTurnInside: return launch_qk_norm_mode<T, VEC, G, 1, kTurnInside>(a, back, blocks, stream);
        case kTurnVectors: return launch_qk_norm_mode<T, VEC, G, 1, kTurnVectors>(a, back, blocks, stream);
        default: return launch_qk_norm_mode<T, VEC, G, 1, kTurnElements>(a, back, blocks, stream);
    }
}

template <class T, int VEC>
hipError_t launch_qk_norm_vec(int lanes, const QkNorm& a, bool back, int blocks, hipStream_t stream) {
    switch (lanes) {
        case 4: return launch_qk_norm_lanes<T, VEC, 4>(a, back, blocks, stream);
        case 8: return launch_qk_norm_lanes<T, VEC, 8>(a, back, blocks, stream);
        case 16: return launch_qk_norm_lanes<T, VEC, 16>(a, back, blocks, stream);
        case 32: return launch_qk_norm_lanes<T, VEC, 32>(a, back, blocks, stream);
        case 64: return launch_qk_norm_lanes<T, VEC, 64>(a, back, blocks, stream);
        default: return hipErrorInvalidValue;
    }
}

template <class T>
hipError_t launch_qk_norm_type(int vec, int lanes, const QkNorm& a, bool back, int blocks, hipStream_t stream) {
    if (vec == 1) return launch_qk_norm_mode<T, 1, 64, 4, kTurnElements>(a, back, blocks, stream);
    if (vec == 4) return launch_qk_norm_vec<T, 4>(lanes, a, back, blocks, stream);
    if constexpr (sizeof(typename T::bits) == 2)
        if (vec == 8) return launch_qk_norm_vec<T, 8>(lanes, a, back, blocks, stream);
    return hipErrorInvalidValue;
}

}  // namespace libred
