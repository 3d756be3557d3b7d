// Verification of drafted tokens, and the token sampled after them.
//
// Draft i is accepted while u_i q_i(d_i) < p_i(d_i); n is the number accepted
// before the first that is not. The next token is drawn from
//     w = max(p_n - q_n, 0)  where a draft was refused (p_n if that is 0 everywhere),
//     w = p_n                where all were accepted:
// the first token whose running sum of w passes r sum(w).
//
// Only row n of p and q is read as a whole: once for the sum, by `segs` blocks
// a sequence (each finds n for itself, from at most two gathers a draft), and
// once more in the one segment where the running sum passes its border, by a
// second launch. Sums run in float64: float32 inputs differ exactly there, and
// a border is then missed by less than 2^-40 of the sum whatever the order.
#include "decode_common.hpp"

namespace libred {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

struct AddF64 {
    __device__ double operator()(double a, double b) const { return a + b; }
};

template <class T>
struct Verifier {
    using B = typename T::bits;
    static constexpr int kVec = 16 / sizeof(B);
    // Rows start on element boundaries only (a vocabulary may be odd).
    typedef B Vector __attribute__((ext_vector_type(16 / sizeof(B)), aligned(sizeof(B))));

    const Verify& a;
    int b, count;
    __device__ Verifier(const Verify& v, int seq) : a(v), b(seq) {
        count = v.count ? min(max(v.count[seq], 0), v.drafts) : v.drafts;
    }
    __device__ const B* row_p(int i) const { return static_cast<const B*>(a.p) + b * a.p_batch + i * a.p_step; }
    __device__ const B* row_q(int i) const { return static_cast<const B*>(a.q) + b * a.q_batch + i * a.q_step; }
    __device__ int64_t drafted(int i) const { return a.drafted[(int64_t)b * a.drafts + i]; }

    // Number of accepted drafts; the same in every lane of the wave. A draft
    // outside the vocabulary is refused.
    __device__ int accepted() const {
        for (int i0 = 0; i0 < count; i0 += kWave) {
            const int i = i0 + threadIdx.x % kWave;
            bool good = false;
            if (i < count) {
                const int64_t d = drafted(i);
                if (d >= 0 && d < a.vocab) {
                    const double p = (double)T::widen(row_p(i)[d]);
                    const double q = a.q ? (double)T::widen(row_q(i)[d]) : 1.0;
                    good = (double)a.u[(int64_t)b * a.drafts + i] * q < p;
                }
            }
            const uint64_t refused = ~__ballot(good);
            const int n = refused ? __ffsll((unsigned long long)refused) - 1 : kWave;
            if (n < kWave) return min(i0 + n, count);
        }
        return count;
    }
};

// What a row's weights are made of.
enum { kAll = 0, kLessRow = 1, kLessToken = 2 };

template <class T>
__device__ __forceinline__ double weight(float p, float q, int kind, bool token) {
    double w = (double)p;
    if (kind == kLessRow) w -= (double)q;
    if (kind == kLessToken && token) w -= 1.0;
    return w < 0.0 ? 0.0 : w;  // a NaN stays one
}

// Sum over the block in a fixed order; every thread gets it.
__device__ __forceinline__ double block_sum(double v, double* lds) {
    v = group_combine<kWave>(v, AddF64());
    __syncthreads();
    if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = v;
    __syncthreads();
    double s = lds[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) s += lds[w];
    return s;
}

template <class T>
__global__ __launch_bounds__(kThreads) void verify_sum_kernel(Verify a) {
    using V = Verifier<T>;
    constexpr int N = V::kVec;
    __shared__ double lds[kWaves];
    const V v(a, blockIdx.y);
    const int n = v.accepted();
    if (blockIdx.x == 0 && threadIdx.x == 0) a.accepted[v.b] = n;
    const int kind = n == v.count ? kAll : a.q ? kLessRow : kLessToken;
    const int64_t token = kind == kLessToken ? v.drafted(n) : -1;
    const typename V::B *p = v.row_p(n), *q = kind == kLessRow ? v.row_q(n) : p;
    const int64_t first = (int64_t)blockIdx.x * a.seg, last = min(first + a.seg, a.vocab);
    double sum = 0.0;
    int64_t i = first + threadIdx.x * N;
    for (; i + N <= last; i += kThreads * N) {
        const typename V::Vector x = *reinterpret_cast<const typename V::Vector*>(p + i);
        typename V::Vector y = x;
        if (kind == kLessRow) y = *reinterpret_cast<const typename V::Vector*>(q + i);
#pragma unroll
        for (int j = 0; j < N; ++j) sum += weight<T>(T::widen(x[j]), T::widen(y[j]), kind, i + j == token);
    }
    for (; i < last; ++i) {  // of one thread: the end of the segment
        sum += weight<T>(T::widen(p[i]), T::widen(q[i]), kind, i == token);
    }
    sum = block_sum(sum, lds);
    if (threadIdx.x == 0) a.sums[(int64_t)v.b * a.segs + blockIdx.x] = sum;
}

// Running sum over the threads of the block, this thread's value included.
__device__ __forceinline__ double block_scan(double v, double* lds) {
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    for (int o = 1; o < kWave; o <<= 1) {
        const double x = __shfl_up(v, o);
        if (lane >= o) v += x;
    }
    __syncthreads();
    if (lane == kWave - 1) lds[wave] = v;
    __syncthreads();
    double before = 0.0;
    for (int w = 0; w < wave; ++w) before += lds[w];
    return before + v;
}

__device__ __forceinline__ int64_t block_min(int64_t v, int64_t* lds) {
    for (int o = 1; o < kWave; o <<= 1) v = min(v, (int64_t)__shfl_xor((long long)v, o));
    __syncthreads();
    if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = v;
    __syncthreads();
    v = lds[0];
    for (int w = 1; w < kWaves; ++w) v = min(v, lds[w]);
    return v;
}

template <class T>
__global__ __launch_bounds__(kThreads) void verify_pick_kernel(Verify a) {
    using V = Verifier<T>;
    __shared__ double lds[kWaves];
    __shared__ int64_t ids[kWaves];
    __shared__ double before_seg;
    const V v(a, blockIdx.x);
    const int n = a.accepted[v.b], tid = threadIdx.x;
    int kind = n == v.count ? kAll : a.q ? kLessRow : kLessToken;
    const int64_t token = kind == kLessToken ? v.drafted(n) : -1;
    const typename V::B *p = v.row_p(n), *q = kind == kLessRow ? v.row_q(n) : p;
    auto at = [&](int64_t i) { return weight<T>(T::widen(p[i]), T::widen(q[i]), kind, i == token); };
    auto range_sum = [&](int64_t first, int64_t last) {  // of this thread's share of a segment
        double s = 0.0;
        for (int64_t i = first; i < last; ++i) s += at(i);
        return s;
    };

    // The segment in which the running sum passes r times the whole.
    double mine = tid < a.segs ? a.sums[(int64_t)v.b * a.segs + tid] : 0.0;
    double run = block_scan(mine, lds);
    if (tid == kThreads - 1) before_seg = run;
    __syncthreads();
    double total = before_seg;
    if (!(total > 0.0)) {
        // p is nowhere above q: the weights are p itself.
        kind = kAll;
        mine = 0.0;
        for (int s = 0; s < a.segs; ++s) {
            const int64_t f = s * a.seg, e = min(f + a.seg, a.vocab);
            double x = 0.0;
            for (int64_t i = f + tid; i < e; i += kThreads) x += at(i);
            x = block_sum(x, lds);
            if (tid == s) mine = x;
        }
        __syncthreads();
        run = block_scan(mine, lds);
        __syncthreads();
        if (tid == kThreads - 1) before_seg = run;
        __syncthreads();
        total = before_seg;
    }
    const double border = (double)a.r[v.b] * total;
    constexpr int64_t kNone = INT64_MAX;
    int64_t seg = block_min(tid < a.segs && mine > 0.0 && run > border ? tid : kNone, ids);
    // No segment passes the border where r is 1 or more: the last with weight.
    const bool past = seg == kNone;
    if (past) seg = -block_min(tid < a.segs && mine > 0.0 ? -tid : kNone, ids);
    int64_t pick = -1;
    if (seg >= 0 && total > 0.0) {
        __syncthreads();
        if (tid == seg) before_seg = run - mine;
        if (tid == 0 && seg == 0) before_seg = 0.0;
        __syncthreads();
        const int64_t f = seg * a.seg, e = min(f + a.seg, a.vocab), share = (e - f + kThreads - 1) / kThreads;
        const int64_t i0 = min(f + tid * share, e), i1 = min(i0 + share, e);
        const double own = range_sum(i0, i1);
        double s = before_seg + (block_scan(own, lds) - own);
        int64_t hit = kNone, top = kNone;
        for (int64_t i = i0; i < i1; ++i) {
            const double w = at(i);
            s += w;
            if (w > 0.0) {
                top = -i;
                if (hit == kNone && s > border) hit = i;
            }
        }
        hit = past ? kNone : block_min(hit, ids);
        // None where the two orders of summation round the border apart.
        const int64_t end = block_min(top, ids);
        pick = hit != kNone ? hit : end != kNone ? -end : -1;
    }
    for (int i = tid; i <= a.drafts; i += kThreads)
        a.tokens[(int64_t)v.b * (a.drafts + 1) + i] = i < n ? v.drafted(i) : i == n ? pick : -1;
}

template <class T>
hipError_t verify(const Verify& a, hipStream_t stream) {
    verify_sum_kernel<T><<<dim3((unsigned)a.segs, (unsigned)a.batch), kThreads, 0, stream>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    verify_pick_kernel<T><<<(unsigned)a.batch, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_verify(int type, const Verify& a, hipStream_t stream) {
    return type == RED_F32 ? verify<F32>(a, stream) : type == RED_F16 ? verify<F16>(a, stream) : verify<BF16>(a, stream);
}

}  // namespace libred
