// Verification of drafted tokens, and the token sampled after them.
//
// Draft i is accepted while u_i q_i(d_i) < p_i(d_i); n is the number accepted
// before the first that is not. The next token is drawn from
//     w = max(p_n - q_n, 0)  where a draft was refused (p_n if that is 0 everywhere),
//     w = p_n                where all were accepted:
// the first token whose running sum of w passes r sum(w).
//
// Only row n of p and q is read as a whole: once for its sums, a wave a
// segment of 1024 tokens (each wave finds n for itself, from at most two
// gathers a draft), and once more in the one segment where the running sum
// passes its border, by a second launch, a block a sequence with 4 tokens a
// thread; or both by one launch, a block of 16 waves a sequence, where a row is
// short. Sums run in float64: float32 inputs differ exactly there, and a
// border is then missed by less than 2^-40 of the sum whatever the order.
// Memory bounds the first launch, latency the second: 192 rows of p and q of
// 131071 float32, 201 MB, 32.1 us (6.3 TB/s) and 4.9 us (in bf16, 101 MB, 27.7 us,
// float32 against certain drafts, 101 MB, 26.8 us); one row of 32000 3.8 us and
// 3.5 us.
#include "decode_common.hpp"

namespace libred {

namespace {

constexpr int kThreads = 256;     // of a block
constexpr int kThreadsOne = 1024;  // where one launch does it all

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

__device__ __forceinline__ double weight(float p, float q, int kind, bool token) {
    double w = (double)p;
    if (kind == kLessRow) w -= (double)q;
    if (kind == kLessToken && token) w -= 1.0;
    return w < 0.0 ? 0.0 : w;  // a NaN stays one
}

constexpr int kStep = 1024;  // tokens of a wave at a time in the sums, of a block in the choice

// Sums of the weights of segments seg, seg + stride, ...
template <class T>
__device__ __forceinline__ void segment_sums(const Verify& a, const Verifier<T>& v, int n, int seg, int stride, double* sums) {
    using V = Verifier<T>;
    constexpr int N = V::kVec, U = kStep / (kWave * N);
    const int lane = threadIdx.x % kWave;
    const int kind = n == v.count ? kAll : a.q ? kLessRow : kLessToken;
    const int64_t token = kind == kLessToken ? v.drafted(n) : -1;
    const typename V::B *p = v.row_p(n), *q = kind == kLessRow ? v.row_q(n) : p;
    for (; seg < a.segs; seg += stride) {
    const int64_t first = (int64_t)seg * a.seg, last = min(first + a.seg, a.vocab);
    double sum = 0.0;
    for (int64_t i0 = first; i0 < last; i0 += kStep) {
        if (i0 + kStep <= last) {
            typename V::Vector x[U], y[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                x[u] = __builtin_nontemporal_load(reinterpret_cast<const typename V::Vector*>(p + i0 + (u * kWave + lane) * N));
                y[u] = __builtin_nontemporal_load(reinterpret_cast<const typename V::Vector*>(q + i0 + (u * kWave + lane) * N));
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < N; ++j)
                    sum += weight(T::widen(x[u][j]), T::widen(y[u][j]), kind, i0 + (u * kWave + lane) * N + j == token);
        } else {
            for (int64_t i = i0 + lane; i < last; i += kWave) sum += weight(T::widen(p[i]), T::widen(q[i]), kind, i == token);
        }
    }
    sum = group_combine<kWave>(sum, AddF64());
    if (lane == 0) sums[seg] = sum;
    }
}

template <class T>
__global__ __launch_bounds__(kThreads) void verify_sum_kernel(Verify a) {
    constexpr int W = kThreads / kWave;
    asm volatile("" ::"s"(a.p), "s"(a.u), "s"(a.vocab));  // one argument of every 64-byte line
    const Verifier<T> v(a, blockIdx.y);
    const int seg = blockIdx.x * W + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (seg >= a.segs) return;
    const int n = v.accepted();
    if (seg == 0 && threadIdx.x % kWave == 0) a.accepted[v.b] = n;
    segment_sums(a, v, n, seg, gridDim.x * W, a.sums + (int64_t)v.b * a.segs);
}

// Running sum over the threads of the block, this thread's value included; and
// the whole sum. In a fixed order.
template <int WAVES>
__device__ __forceinline__ double block_scan(double v, double* lds, double* total) {
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    v += dpp_move<0x111, 0xF>(0.0, v);  // shifted by 1, 2, 4 and 8 in rows of 16
    v += dpp_move<0x112, 0xF>(0.0, v);
    v += dpp_move<0x114, 0xF>(0.0, v);
    v += dpp_move<0x118, 0xF>(0.0, v);
    v += dpp_move<0x142, 0xA>(0.0, v);  // rows 0 and 2 into 1 and 3
    v += dpp_move<0x143, 0xC>(0.0, v);  // the first half into the second
    __syncthreads();
    if (lane == kWave - 1) lds[wave] = v;
    __syncthreads();
    double before = 0.0, all = 0.0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        if (w == wave) before = all;
        all += lds[w];
    }
    *total = all;
    return before + v;
}

// The first (or last) thread for which `is` holds, -1 if none.
template <int WAVES>
__device__ __forceinline__ int block_find(bool is, bool last, int* lds) {
    const uint64_t mask = __ballot(is);
    const int wave = threadIdx.x / kWave;
    __syncthreads();
    if (threadIdx.x % kWave == 0)
        lds[wave] = !mask ? -1 : wave * kWave + (last ? 63 - __clzll((long long)mask) : __ffsll((unsigned long long)mask) - 1);
    __syncthreads();
    int found = -1;
#pragma unroll
    for (int w = 0; w < WAVES; ++w)
        if (lds[w] >= 0 && (last || found < 0)) found = lds[w];
    return found;
}

// The token, from the sums of the segments (this thread's: `mine`), and what
// the sequence's tokens are.
template <class T, int THREADS>
__device__ __forceinline__ void choose(const Verify& a, const Verifier<T>& v, int n, double r, double mine) {
    using V = Verifier<T>;
    constexpr int N = kStep / THREADS;  // tokens of a thread at a time
    constexpr int W = THREADS / kWave;
    __shared__ double lds[W], start;
    // `element`, of the thread that was found, has a word of its own: block_find
    // ends with reads of all of `ids`, and a wave that is done with them must
    // not change them under one that is not.
    __shared__ int ids[W], element;
    const int tid = threadIdx.x;
    int kind = n == v.count ? kAll : a.q ? kLessRow : kLessToken;
    const int64_t token = kind == kLessToken ? v.drafted(n) : -1;
    const typename V::B *p = v.row_p(n), *q = kind == kLessRow ? v.row_q(n) : p;
    auto at = [&](int64_t i) { return weight(T::widen(p[i]), T::widen(q[i]), kind, i == token); };

    // The segment in which the running sum passes r times the whole.
    double total, all;
    double run = block_scan<W>(mine, lds, &total);
    if (total == 0.0) {  // a NaN is no such sum: it draws nothing
        // p is nowhere above q: the weights are p itself.
        kind = kAll;
        mine = 0.0;
        for (int s = 0; s < a.segs; ++s) {
            const int64_t f = s * a.seg, e = min(f + a.seg, a.vocab);
            double x = 0.0;
            for (int64_t i = f + tid; i < e; i += THREADS) x += at(i);
            block_scan<W>(x, lds, &all);
            if (tid == s) mine = all;
        }
        run = block_scan<W>(mine, lds, &total);
    }
    const double border = r * total;
    const bool some = tid < a.segs && mine > 0.0;
    int seg = block_find<W>(some && run > border, false, ids);
    // No segment passes the border where r is 1 or more: the last with weight.
    const bool past = seg < 0;
    if (past) seg = block_find<W>(some, true, ids);
    int64_t pick = -1;
    if (seg >= 0 && total > 0.0) {
        if (tid == seg) start = seg == 0 ? 0.0 : run - mine;
        __syncthreads();
        double before = start;
        const int64_t f = seg * a.seg, e = min(f + a.seg, a.vocab);
        for (int64_t i0 = f; i0 < e; i0 += kStep) {
            double w[N], own = 0.0;
            const int64_t i = i0 + tid * N;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                w[j] = at(min(i + j, e - 1));
                if (i + j >= e) w[j] = 0.0;
                own += w[j];
            }
            double s = before + (block_scan<W>(own, lds, &all) - own);
            int hit = -1, top = -1;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                s += w[j];
                if (w[j] > 0.0) {
                    top = j;
                    if (hit < 0 && s > border) hit = j;
                }
            }
            // Of the last element with weight so far in case none passes: the
            // two orders of summation may round the border apart.
            const int who = past ? -1 : block_find<W>(hit >= 0, false, ids);
            const int end = who >= 0 ? who : block_find<W>(top >= 0, true, ids);
            if (end >= 0) {
                if (tid == end) element = who >= 0 ? hit : top;
                __syncthreads();
                pick = i0 + end * N + element;  // barriers of the next scan lie before the next write
            }
            if (who >= 0) break;
            before += all;
        }
    }
    for (int i = tid; i <= a.drafts; i += THREADS)
        a.tokens[(int64_t)v.b * (a.drafts + 1) + i] = i < n ? v.drafted(i) : i == n ? pick : -1;
}

template <class T>
__global__ __launch_bounds__(kThreads) void verify_pick_kernel(Verify a) {
    asm volatile("" ::"s"(a.p), "s"(a.u), "s"(a.vocab));
    const Verifier<T> v(a, blockIdx.x);
    const int tid = threadIdx.x;
    const double mine = tid < a.segs ? a.sums[(int64_t)v.b * a.segs + tid] : 0.0;
    choose<T, kThreads>(a, v, a.accepted[v.b], (double)a.r[v.b], mine);
}

template <class T>
__global__ __launch_bounds__(kThreadsOne) void verify_one_kernel(Verify a) {
    __shared__ double sums[kVerifyMaxSegs];
    asm volatile("" ::"s"(a.p), "s"(a.u), "s"(a.vocab));
    const Verifier<T> v(a, blockIdx.x);
    const int tid = threadIdx.x;
    const double r = (double)a.r[v.b];
    const int n = v.accepted();
    if (tid == 0) a.accepted[v.b] = n;
    segment_sums(a, v, n, __builtin_amdgcn_readfirstlane(tid / kWave), kThreadsOne / kWave, sums);
    __syncthreads();
    choose<T, kThreadsOne>(a, v, n, r, tid < a.segs ? sums[tid] : 0.0);
}

template <class T>
hipError_t verify(const Verify& a, hipStream_t stream) {
    if (a.blocks == 0) {
        verify_one_kernel<T><<<(unsigned)a.batch, kThreadsOne, 0, stream>>>(a);
        return hipGetLastError();
    }
    verify_sum_kernel<T><<<dim3((unsigned)a.blocks, (unsigned)a.batch), kThreads, 0, stream>>>(a);
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
