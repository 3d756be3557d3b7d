// Selection of the pages of a cache that are worth reading for a query.
//
// A key between the bounds lo and hi of its page has q.k of at most
// sum_d max(q_d lo_d, q_d hi_d). Summed over the rows that share a kv head that
// is linear in the bounds,
//     score = sum_d (U_d hi_d + D_d lo_d),  U = sum max(q, 0), D = sum min(q, 0),
// so a page costs 2 dim multiply-adds however many rows there are, in float64:
// pages that float32 would leave in doubt are told apart, and the order of the
// sum does not matter to the choice.
//
// First launch: scores. A block has 64 pages of one kv head; G lanes take a
// page, 8 neighbouring elements each of both bounds. Second launch: a block a
// (sequence, kv head) finds the budget-th largest score digit by digit (8 bits
// at a time, from the first byte in which the scores differ) and lists the pages
// above it, and of those equal to it the lowest, in order.
#include "decode_common.hpp"
#include "serve.hpp"

namespace libred {

namespace {

struct AddF64 {
    __device__ double operator()(double a, double b) const { return a + b; }
};

// Pages of sequence b, how many of them are selected, and the first of the
// last ones that always are.
struct Pages {
    int all, chosen, tail, count, len;
    __device__ Pages(const SelectPages& a, int b) {
        count = a.count ? min(max(a.count[b], 0), a.nodes) : a.nodes;
        len = max(a.lens[b], 0);
        const int tokens = (int)min((int64_t)len + count, (int64_t)a.max_len);
        all = count > 0 ? (tokens + a.places - 1) / a.places : 0;
        chosen = min(all, a.budget);
        tail = max(len / a.places - a.last, 0);
    }
};

constexpr int kScoreThreads = 256;

// A score as a number whose order is that of the scores; NaN below all others.
__device__ __forceinline__ uint64_t ordered(double s) {
    const uint64_t u = __builtin_bit_cast(uint64_t, s + 0.0);  // -0 is 0
    if (s != s) return 0;
    return u >> 63 ? ~u : u | 1ull << 63;
}

template <class T, int VEC, int G>
__global__ __launch_bounds__(kScoreThreads) void score_kernel(SelectPages a) {
    constexpr int N = VEC == 8 ? 8 : 4, R = kWave / G, W = kScoreThreads / kWave;
    __shared__ double up[RED_HEAD_MAX_DIM], down[RED_HEAD_MAX_DIM];
    __shared__ double parts[2][kScoreThreads];
    const int b = blockIdx.z, h = blockIdx.y, first = blockIdx.x * kSelectPages;
    const Pages p(a, b);
    const int last = min(first + kSelectPages, min(p.all, p.tail));
    if (p.all <= a.budget || first >= last) return;  // all are selected, or none of these is scored

    // U and D: `dims` threads side by side, the rows shared among the rest.
    const int tid = threadIdx.x;
    int dims = 1;
    while (dims < a.dim) dims <<= 1;
    const int d = tid % dims, share = tid / dims, shares = kScoreThreads / dims;
    double u = 0.0, v = 0.0;
    if (d < a.dim) {
        const typename T::bits* q = static_cast<const typename T::bits*>(a.q) + b * a.q_batch + d;
        for (int r = share; r < p.count * a.group; r += shares) {
            const int node = r / a.group, g = r - node * a.group;
            const double x = (double)T::widen(q[node * a.q_node + (h * a.group + g) * a.q_head]);
            // A NaN takes part in both.
            u += x < 0.0 ? 0.0 : x;
            v += x > 0.0 ? 0.0 : x;
        }
    }
    parts[0][tid] = u, parts[1][tid] = v;
    __syncthreads();
    if (tid < a.dim) {
        for (int s = 1; s < shares; ++s) u += parts[0][s * dims + tid], v += parts[1][s * dims + tid];
        up[tid] = u, down[tid] = v;
    }
    __syncthreads();

    const int lane = tid % kWave, in = lane % G, wave = tid / kWave;
    double pu[N], pd[N];
    bool there[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = VEC == 8 ? in * 8 + i : in + i * kWave;
        there[i] = e < a.dim;
        pu[i] = there[i] ? up[e] : 0.0, pd[i] = there[i] ? down[e] : 0.0;
    }
    const int32_t* table = a.table + b * a.table_stride;
    const typename T::bits* lo = static_cast<const typename T::bits*>(a.lo) + h * a.bound_head;
    const typename T::bits* hi = static_cast<const typename T::bits*>(a.hi) + h * a.bound_head;
    uint64_t* keys = a.keys + ((int64_t)b * a.heads + h) * a.most;
    for (int j0 = first + wave * R; j0 < last; j0 += W * R) {
        const int j = j0 + lane / G;
        const int page = j < last ? table[j] : -1;
        const bool good = page >= 0 && page < a.pages;
        const int64_t at = good ? page * a.bound_page : 0;
        double s = 0.0;
        if (good) {
            if constexpr (VEC == 8) {
                float fl[8], fh[8];
                const int c = there[0] ? in : 0;
                widen_vec<T, 8>(reinterpret_cast<const typename Vec<T, 8>::type*>(lo + at)[c], fl);
                widen_vec<T, 8>(reinterpret_cast<const typename Vec<T, 8>::type*>(hi + at)[c], fh);
                if (there[0])
#pragma unroll
                    for (int i = 0; i < 8; ++i) s += pu[i] * (double)fh[i] + pd[i] * (double)fl[i];
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (there[i]) s += pu[i] * (double)T::widen(hi[at + in + i * kWave]) + pd[i] * (double)T::widen(lo[at + in + i * kWave]);
            }
        }
        s = group_combine<G>(s, AddF64());
        if (in == 0 && j < last) keys[j] = good ? ordered(s) : 0;
    }
}

constexpr int kThreads = 1024, kBits = 8, kBins = 1 << kBits;

__global__ __launch_bounds__(kThreads) void choose_kernel(SelectPages a) {
    constexpr int W = kThreads / kWave;
    __shared__ int bins[kBins], lds[W], digit, rest, held;
    __shared__ unsigned long long differ;
    const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const Pages p(a, b);
    int32_t* out = a.selected + ((int64_t)b * a.heads + h) * a.budget;
    const int32_t* table = a.table + b * a.table_stride;
    if (h == 0 && tid == 0) a.selected_lens[b] = p.count > 0 ? (int)(p.len - (int64_t)(p.all - p.chosen) * a.places) : 0;
    if (p.all <= a.budget) {
        for (int i = tid; i < a.budget; i += kThreads) out[i] = i < p.all ? table[i] : -1;
        return;
    }
    const uint64_t* keys = a.keys + ((int64_t)b * a.heads + h) * a.most;
    auto key = [&](int j) { return j < a.first || j >= p.tail ? ~0ull : keys[j]; };
    // The budget-th largest key: `prefix` above bit `shift`, zeros below; of the
    // keys that begin like it the largest `need` are selected.
    const uint64_t one = key(0);
    if (tid == 0) differ = 0;
    __syncthreads();
    uint64_t x = 0;
    for (int j = tid; j < p.all; j += kThreads) x |= key(j) ^ one;
    if (x) atomicOr(&differ, x);
    __syncthreads();
    int shift = bytes_of(differ) * 8;                 // bits below this one differ
    uint64_t prefix = shift < 64 ? one >> shift : 0;  // the keys' bits from `shift` on
    int need = a.budget;
    while (shift > 0) {
        const int down = shift - kBits;
        for (int i = tid; i < kBins; i += kThreads) bins[i] = 0;
        __syncthreads();
        for (int j = tid; j < p.all; j += kThreads) {
            const uint64_t k = key(j);
            if (shift == 64 || k >> shift == prefix) atomicAdd(&bins[k >> down & (kBins - 1)], 1);
        }
        __syncthreads();
        if (wave == 0) {
            // Lane l has bins 255 - 4 l and the 3 below; `upto` counts from the top.
            int own[4], sum = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) own[i] = bins[kBins - 1 - 4 * lane - i], sum += own[i];
            int upto = sum;
            upto += dpp_move<0x111, 0xF>(0, upto);
            upto += dpp_move<0x112, 0xF>(0, upto);
            upto += dpp_move<0x114, 0xF>(0, upto);
            upto += dpp_move<0x118, 0xF>(0, upto);
            upto += dpp_move<0x142, 0xA>(0, upto);
            upto += dpp_move<0x143, 0xC>(0, upto);
            int before = upto - sum;
            if (before < need && upto >= need) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (before < need && before + own[i] >= need) digit = kBins - 1 - 4 * lane - i, rest = need - before, held = own[i];
                    before += own[i];
                }
            }
        }
        __syncthreads();
        prefix = (shift == 64 ? 0 : prefix << kBits) | (uint64_t)digit;
        need = rest;
        shift = down;
        if (held == need) break;  // all that begin like this
    }
    // Pages above, and the lowest `need` of those that begin like the border.
    int above = 0, equal = 0;
    for (int j0 = 0; j0 < p.all; j0 += kThreads) {
        const int j = j0 + tid;
        int more = 0, same = 0;
        if (j < p.all) {
            const uint64_t k = key(j) >> shift;
            more = k > prefix, same = k == prefix;
        }
        const uint64_t ms = __ballot(more), ss = __ballot(same), below = (1ull << lane) - 1;
        const int m = __popcll(ms & below), s = __popcll(ss & below);
        __syncthreads();
        if (lane == 0) lds[wave] = __popcll(ms) << 16 | __popcll(ss);
        __syncthreads();
        int before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w == wave) before = all;
            all += lds[w];
        }
        const int mb = above + (before >> 16) + m, sb = equal + (before & 0xFFFF) + s;
        if (more || (same && sb < need)) out[mb + min(sb, need)] = table[j];
        above += all >> 16, equal += all & 0xFFFF;
    }
}

template <class T>
hipError_t select_pages(int vec, int lanes, const SelectPages& a, hipStream_t stream) {
    const dim3 grid((unsigned)((a.most + kSelectPages - 1) / kSelectPages), (unsigned)a.heads, (unsigned)a.batch);
    if (a.most > a.budget) {
        if (vec == 1) score_kernel<T, 1, 64><<<grid, kScoreThreads, 0, stream>>>(a);
        else if (lanes == 8) score_kernel<T, 8, 8><<<grid, kScoreThreads, 0, stream>>>(a);
        else if (lanes == 16) score_kernel<T, 8, 16><<<grid, kScoreThreads, 0, stream>>>(a);
        else score_kernel<T, 8, 32><<<grid, kScoreThreads, 0, stream>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    choose_kernel<<<dim3((unsigned)a.heads, (unsigned)a.batch), kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_select_pages(int type, int vec, int lanes, const SelectPages& a, hipStream_t stream) {
    return type == RED_F16 ? select_pages<F16>(vec, lanes, a, stream) : select_pages<BF16>(vec, lanes, a, stream);
}

}  // namespace libred
