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
// First launch: scores. A block has some pages of one kv head; G lanes take a
// page, 8 neighbouring elements each of both bounds. Second launch: a block a
// (sequence, kv head) finds the border among the scores by bins of equal width,
// in whose one a wave ranks the rest (where many are close or equal, after bins
// of their bits), and lists the pages above it, and of those equal to it the
// lowest, in order.
//
// Scores (32 query and 8 kv heads of 128): 5.2 us for one sequence of 2048 pages, 10.7
// for 32 of up to 512 (36 MB of bounds, 3.4 TB/s), 14.8 for 8 of up to 2048 with 8
// nodes (41 MB). In the last the chain to the first score (lengths, page numbers, bounds,
// queries) is 8, the queries' sums 2 and the other steps 5. 1 or 4 pages in flight
// instead of 2, two steps ahead instead of one, 64 or 256 pages a block, 6 waves a SIMD
// were slower or even; queries added up an element a thread took 16.5. The choice: 5.3 to 7 us for up to 2048 pages,
// seven steps of the block one after another, which the pages of a thread lengthen
// (8 of them: 8 to 9 us).
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

__device__ __forceinline__ double score_of(uint64_t key) { return __builtin_bit_cast(double, key >> 63 ? key & ~(1ull << 63) : ~key); }

template <class T, int VEC, int G>
__global__ __launch_bounds__(kScoreThreads) void score_kernel(SelectPages a) {
    constexpr int N = VEC == 8 ? 8 : 4, R = kWave / G, W = kScoreThreads / kWave;
    __shared__ double up[RED_HEAD_MAX_DIM], down[RED_HEAD_MAX_DIM];
    constexpr int Q = VEC == 8 ? 4 : 1;  // elements of a query that a thread adds up
    __shared__ double parts[2][kScoreThreads * Q];
    const int b = blockIdx.z, h = blockIdx.x, first = blockIdx.y * a.share;  // the heads of the same pages side by side
    const Pages p(a, b);
    const int last = min(first + a.share, min(p.all, p.tail));
    if (p.all <= a.budget || first >= last) return;  // all are selected, or none of these is scored

    const int tid = threadIdx.x, lane = tid % kWave, in = lane % G, wave = tid / kWave;
    const int32_t* table = a.table + b * a.table_stride;
    const typename T::bits* lo = static_cast<const typename T::bits*>(a.lo) + h * a.bound_head;
    const typename T::bits* hi = static_cast<const typename T::bits*>(a.hi) + h * a.bound_head;
    uint64_t* keys = a.keys + ((int64_t)b * a.heads + h) * a.most;
    // U pages of each group of lanes at a time, the next ones on their way: the
    // first before the queries are added up, page numbers a step earlier still.
    constexpr int U = VEC == 8 ? 2 : 1, P = VEC == 8 ? 1 : N;
    constexpr int kStep = W * R * U;
    using V = typename Vec<T, VEC>::type;
    struct Bounds {
        V l[U][P], m[U][P];
        bool good[U];
    };
    int page[U];
    auto look = [&](int j0) {
#pragma unroll
        for (int k = 0; k < U; ++k) page[k] = table[min(j0 + (wave * U + k) * R + lane / G, last - 1)];
    };
    auto load = [&](Bounds& x) {
#pragma unroll
        for (int k = 0; k < U; ++k) x.good[k] = page[k] >= 0 && page[k] < a.pages;
        if (a.pages == 0) return;  // nothing may be read
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int64_t at = x.good[k] ? page[k] * a.bound_page : 0;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int e = (in + i * kWave) * VEC < a.dim ? in + i * kWave : 0;
                x.l[k][i] = reinterpret_cast<const V*>(lo + at)[e];
                x.m[k][i] = reinterpret_cast<const V*>(hi + at)[e];
            }
        }
    };
    Bounds x = {};
    look(first);
    load(x);
    look(first + kStep);

    // U and D: threads side by side take Q elements each of a row, the rows are shared
    // among the rest. A row's place follows from the last one's: the division by the
    // group for each took as long as the pages.
    int log2 = 0;
    while (Q << log2 < a.dim) ++log2;
    const int d = (tid & ((1 << log2) - 1)) * Q, share = tid >> log2, shares = kScoreThreads >> log2, rows = p.count * a.group;
    double u[Q] = {}, v[Q] = {};
    if (d < a.dim && share < rows) {
        typedef typename T::bits QV __attribute__((ext_vector_type(Q)));
        const int node = share / a.group, skip = shares / a.group, over = shares - skip * a.group;
        int member = share - node * a.group, r = share;
        const typename T::bits* q = static_cast<const typename T::bits*>(a.q) + b * a.q_batch + node * a.q_node + (h * a.group + member) * a.q_head + d;
        const int64_t step = skip * a.q_node + over * a.q_head, wrap = a.q_node - a.group * a.q_head;
        constexpr int K = 2;
        while (r < rows) {
            QV f[K];
            bool good[K];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                good[k] = r < rows;
                f[k] = *reinterpret_cast<const QV*>(q);
                r += shares;
                if (r < rows) {  // else the last row again
                    q += step, member += over;
                    if (member >= a.group) q += wrap, member -= a.group;
                }
            }
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (good[k])
#pragma unroll
                    for (int i = 0; i < Q; ++i) {
                        // A NaN takes part in both.
                        const double z = (double)T::widen(f[k][i]);
                        u[i] += z < 0.0 ? 0.0 : z;
                        v[i] += z > 0.0 ? 0.0 : z;
                    }
        }
    }
#pragma unroll
    for (int i = 0; i < Q; ++i) parts[0][tid * Q + i] = u[i], parts[1][tid * Q + i] = v[i];
    __syncthreads();
    if (tid < a.dim) {
        double all_u = 0.0, all_v = 0.0;
        for (int s = 0; s < min(shares, rows); ++s) all_u += parts[0][(s * Q << log2) + tid], all_v += parts[1][(s * Q << log2) + tid];
        up[tid] = all_u, down[tid] = all_v;
    }
    __syncthreads();
    double pu[N], pd[N];
    bool there[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = VEC == 8 ? in * 8 + i : in + i * kWave;
        there[i] = e < a.dim;
        pu[i] = there[i] ? up[e] : 0.0, pd[i] = there[i] ? down[e] : 0.0;
    }
    bool none = false;  // a score is no number
    for (int j0 = first; j0 < last; j0 += kStep) {
        const Bounds now = x;
        if (j0 + kStep < last) {
            load(x);
            look(j0 + 2 * kStep);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            float fl[N], fh[N];
            if constexpr (VEC == 8) {
                widen_vec<T, 8>(now.l[k][0], fl);
                widen_vec<T, 8>(now.m[k][0], fh);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) fl[i] = T::widen(now.l[k][i]), fh[i] = T::widen(now.m[k][i]);
            }
            double s = 0.0;
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (VEC == 8 || there[i]) s = __builtin_fma(pd[i], (double)fl[i], __builtin_fma(pu[i], (double)fh[i], s));
            if (VEC == 8 && !there[0]) s = 0.0;  // a lane's elements are all there, or none
            none |= s != s;
            s = group_combine<G>(s, AddF64());
            const int j = j0 + (wave * U + k) * R + lane / G;
            if (in == 0 && j < last) keys[j] = now.good[k] ? ordered(s) : 0;
        }
    }
    // 0 times an infinite bound is no number, though no query takes that bound: the
    // wave's pages again, without these products. (In the loop above it takes 104
    // registers instead of 86, a wave a SIMD less.)
    if (!__any(none)) return;
#pragma unroll 1
    for (int j0 = first + wave * U * R; j0 < last; j0 += kStep)
#pragma unroll 1
        for (int k = 0; k < U; ++k) {
            const int j = j0 + k * R + lane / G, number = table[min(j, last - 1)];
            const bool good = number >= 0 && number < a.pages;
            const int64_t at = good ? number * a.bound_page : 0;
            double s = 0.0;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int e = VEC == 8 ? in * 8 + i : in + i * kWave;
                if (!there[i] || a.pages == 0) continue;
                const double most = (double)T::widen(hi[at + e]), least = (double)T::widen(lo[at + e]);
                if (pu[i] != 0.0 || most != most) s = __builtin_fma(pu[i], most, s);
                if (pd[i] != 0.0 || least != least) s = __builtin_fma(pd[i], least, s);
            }
            s = group_combine<G>(s, AddF64());
            if (in == 0 && j < last) keys[j] = good ? ordered(s) : 0;
        }
}

constexpr int kBits = 8, kBins = 1 << kBits;

__device__ __forceinline__ int wave_scan(int v) {
    v += dpp_move<0x111, 0xF>(0, v);  // shifted by 1, 2, 4 and 8 in rows of 16
    v += dpp_move<0x112, 0xF>(0, v);
    v += dpp_move<0x114, 0xF>(0, v);
    v += dpp_move<0x118, 0xF>(0, v);
    v += dpp_move<0x142, 0xA>(0, v);  // rows 0 and 2 into 1 and 3
    v += dpp_move<0x143, 0xC>(0, v);  // the first half into the second
    return v;
}

// A thread has OWN pages side by side of every tile.
template <int THREADS, int OWN>
__global__ __launch_bounds__(THREADS) void choose_kernel(SelectPages a) {
    constexpr int W = THREADS / kWave, kTile = THREADS * OWN;
    __shared__ int bins[kBins], lds[W], digit, rest, held, few_pages[kWave];
    __shared__ unsigned long long least, most, few[kWave], border;
    const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const Pages p(a, b);
    int32_t* out = a.selected + ((int64_t)b * a.heads + h) * a.budget;
    const int32_t* table = a.table + b * a.table_stride;
    if (h == 0 && tid == 0) a.selected_lens[b] = p.count > 0 ? (int)(p.len - (int64_t)(p.all - p.chosen) * a.places) : 0;
    if (p.all <= a.budget) {
        for (int i = tid; i < a.budget; i += THREADS) out[i] = i < p.all ? table[i] : -1;
        return;
    }
    // Pages from `begin` to `end` have scores, all others are selected.
    const uint64_t* keys = a.keys + ((int64_t)b * a.heads + h) * a.most;
    const int begin = min(a.first, p.all), end = max(min(p.tail, p.all), begin);
    int need = a.budget - (p.all - (end - begin));
    // The pages of the first tile stay in registers, most sequences have no more.
    uint64_t own[OWN];
    int32_t pages[OWN];
    auto load = [&](int j0, int i) -> uint64_t {
        const int j = j0 + tid * OWN + i;
        return keys[min(max(j, begin), max(end - 1, begin))];
    };
#pragma unroll
    for (int i = 0; i < OWN; ++i) own[i] = load(0, i), pages[i] = table[min(tid * OWN + i, p.all - 1)];
    auto each = [&](auto f) __attribute__((always_inline)) {
        for (int j0 = 0; j0 < end; j0 += kTile)
#pragma unroll
            for (int i = 0; i < OWN; ++i) {
                const int j = j0 + tid * OWN + i;
                if (j >= begin && j < end) f(j0 == 0 ? own[i] : load(j0, i), j);
            }
    };
    // The need-th largest. First by bins of equal width between the least and the
    // largest score that are finite, which leaves few in the border's bin.
    if (tid == 0) least = ~0ull, most = 0, held = 0;
    for (int i = tid; i < kBins; i += THREADS) bins[i] = 0;
    __syncthreads();
    constexpr uint64_t kLow = 0x0010000000000000ull, kHigh = 0xFFEFFFFFFFFFFFFFull;  // of the finite scores
    uint64_t low = ~0ull, high = 0;
    each([&](uint64_t k, int) {
        if (k >= kLow && k <= kHigh) low = k < low ? k : low, high = k > high ? k : high;
    });
    low = group_combine<kWave>(low, [](uint64_t m, uint64_t n) { return m < n ? m : n; });
    high = group_combine<kWave>(high, [](uint64_t m, uint64_t n) { return m > n ? m : n; });
    if (lane == 0 && low <= high) atomicMin(&least, (unsigned long long)low), atomicMax(&most, (unsigned long long)high);
    __syncthreads();
    const double from = score_of(least), width = score_of(most) - from, per = width > 0.0 && width < __builtin_inf() ? kBins / width : 0.0;
    auto bin = [&](uint64_t k) { return k < kLow ? 0 : k > kHigh ? kBins - 1 : min(max((int)((score_of(k) - from) * per), 0), kBins - 1); };
    // The bin (from the last down) in which the need-th is, of those counted.
    auto find = [&]() {
        __syncthreads();
        if (wave == 0) {
            // Lane l has bins 255 - 4 l and the 3 below.
            int of[4], sum = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) of[i] = bins[kBins - 1 - 4 * lane - i], sum += of[i];
            const int upto = wave_scan(sum);
            int before = upto - sum;
            if (before < need && upto >= need) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (before < need && before + of[i] >= need) digit = kBins - 1 - 4 * lane - i, rest = need - before, held = of[i];
                    before += of[i];
                }
            }
        }
        __syncthreads();
    };
    // The border is a key: `prefix`, of which the lowest `need` pages are selected.
    uint64_t prefix = ~0ull;
    if (need > 0) {
        each([&](uint64_t k, int) { atomicAdd(&bins[bin(k)], 1); });
        find();
        const int where = digit;
        need = rest;
        int in = held, shift = 64;
        prefix = 0;
        auto inside = [&](uint64_t k) { return bin(k) == where && (shift == 64 || k >> shift == prefix); };
        // Then, where many scores are close or equal, by digits of their bits.
        while (in > kWave && shift > 0) {
            const int down = shift - kBits;
            __syncthreads();
            for (int i = tid; i < kBins; i += THREADS) bins[i] = 0;
            __syncthreads();
            each([&](uint64_t k, int) {
                if (inside(k)) atomicAdd(&bins[k >> down & (kBins - 1)], 1);
            });
            find();
            prefix = (shift == 64 ? 0 : prefix << kBits) | (uint64_t)digit;
            need = rest, in = held;
            shift = down;
        }
        // A wave ranks what is left.
        if (shift > 0) {
            __syncthreads();
            if (tid == 0) held = 0;
            __syncthreads();
            each([&](uint64_t k, int j) {
                if (!inside(k)) return;
                const int at = atomicAdd(&held, 1);
                if (at < kWave) few[at] = k, few_pages[at] = j;
            });
            __syncthreads();
            if (wave == 0) {
                const int n = min(held, kWave);
                const uint64_t mine = lane < n ? few[lane] : 0;
                const int page = lane < n ? few_pages[lane] : 0;
                int ahead = 0, larger = 0;
                for (int i = 0; i < n; ++i) {
                    const uint64_t k = read_lane(mine, i);
                    larger += k > mine, ahead += k > mine || (k == mine && read_lane(page, i) < page);
                }
                if (lane < n && ahead == need - 1) border = mine, rest = need - larger;
            }
            __syncthreads();
            prefix = border, need = rest;
        }
    }
    // The selected ones in order: those without a score, those above the border, and
    // of those that begin like it the lowest `need`.
    int more_before = 0, same_before = 0;
    for (int j0 = 0; j0 < p.all; j0 += kTile) {
        uint64_t k[OWN];
        int more = 0, same = 0;
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            const int j = j0 + tid * OWN + i;
            k[i] = j0 == 0 ? own[i] : load(j0, i);
            const bool scored = j >= begin && j < end;
            more += j < p.all && (!scored || k[i] > prefix);
            same += scored && k[i] == prefix;
        }
        const int v = more << 16 | same, upto = wave_scan(v);  // at most kTile each
        __syncthreads();
        if (lane == kWave - 1) lds[wave] = upto;
        __syncthreads();
        int before = upto - v, all = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w == wave) before += all;
            all += lds[w];
        }
        int m = more_before + (before >> 16), s = same_before + (before & 0xFFFF);
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            const int j = j0 + tid * OWN + i;
            if (j >= p.all) continue;
            const bool scored = j >= begin && j < end, is_more = !scored || k[i] > prefix, is_same = scored && k[i] == prefix;
            if (is_more || (is_same && s < need)) out[m + min(s, need)] = j0 == 0 ? pages[i] : table[j];
            m += is_more, s += is_same;
        }
        more_before += all >> 16, same_before += all & 0xFFFF;
    }
}

template <class T>
hipError_t select_pages(int vec, int lanes, const SelectPages& a, hipStream_t stream) {
    const dim3 grid((unsigned)a.heads, (unsigned)((a.most + a.share - 1) / a.share), (unsigned)a.batch);
    if (a.most > a.budget) {
        if (vec == 1) score_kernel<T, 1, 64><<<grid, kScoreThreads, 0, stream>>>(a);
        else if (lanes == 8) score_kernel<T, 8, 8><<<grid, kScoreThreads, 0, stream>>>(a);
        else if (lanes == 16) score_kernel<T, 8, 16><<<grid, kScoreThreads, 0, stream>>>(a);
        else score_kernel<T, 8, 32><<<grid, kScoreThreads, 0, stream>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    // (Microseconds of 300 / 1024 / 2048 / 4096 / 32768 pages: 512 threads with 2 pages
    // each 5.3 / 5.5 / 7.3 / 11.4 / 68, with 4 pages 6.1 / 6.5 / 6.4 / 10.3 / 59, 1024
    // threads with 4 pages 6.8 / 7.0 / 7.1 / 8.8 / 40.)
    const dim3 each((unsigned)a.heads, (unsigned)a.batch);
    if (a.most <= 1024) choose_kernel<512, 2><<<each, 512, 0, stream>>>(a);
    else if (a.most <= 2048) choose_kernel<512, 4><<<each, 512, 0, stream>>>(a);
    else choose_kernel<1024, 4><<<each, 1024, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_select_pages(int type, int vec, int lanes, const SelectPages& a, hipStream_t stream) {
    return type == RED_F16 ? select_pages<F16>(vec, lanes, a, stream) : select_pages<BF16>(vec, lanes, a, stream);
}

}  // namespace libred
