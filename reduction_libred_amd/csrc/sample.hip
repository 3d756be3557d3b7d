// Sampling: short rows, a block a row in one launch, and the choice of the kernel by
// types and length.
//
// A block holds the row in registers, OWN neighbouring logits a thread, so the row is
// read and its weights are computed once; everything after that is sums over the
// block. A border (see sample_common.hpp) is found by the weights' bins, then by bins
// of equal numbers of codes, until a wave can rank what is left. Latency bounds a few
// rows (4000 logits: 5.9 us without filters, 10.4 with top-p, 11.3 with top-k as well;
// read again for every step they took 16.5 and 19), float64 instructions many (1900
// rows 74 us, of which a read is 4).
#include "sample_common.hpp"

namespace libred {

namespace {

// The logits of a thread, as codes (0: none), weights and bins.
template <class T, int OWN>
struct Held {
    uint64_t code[OWN], units[OWN];
    double weight[OWN];
    int bin[OWN];
};

// The code at which the running sum of the weights (`ones`: of ones) along the order,
// among those from `from` on, reaches `want`, which is not 0 and not more than their
// sum. By the block.
template <class T, int OWN>
__device__ __forceinline__ uint64_t held_border(const Held<T, OWN>& x, Sums& s, uint64_t from, uint64_t want, bool ones) {
    const int tid = threadIdx.x, lane = tid % kWave;
    clear_bins(s);
    uint64_t last = 0;  // of the last bin, which may hold most tokens: not by atomics
    unsigned int lasts = 0;
#pragma unroll
    for (int j = 0; j < OWN; ++j) {
        const uint64_t v = x.code[j] == 0 || x.code[j] < from ? 0 : ones ? 1 : x.units[j];
        if (v == 0) continue;
        if (x.bin[j] == kBins - 1) {
            last += v, ++lasts;
        } else {
            atomicAdd(&s.mass[x.bin[j]], (unsigned long long)v);
            atomicAdd(&s.count[x.bin[j]], 1u);
        }
    }
    if (__any(lasts != 0)) {
        last = group_combine<kWave>(last, AddU64());
        lasts = group_combine<kWave>(lasts, [](unsigned a, unsigned b) { return a + b; });
        if (lane == 0) atomicAdd(&s.mass[kBins - 1], (unsigned long long)last), atomicAdd(&s.count[kBins - 1], lasts);
    }
    find_bin(s, want, false);
    const int bin = s.bin;
    want = s.rest;
    unsigned int in = s.count[bin];
    uint64_t low = from, high = ~0ull;  // of codes that are in question
    auto inside = [&](int j) { return x.code[j] != 0 && x.bin[j] == bin && x.code[j] >= low && x.code[j] < high && (ones || x.units[j] > 0); };
    if (in > kWave) {
        // From the least of them to the largest.
        uint64_t least = ~0ull, most = 0;
#pragma unroll
        for (int j = 0; j < OWN; ++j)
            if (inside(j)) least = min(least, x.code[j]), most = max(most, x.code[j]);
        most = block_combine(most, s, MaxU64());
        least = ~block_combine(~least, s, MaxU64());
        low = least, high = most + 1;
    }
    while (in > kWave) {
        const int bits = 64 - __builtin_clzll((high - low - 1) | 1), to = bits > 8 ? bits - 8 : 0;
        clear_bins(s);
#pragma unroll
        for (int j = 0; j < OWN; ++j) {
            if (!inside(j)) continue;
            const int d = (int)((x.code[j] - low) >> to);
            atomicAdd(&s.mass[d], (unsigned long long)(ones ? 1 : x.units[j]));
            atomicAdd(&s.count[d], 1u);
        }
        find_bin(s, want, true);
        low += (uint64_t)s.bin << to;
        high = high - low < (1ull << to) ? high : low + (1ull << to);
        want = s.rest, in = s.count[s.bin];
    }
    __syncthreads();
    if (tid == 0) s.held = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < OWN; ++j) {
        if (!inside(j)) continue;
        const unsigned int at = atomicAdd(&s.held, 1u);
        if (at < kWave) s.few[at] = x.code[j], s.few_own[at] = ones ? 1 : x.units[j];
    }
    __syncthreads();
    if (tid < kWave) {
        const int held = min((int)s.held, kWave);
        const uint64_t found = rank_border(lane < held ? s.few[lane] : 0, lane < held ? s.few_own[lane] : 0, held, want);
        if (lane == 0) s.found = found;
    }
    __syncthreads();
    return s.found;
}

template <class T, class P, int OWN>
__global__ __launch_bounds__(kThreads) void sample_row_kernel(Sample a) {
    using R = Row<T>;
    __shared__ Sums s;
    const int at = a.first_row + blockIdx.x, b = at / a.steps, step = at - b * a.steps, tid = threadIdx.x, i0 = tid * OWN;
    R row(a, b, step);
    float x[OWN];
    row.template neighbours<OWN>(i0, x);
    const float r = a.tokens ? a.r[at] : 0.f;
    const Settings set(a, b);
    uint64_t first = 0;
#pragma unroll
    for (int j = 0; j < OWN; ++j)
        if (i0 + j < a.vocab) first = max(first, R::C::of(x[j], i0 + j));
    first = block_combine(first, s, MaxU64());
    const bool none = R::C::logit(first) == kNone;
    first = row.settle(first, set.scale, a.shift);
    Held<T, OWN> h;
#pragma unroll
    for (int j = 0; j < OWN; ++j) {
        if (row.infinite) x[j] = x[j] == __builtin_inff() ? 0.f : kNone;
        h.code[j] = x[j] == kNone ? 0 : R::C::of(x[j], i0 + j);
        h.weight[j] = row.weight(x[j]), h.units[j] = row.units(h.weight[j]), h.bin[j] = row.bin(x[j]);
    }
    uint64_t border = none ? ~0ull : set.k == 1 ? first : 0;
    if (!none && set.k > 1) {
        if (set.k < a.vocab) {
            uint64_t count = 0;
#pragma unroll
            for (int j = 0; j < OWN; ++j) count += h.code[j] != 0;
            if (block_combine(count, s, AddU64()) > (uint64_t)set.k) border = held_border(h, s, 0, (uint64_t)set.k, true);
        }
        if (set.p < 2.0) {
            uint64_t all = 0;
#pragma unroll
            for (int j = 0; j < OWN; ++j) all += h.code[j] >= border ? h.units[j] : 0;
            const uint64_t found = held_border(h, s, border, top_p_target(set.p, block_combine(all, s, AddU64())), false);
            border = found > border ? found : border;
        }
    }
    // What is kept, its sum, and the token at which that passes the target.
    uint64_t mine = 0, total;
#pragma unroll
    for (int j = 0; j < OWN; ++j) {
        const bool kept = h.code[j] != 0 && h.code[j] >= border && h.weight[j] >= set.m;
        if (!kept) h.weight[j] = 0.0, h.units[j] = 0;
        mine += h.units[j];
    }
    uint64_t before = block_before(mine, s, &total);
    if (a.tokens) {
        const uint64_t want = draw_target(r, total);
        if (none && tid == 0) a.tokens[at] = -1;
#pragma unroll
        for (int j = 0; j < OWN; ++j) {
            if (before < want && before + h.units[j] >= want) a.tokens[at] = i0 + j;
            before += h.units[j];
        }
    }
    if (a.probs) {
        typename P::bits* probs = static_cast<typename P::bits*>(a.probs) + b * a.probs_batch + step * a.probs_step;
        const double share = none ? 0.0 : row.unit / (double)total;
        typedef typename P::bits Out __attribute__((ext_vector_type(4), aligned(sizeof(typename P::bits))));
#pragma unroll
        for (int j = 0; j < OWN; j += 4) {
            Out v;
            // A second rounding, from float32, moves a 16-bit one by 2^-16 of its step at most.
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = P::narrow((float)(h.weight[j + k] * share));
            if (i0 + j + 4 <= a.vocab) {
                *reinterpret_cast<Out*>(probs + i0 + j) = v;
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (i0 + j + k < a.vocab) probs[i0 + j + k] = v[k];
            }
        }
    }
}

template <class T, class P>
hipError_t launch_row(const Sample& a, unsigned int rows, hipStream_t stream) {
    static_assert(kSampleRow == 2 * kThreads * 4, "4 or 8 logits a thread");
    if (a.vocab <= kThreads * 4) sample_row_kernel<T, P, 4><<<rows, kThreads, 0, stream>>>(a);
    else sample_row_kernel<T, P, 8><<<rows, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

template <class T>
hipError_t launch_row_type(int probs_type, const Sample& a, unsigned int rows, hipStream_t stream) {
    return probs_type == RED_F16    ? launch_row<T, F16>(a, rows, stream)
           : probs_type == RED_BF16 ? launch_row<T, BF16>(a, rows, stream)
                                    : launch_row<T, F32>(a, rows, stream);
}

}  // namespace

hipError_t launch_sample(int type, int probs_type, const Sample& a, unsigned int rows, hipStream_t stream) {
    if (a.chunks > 0) return launch_sample_split(type, probs_type, a, rows, stream);
    return type == RED_F32   ? launch_row_type<F32>(probs_type, a, rows, stream)
           : type == RED_F16 ? launch_row_type<F16>(probs_type, a, rows, stream)
                             : launch_row_type<BF16>(probs_type, a, rows, stream);
}

}  // namespace libred
