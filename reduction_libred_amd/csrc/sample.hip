// Sampling from a row of logits with temperature, top-k, top-p and min-p.
//
// The tokens' order (falling logits, ties by number) is that of one whole
// number a token, its code: the logit's bits, turned so that they order, above
// the number's complement. What top-k and top-p keep are the codes from a
// border on, so each is a search for one code: the first at which a running
// sum along the order, of ones or of weights, reaches a target. It is found by
// sums over bins, not by sorting: first bins of an eighth of a power of two of
// the weight, 32 powers down from the largest; then, with what is in the
// border's bin gathered in the LDS, bins of the codes' digits, 8 bits at a time.
//
// Weights exp((x - max) / T) are float64. Their sums are held in whole numbers
// of 2^-shift (45 bits for 131072 tokens), so they come out the same in any
// order: a border is missed where the target is within about 2^-37 of the
// largest weight of it, and atomics do no harm.
#include "decode_common.hpp"
#include "serve.hpp"

namespace libred {

namespace {

constexpr int kThreads = 1024, kWaves = kThreads / kWave;
constexpr int kBins = 256;
constexpr int kHeld = 2048;        // codes that are gathered in the LDS
constexpr int kCodeBits = 52;      // 32 of the logit, 20 of the number
constexpr int kMaxVocab = 1 << 20;

struct AddU64 {
    __device__ uint64_t operator()(uint64_t a, uint64_t b) const { return a + b; }
};
struct MaxU64 {
    __device__ uint64_t operator()(uint64_t a, uint64_t b) const { return a > b ? a : b; }
};

__device__ __forceinline__ uint64_t code_of(float x, int i) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const uint32_t k = u >> 31 ? ~u : u | 0x80000000u;
    return (uint64_t)k << 20 | (uint32_t)(kMaxVocab - 1 - i);
}
__device__ __forceinline__ float logit_of(uint64_t code) {
    const uint32_t k = (uint32_t)(code >> 20);
    return __builtin_bit_cast(float, k >> 31 ? k & 0x7FFFFFFFu : ~k);
}
__device__ __forceinline__ int token_of(uint64_t code) { return kMaxVocab - 1 - (int)(code & (kMaxVocab - 1)); }

constexpr float kNone = -__builtin_inff();

// What the block shares.
struct Shared {
    unsigned long long mass[kBins];
    unsigned int count[kBins];
    unsigned long long code[kHeld];  // what is in the border's bin
    unsigned long long own[kHeld];   // the weights of those
    unsigned long long part[kWaves], found, rest;
    unsigned int held, bin;
};

template <class Op>
__device__ __forceinline__ uint64_t block_combine(uint64_t v, Shared& s, Op op) {
    v = group_combine<kWave>(v, op);
    __syncthreads();
    if (threadIdx.x % kWave == 0) s.part[threadIdx.x / kWave] = v;
    __syncthreads();
    v = s.part[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v = op(v, s.part[w]);
    return v;
}

// Running sum over the wave's lanes, this one's value included.
__device__ __forceinline__ uint64_t wave_scan(uint64_t v) {
    const uint64_t none = 0;
    v += dpp_move<0x111, 0xF>(none, v);  // shifted by 1, 2, 4 and 8 in rows of 16
    v += dpp_move<0x112, 0xF>(none, v);
    v += dpp_move<0x114, 0xF>(none, v);
    v += dpp_move<0x118, 0xF>(none, v);
    v += dpp_move<0x142, 0xA>(none, v);  // rows 0 and 2 into 1 and 3
    v += dpp_move<0x143, 0xC>(none, v);  // the first half into the second
    return v;
}
// The sum of the threads before this one.
__device__ __forceinline__ uint64_t block_before(uint64_t v, Shared& s) {
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const uint64_t upto = wave_scan(v);
    __syncthreads();
    if (lane == kWave - 1) s.part[wave] = upto;
    __syncthreads();
    uint64_t before = upto - v;
    for (int w = 0; w < wave; ++w) before += s.part[w];
    return before;
}

template <class T>
struct Row {
    using B = typename T::bits;
    static constexpr int kVec = 16 / sizeof(B), kTile = kThreads * kVec;
    // Rows start on element boundaries only (a vocabulary may be odd).
    typedef B Vector __attribute__((ext_vector_type(16 / sizeof(B)), aligned(sizeof(B))));

    const B* p;
    int vocab;
    bool infinite;   // the largest logit is +inf: those count as 0, all others as -inf
    double top, scale, unit;

    __device__ __forceinline__ float seen(B bits) const {
        const float x = T::widen(bits) + 0.f;  // -0 is 0
        if (infinite) return x == __builtin_inff() ? 0.f : kNone;
        return x == x ? x : kNone;
    }
    // f(number of the first, logits) of this thread's kVec neighbours in every
    // tile of the block; kNone behind the last.
    template <class F>
    __device__ __forceinline__ void tiles(F f) const {
        for (int i0 = 0; i0 < vocab; i0 += kTile) {
            const int i = i0 + threadIdx.x * kVec;
            float x[kVec];
            if (i0 + kTile <= vocab) {
                const Vector v = *reinterpret_cast<const Vector*>(p + i);
#pragma unroll
                for (int j = 0; j < kVec; ++j) x[j] = seen(v[j]);
            } else {
#pragma unroll
                for (int j = 0; j < kVec; ++j) x[j] = i + j < vocab ? seen(p[i + j]) : kNone;
            }
            f(i, x);
        }
    }
    // f(number, logit) of every token of this thread.
    template <class F>
    __device__ __forceinline__ void each(F f) const {
        tiles([&](int i, const float(&x)[kVec]) {
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                if (i + j < vocab) f(i + j, x[j]);
        });
    }
    __device__ __forceinline__ double weight(float x) const {
        return x == kNone ? 0.0 : exp2(((double)x - top) * scale);
    }
    // In units: 2^52 more than a number below it has that number as its last bits.
    __device__ __forceinline__ uint64_t units(double w) const {
        return __builtin_bit_cast(uint64_t, w * unit + 0x1p52) & 0xFFFFFFFFFFFFFull;
    }
    // Bins of an eighth of a power of two, from the largest weight down. The
    // order of the logits holds after each rounding.
    __device__ __forceinline__ int bin(float x) const {
        const double d = (top - (double)x) * scale * 8.0;
        return d < (double)(kBins - 1) ? (int)d : kBins - 1;
    }
};

// The bin in which the running sum of `own` (bin tid) reaches `target`, what is
// missing of the target there, or bin kBins. By the block's first waves.
__device__ __forceinline__ void find_bin(Shared& s, uint64_t target, bool codes) {
    __syncthreads();
    if (threadIdx.x < kWave) {
        const int lane = threadIdx.x;
        uint64_t own[4], sum = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // Bins of weights go down from bin 0, digits of codes from the last.
            own[i] = s.mass[codes ? kBins - 1 - 4 * lane - i : 4 * lane + i];
            sum += own[i];
        }
        const uint64_t upto = wave_scan(sum);
        if (lane == 0) s.bin = kBins;
        uint64_t before = upto - sum;
        wave_lds_fence();
        if (before < target && upto >= target) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (before < target && before + own[i] >= target) {
                    s.bin = codes ? kBins - 1 - 4 * lane - i : 4 * lane + i;
                    s.rest = target - before;
                }
                before += own[i];
            }
        }
    }
    __syncthreads();
}

__device__ __forceinline__ void clear_bins(Shared& s) {
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += kThreads) s.mass[i] = 0, s.count[i] = 0;
    __syncthreads();
}

// The first code of the order, among those from `from` on, at which the running
// sum of value(number, logit) reaches target(whole sum); 0 if it does not.
// Codes of value 0 are passed over.
template <class T, class V, class G>
__device__ __forceinline__ uint64_t find_border(const Row<T>& row, Shared& s, uint64_t from, V value, G target) {
    clear_bins(s);
    uint64_t last = 0;  // of the last bin, which may hold most tokens: not by atomics
    unsigned int lasts = 0;
    row.each([&](int i, float x) {
        if (x == kNone || code_of(x, i) < from) return;
        const uint64_t v = value(x);
        if (v == 0) return;
        const int j = row.bin(x);
        if (j == kBins - 1) {
            last += v, ++lasts;
        } else {
            atomicAdd(&s.mass[j], (unsigned long long)v);
            atomicAdd(&s.count[j], 1u);
        }
    });
    last = group_combine<kWave>(last, AddU64());
    lasts = group_combine<kWave>(lasts, [](unsigned a, unsigned b) { return a + b; });
    if (threadIdx.x % kWave == 0 && lasts) {
        atomicAdd(&s.mass[kBins - 1], (unsigned long long)last);
        atomicAdd(&s.count[kBins - 1], lasts);
    }
    __syncthreads();
    const uint64_t all = block_combine(threadIdx.x < kBins ? s.mass[threadIdx.x] : 0, s, AddU64());
    uint64_t want = target(all);
    if (want > all || want == 0) return 0;
    find_bin(s, want, false);
    const int bin = s.bin;
    want = s.rest;
    unsigned int in = s.count[bin];
    // Too many to gather: digits of the codes in that bin, over the whole row.
    int shift = kCodeBits;
    uint64_t prefix = 0;
    auto inside = [&](uint64_t code, float x) { return x != kNone && code >= from && row.bin(x) == bin && code >> shift == prefix; };
    while (in > kHeld && shift > 0) {
        const int width = min(shift, 8), down = shift - width;
        clear_bins(s);
        row.each([&](int i, float x) {
            const uint64_t code = code_of(x, i);
            if (!inside(code, x)) return;
            const uint64_t v = value(x);
            if (v == 0) return;
            const int d = (int)(code >> down) & (255 >> (8 - width));
            atomicAdd(&s.mass[d], (unsigned long long)v);
            atomicAdd(&s.count[d], 1u);
        });
        find_bin(s, want, true);
        prefix = prefix << width | s.bin;
        want = s.rest;
        in = s.count[s.bin];
        shift = down;
    }
    __syncthreads();
    if (threadIdx.x == 0) s.held = 0, s.found = 0;
    __syncthreads();
    row.each([&](int i, float x) {
        const uint64_t code = code_of(x, i);
        if (!inside(code, x)) return;
        const uint64_t v = value(x);
        if (v == 0) return;
        const unsigned int at = atomicAdd(&s.held, 1u);
        if (at < kHeld) s.code[at] = code, s.own[at] = v;
    });
    __syncthreads();
    const int held = (int)min(s.held, (unsigned)kHeld);
    // From the first digit in which they differ on.
    const uint64_t one = s.code[0];
    for (int i = threadIdx.x; i < held; i += kThreads)
        if (const uint64_t x = s.code[i] ^ one) atomicOr(&s.found, (unsigned long long)x);
    __syncthreads();
    int down = bytes_of(s.found) * 8;
    prefix = one >> down;
    while (down > 0) {
        const int width = min(down, 8), to = down - width;
        clear_bins(s);
        for (int i = threadIdx.x; i < held; i += kThreads)
            if (s.code[i] >> down == prefix) atomicAdd(&s.mass[(s.code[i] >> to) & (255 >> (8 - width))], s.own[i]);
        find_bin(s, want, true);
        prefix = prefix << width | s.bin;
        want = s.rest;
        down = to;
    }
    return prefix;
}

struct Settings {
    double p, m, scale;  // p 2: no top-p
    int64_t k;
    __device__ Settings(const Sample& a, int b) {
        const float t = a.temperature ? a.temperature[b] : 1.f;
        const bool greedy = !(t > 0.f);
        k = a.top_k ? a.top_k[b] : 0;
        if (k < 1 || k > a.vocab) k = a.vocab;
        if (greedy) k = 1;
        const float tp = a.top_p ? a.top_p[b] : 1.f, mp = a.min_p ? a.min_p[b] : 0.f;
        p = tp < 1.f && k > 1 ? fmax((double)tp, 0.0) : 2.0;
        m = mp > 0.f ? fmin((double)mp, 1.0) : 0.0;
        scale = 1.4426950408889634 / (greedy ? 1.0 : (double)t);
    }
};

template <class T, class P>
__global__ __launch_bounds__(kThreads) void sample_kernel(Sample a) {
    using R = Row<T>;
    constexpr int kRun = kWave * R::kVec;  // tokens of a wave at a time
    __shared__ Shared s;
    __shared__ unsigned long long runs[kMaxVocab / kRun];
    const int b = blockIdx.x / a.steps, step = blockIdx.x - b * a.steps, tid = threadIdx.x, lane = tid % kWave;
    const Settings set(a, b);
    R row;
    row.p = static_cast<const typename T::bits*>(a.x) + b * a.batch_stride + step * a.step_stride;
    row.vocab = a.vocab, row.infinite = false;
    typename P::bits* probs = a.probs ? static_cast<typename P::bits*>(a.probs) + b * a.probs_batch + step * a.probs_step : nullptr;

    uint64_t first = 0;
    row.each([&](int i, float x) { first = max(first, code_of(x, i)); });
    first = block_combine(first, s, MaxU64());
    float top = logit_of(first);
    if (top == kNone) {
        if (a.tokens && tid == 0) a.tokens[blockIdx.x] = -1;
        if (probs)
            for (int i = tid; i < a.vocab; i += kThreads) probs[i] = P::narrow(0.f);
        return;
    }
    if (top == __builtin_inff()) {
        row.infinite = true;
        first = code_of(0.f, token_of(first));
        top = 0.f;
    }
    row.top = top;
    row.scale = set.scale;
    row.unit = __builtin_ldexp(1.0, a.shift);

    uint64_t border = 0;
    if (set.k == 1) border = first;
    else if (set.k < a.vocab) border = find_border(row, s, 0, [](float) -> uint64_t { return 1; }, [&](uint64_t) { return (uint64_t)set.k; });
    if (set.p < 2.0) {
        const uint64_t found = find_border(row, s, border, [&](float x) { return row.units(row.weight(x)); },
                                           [&](uint64_t all) { return max((uint64_t)__builtin_ceil(set.p * (double)all), (uint64_t)1); });
        border = max(border, found);
    }
    // The kept weights, summed over the tokens that a wave reads at a time.
    auto kept = [&](int i, float x) {
        if (x == kNone || code_of(x, i) < border) return 0.0;
        const double w = row.weight(x);
        return w >= set.m ? w : 0.0;
    };
    __syncthreads();
    uint64_t total = 0;
    row.tiles([&](int i, const float(&x)[R::kVec]) {
        uint64_t sum = 0;
#pragma unroll
        for (int j = 0; j < R::kVec; ++j) sum += row.units(kept(i + j, x[j]));
        sum = group_combine<kWave>(sum, AddU64());
        const int run = i / kRun;
        if (lane == 0 && i < a.vocab) runs[run] = sum;
        total += sum;
    });
    total = block_combine(lane == 0 ? total : 0, s, AddU64());
    if (a.tokens) {
        // The first token at which the running sum reaches this.
        const double r = (double)a.r[blockIdx.x];
        const uint64_t want = r < 1.0 ? (uint64_t)(fmax(r, 0.0) * (double)total) + 1 : total;
        const int count = (a.vocab + kRun - 1) / kRun;
        constexpr int kOwn = (kMaxVocab / kRun + kThreads - 1) / kThreads;
        uint64_t own[kOwn], sum = 0;
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
            own[j] = tid * kOwn + j < count ? runs[tid * kOwn + j] : 0;
            sum += own[j];
        }
        uint64_t before = block_before(sum, s);
        if (before < want && before + sum >= want)
#pragma unroll
            for (int j = 0; j < kOwn; ++j) {
                if (before < want && before + own[j] >= want) s.bin = tid * kOwn + j, s.rest = want - before;
                before += own[j];
            }
        __syncthreads();
        if (tid < kWave) {
            const int i = (int)s.bin * kRun + lane * R::kVec;
            uint64_t w[R::kVec], mine = 0;
#pragma unroll
            for (int j = 0; j < R::kVec; ++j) {
                w[j] = i + j < a.vocab ? row.units(kept(i + j, row.seen(row.p[i + j]))) : 0;
                mine += w[j];
            }
            uint64_t upto = wave_scan(mine) - mine;
            const uint64_t rest = s.rest;
#pragma unroll
            for (int j = 0; j < R::kVec; ++j) {
                if (upto < rest && upto + w[j] >= rest) a.tokens[blockIdx.x] = i + j;
                upto += w[j];
            }
        }
    }
    if (probs) {
        const double share = row.unit / (double)total;
        row.tiles([&](int i, const float(&x)[R::kVec]) {
            typename P::bits v[R::kVec];
            // A second rounding, from float32, moves a 16-bit one by 2^-16 of its step at most.
#pragma unroll
            for (int j = 0; j < R::kVec; ++j) v[j] = P::narrow((float)(kept(i + j, x[j]) * share));
            for (int j = 0; j < R::kVec; ++j)
                if (i + j < a.vocab) probs[i + j] = v[j];
        });
    }
}

template <class T, class P>
hipError_t launch_types(const Sample& a, unsigned int rows, hipStream_t stream) {
    sample_kernel<T, P><<<rows, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

template <class T>
hipError_t launch_logits(int probs_type, const Sample& a, unsigned int rows, hipStream_t stream) {
    return probs_type == RED_F16    ? launch_types<T, F16>(a, rows, stream)
           : probs_type == RED_BF16 ? launch_types<T, BF16>(a, rows, stream)
                                    : launch_types<T, F32>(a, rows, stream);
}

}  // namespace

hipError_t launch_sample(int type, int probs_type, const Sample& a, unsigned int rows, hipStream_t stream) {
    return type == RED_F32   ? launch_logits<F32>(probs_type, a, rows, stream)
           : type == RED_F16 ? launch_logits<F16>(probs_type, a, rows, stream)
                             : launch_logits<BF16>(probs_type, a, rows, stream);
}

}  // namespace libred
