// sample_common.hpp -- sampling from a row of logits with temperature, top-k,
// top-p and min-p: what the kernels share, and the way that takes a row of any
// length by one block alone.
//
// The tokens' order (falling logits, ties by number) is that of one whole
// number a token, its code: the logit's bits, turned so that they order, above
// the number's complement. What top-k, top-p and min-p keep are the codes from
// a border on. For top-k and top-p it is the first code at which a running sum
// along the order, of ones or of weights, reaches a target, and it is found by
// sums over bins, not by sorting: first bins of equal ratios of the weight,
// down from the largest; then, for what is in the border's bin, bins of the
// codes' digits, 8 bits at a time.
//
// Weights exp((x - max) / T) are float64. Their sums are held in whole numbers
// of 2^-shift (45 bits for 131072 tokens), so they come out the same in any
// order, and atomics do no harm.
#pragma once

#include "decode_common.hpp"
#include "serve.hpp"

namespace libred {

constexpr int kThreads = 1024, kWaves = kThreads / kWave;
static_assert(kWaves == 16, "the waves' sums are joined by the lanes of a row of 16");
constexpr int kBins = 256;
constexpr int kHeld = 2048;        // codes that are gathered in the LDS
constexpr int kMaxVocab = 1 << 20;
static_assert(2 * kHeld >= kMaxVocab / (kWave * 4), "a run is what a wave reads at a time");

struct AddU64 {
    __device__ __forceinline__ uint64_t operator()(uint64_t a, uint64_t b) const { return a + b; }
};
struct MaxU64 {
    __device__ __forceinline__ uint64_t operator()(uint64_t a, uint64_t b) const { return a > b ? a : b; }
};

// Codes of logits of type T: the bits that order as they do (the key) above 20 of
// the number's complement.
template <class T>
struct Code {
    static constexpr int kKeyBits = 8 * sizeof(typename T::bits), kBits = kKeyBits + 20;
    static constexpr uint32_t kSign = 1u << (kKeyBits - 1), kMask = kSign - 1 + kSign;
    // Of the least finite logit: one above that of -inf.
    static constexpr uint32_t kLeast = sizeof(typename T::bits) == 4 ? 0x00800000u : std::is_same_v<T, F16> ? 0x0400u : 0x0080u;

    static __device__ __forceinline__ uint64_t of(float x, int i) {
        const uint32_t u = T::narrow(x);  // exact: x was of this type
        return (uint64_t)(u & kSign ? ~u & kMask : u | kSign) << 20 | (uint32_t)(kMaxVocab - 1 - i);
    }
    static __device__ __forceinline__ float logit_of_key(uint32_t k) {
        return T::widen((typename T::bits)(k & kSign ? k & ~kSign : ~k & kMask));
    }
    static __device__ __forceinline__ float logit(uint64_t code) { return logit_of_key((uint32_t)(code >> 20)); }
    static __device__ __forceinline__ int token(uint64_t code) { return kMaxVocab - 1 - (int)(code & (kMaxVocab - 1)); }

    // The first of the keys from kLeast to `top` for which `is` holds; it holds
    // for `top` and for all above one for which it does. By one wave.
    template <class F>
    static __device__ __forceinline__ uint32_t first_key(uint32_t top, F is) {
        const uint32_t lane = threadIdx.x % kWave;
        uint32_t low = kLeast, high = top;
        while (low < high) {
            const uint32_t step = (high - low) / kWave + 1, probe = min(low + lane * step, high);
            const uint64_t yes = __ballot(is(logit_of_key(probe)));
            if (!yes) {
                low = min(low + (kWave - 1) * step, high - 1) + 1;
            } else {
                const uint32_t at = (uint32_t)__ffsll((unsigned long long)yes) - 1;
                const uint32_t found = min(low + at * step, high);
                if (at > 0) low = low + (at - 1) * step + 1;
                high = found;
            }
        }
        return high;
    }
};

constexpr float kNone = -__builtin_inff();

// 2^t for t <= 0: a polynomial over half a power to either side, that is 1 at 0;
// N terms leave out 2^-55 (11) or 2^-38 (8) of it. They interpolate (2^f - 1) / f
// at the Chebyshev points. Where t is a product, f is of it before it is rounded (the
// compiler fuses the two), which for t far below the last power is anything: not used.
template <int N>
__device__ __forceinline__ double power2(double t) {
    static_assert(N == 11 || N == 8, "terms");
    if (t < -1100.0) return 0.0;
    const double n = __builtin_rint(t), f = t - n;
    double p;
    if constexpr (N == 11) {
        p = __builtin_fma(4.4549605981865186e-10, f, 7.072585949269223e-09);
        p = __builtin_fma(p, f, 1.0178062445845774e-07);
        p = __builtin_fma(p, f, 1.321544258792169e-06);
        p = __builtin_fma(p, f, 1.525273382983612e-05);
        p = __builtin_fma(p, f, 0.0001540353044173605);
        p = __builtin_fma(p, f, 0.0013333558146416936);
        p = __builtin_fma(p, f, 0.009618129107606888);
        p = __builtin_fma(p, f, 0.0555041086648216);
        p = __builtin_fma(p, f, 0.24022650695910097);
        p = __builtin_fma(p, f, 0.6931471805599453);
    } else {
        p = __builtin_fma(1.325080551750225e-06, f, 1.5303700711365693e-05);
        p = __builtin_fma(p, f, 0.00015403475186530786);
        p = __builtin_fma(p, f, 0.0013333478473685416);
        p = __builtin_fma(p, f, 0.00961812913523614);
        p = __builtin_fma(p, f, 0.055504109063258665);
        p = __builtin_fma(p, f, 0.24022650695888503);
        p = __builtin_fma(p, f, 0.6931471805568324);
    }
    return __builtin_amdgcn_ldexp(__builtin_fma(p, f, 1.0), (int)n);
}

// What the block shares: for sums and borders, and for rows and lists that are not
// held in registers.
struct Sums {
    unsigned long long mass[kBins];
    unsigned int count[kBins];
    unsigned long long part[kWaves], found, rest;
    unsigned long long few[kWave], few_own[kWave];  // what a wave takes
    unsigned int held, bin, cut;
};
struct Shared : Sums {
    union {
        struct {
            unsigned long long code[kHeld];  // what is in the border's bin
            unsigned long long own[kHeld];   // the weights of those
            unsigned long long runs[2 * kHeld];  // a row's kept weights, in runs
        };
        struct {  // where no runs are needed
            unsigned long long list[2 * kHeld], list_own[2 * kHeld];
        };
    };
};

template <class Op>
__device__ __forceinline__ uint64_t block_combine(uint64_t v, Sums& s, Op op) {
    v = group_combine<kWave>(v, op);
    __syncthreads();
    if (threadIdx.x % kWave == 0) s.part[threadIdx.x / kWave] = v;
    __syncthreads();
    return group_combine<kWaves>((uint64_t)s.part[threadIdx.x % kWaves], op);  // in every 16 lanes
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
// The sum of the threads before this one, and of all.
__device__ __forceinline__ uint64_t block_before(uint64_t v, Sums& s, uint64_t* all) {
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const uint64_t upto = wave_scan(v);
    __syncthreads();
    if (lane == kWave - 1) s.part[wave] = upto;
    __syncthreads();
    // The waves' sums, in each 16 lanes.
    const uint64_t part = s.part[lane % kWaves];
    uint64_t sums = part;
    sums += dpp_move<0x111, 0xF>((uint64_t)0, sums);
    sums += dpp_move<0x112, 0xF>((uint64_t)0, sums);
    sums += dpp_move<0x114, 0xF>((uint64_t)0, sums);
    sums += dpp_move<0x118, 0xF>((uint64_t)0, sums);
    const int own = __builtin_amdgcn_readfirstlane(wave);
    const uint64_t before = read_lane(sums, own) - read_lane(part, own), whole = read_lane(sums, kWaves - 1);
    *all = whole;
    return before + upto - v;
}

template <class T>
struct Row {
    using B = typename T::bits;
    using C = Code<T>;
    static constexpr int kVec = 4, kTile = kThreads * kVec;
    static constexpr int kRun = kWave * kVec;  // tokens that a wave reads at a time
    // Rows start on element boundaries only (a vocabulary may be odd).
    typedef B Vector __attribute__((ext_vector_type(4), aligned(sizeof(B))));

    const B* p;
    int vocab;
    bool infinite = false;  // the largest logit is +inf: those count as 0, all others as -inf
    float top_logit = 0.f;
    double top = 0.0, scale = 0.0, unit = 0.0;

    __device__ __forceinline__ Row(const Sample& a, int b, int step)
        : p(static_cast<const B*>(a.x) + b * a.batch_stride + step * a.step_stride), vocab(a.vocab) {}
    // By the first code of the order; -> it, as the row then counts.
    __device__ __forceinline__ uint64_t settle(uint64_t first, double row_scale, int shift) {
        top_logit = C::logit(first);
        infinite = top_logit == __builtin_inff();
        if (infinite) top_logit = 0.f, first = C::of(0.f, C::token(first));
        top = top_logit, scale = row_scale, unit = __builtin_ldexp(1.0, shift);
        return first;
    }

    __device__ __forceinline__ float seen(B bits) const {
        const float x = T::widen(bits) + 0.f;  // -0 is 0
        if (infinite) return x == __builtin_inff() ? 0.f : kNone;
        return x == x ? x : kNone;
    }
    // N logits from number i on, kNone behind the last.
    template <int N>
    __device__ __forceinline__ void neighbours(int i, float (&x)[N]) const {
        static_assert(N % kVec == 0, "whole vectors");
        if (i + N <= vocab) {
            Vector v[N / kVec];
#pragma unroll
            for (int u = 0; u < N / kVec; ++u) v[u] = *reinterpret_cast<const Vector*>(p + i + u * kVec);
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] = seen(v[j / kVec][j % kVec]);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] = i + j < vocab ? seen(p[i + j]) : kNone;
        }
    }
    // f(number of the first, logits) of this thread's kVec neighbours in every
    // tile of the block; kNone behind the last.
    template <class F>
    __device__ __forceinline__ void tiles(F f) const {
        for (int i0 = 0; i0 < vocab; i0 += kTile) {
            const int i = i0 + threadIdx.x * kVec;
            float x[kVec];
            neighbours<kVec>(i, x);
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
        return x == kNone ? 0.0 : power2<11>(((double)x - top) * scale);
    }
    // In units: 2^52 more than a number below it has that number as its last bits.
    __device__ __forceinline__ uint64_t units(double w) const {
        return __builtin_bit_cast(uint64_t, w * unit + 0x1p52) & 0xFFFFFFFFFFFFFull;
    }
    __device__ __forceinline__ uint64_t kept_units(int i, float x, uint64_t border) const {
        return x == kNone || C::of(x, i) < border ? 0 : units(weight(x));
    }
    // Bins of an eighth of a power of two, from the largest weight down. The
    // order of the logits holds after each rounding.
    __device__ __forceinline__ int bin(float x) const {
        const double d = (top - (double)x) * scale * 8.0;
        return d < (double)(kBins - 1) ? (int)d : kBins - 1;
    }
};

// The bin in which the running sum of the bins' reaches `target`, the last that
// is not empty where it does not, kBins if all are; and what is missing of the
// target there.
__device__ __forceinline__ void find_bin(Sums& s, uint64_t target, bool codes) {
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
        const uint64_t whole = read_lane(upto, kWave - 1);
        target = target < whole ? target : whole;
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

__device__ __forceinline__ void clear_bins(Sums& s) {
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += kThreads) s.mass[i] = 0, s.count[i] = 0;
    __syncthreads();
}

// Of up to kWave codes and their weights, one a lane (0: none): the code at which
// the sum of the weights, in the order of the codes, reaches `want`, the last where
// it does not; ~0 for none. By a wave; -> in all lanes.
__device__ __forceinline__ uint64_t rank_border(uint64_t c, uint64_t own, int n, uint64_t want) {
    uint64_t before = 0, all = 0;
    for (int i = 0; i < n; ++i) {
        const uint64_t other = read_lane(own, i);
        all += other;
        before += read_lane(c, i) > c ? other : 0;
    }
    want = want > 0 ? want : 1;
    const uint64_t goal = want < all ? want : all, is = __ballot(own > 0 && before < goal && before + own >= goal);
    return is ? read_lane(c, __ffsll((unsigned long long)is) - 1) : ~0ull;
}

// What a running sum of weights must reach for top-p.
__device__ __forceinline__ uint64_t top_p_target(double p, uint64_t all) {
    const uint64_t want = (uint64_t)__builtin_ceil(p * (double)all);
    return want > 0 ? want : 1;
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
        if (x == kNone || Code<T>::of(x, i) < from) return;
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
    int shift = Code<T>::kBits;
    uint64_t prefix = 0;
    auto inside = [&](uint64_t code, float x) { return x != kNone && code >= from && row.bin(x) == bin && code >> shift == prefix; };
    while (in > kHeld && shift > 0) {
        const int width = min(shift, 8), down = shift - width;
        clear_bins(s);
        row.each([&](int i, float x) {
            const uint64_t code = Code<T>::of(x, i);
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
        const uint64_t code = Code<T>::of(x, i);
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
    __device__ __forceinline__ Settings(const Sample& a, int b) {
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


// The border of what a row keeps, `first` being the first code of the order.
template <class T>
__device__ __forceinline__ uint64_t row_border(const Row<T>& row, Shared& s, const Settings& set, uint64_t first) {
    if (set.k == 1) return first;
    uint64_t border = 0;
    if (set.k < row.vocab) border = find_border(row, s, 0, [](float) -> uint64_t { return 1; }, [&](uint64_t) { return (uint64_t)set.k; });
    if (set.p < 2.0) {
        const uint64_t found = find_border(row, s, border, [&](float x) { return row.units(row.weight(x)); },
                                           [&](uint64_t all) { return top_p_target(set.p, all); });
        border = found > border ? found : border;
    }
    if (set.m > 0.0) {
        __syncthreads();
        if (threadIdx.x < kWave) {
            const uint32_t cut = Code<T>::first_key((uint32_t)(first >> 20), [&](float x) { return row.weight(x) >= set.m; });
            if (threadIdx.x == 0) s.cut = cut;
        }
        __syncthreads();
        const uint64_t cut = (uint64_t)s.cut << 20;
        border = cut > border ? cut : border;
    }
    return border;
}

// The sum of the kept weights, and in s.runs those of the tokens a wave reads at
// a time.
template <class T>
__device__ __forceinline__ uint64_t row_total(const Row<T>& row, Shared& s, uint64_t border) {
    using R = Row<T>;
    const int lane = threadIdx.x % kWave;
    uint64_t total = 0;
    __syncthreads();
    row.tiles([&](int i, const float(&x)[R::kVec]) {
        uint64_t sum = 0;
#pragma unroll
        for (int j = 0; j < R::kVec; ++j) sum += row.kept_units(i + j, x[j], border);
        sum = group_combine<kWave>(sum, AddU64());
        if (lane == 0 && i < row.vocab) s.runs[i / R::kRun] = sum;
        total += sum;
    });
    return block_combine(lane == 0 ? total : 0, s, AddU64());
}

// What the running sum of the kept weights must reach for the token.
__device__ __forceinline__ uint64_t draw_target(float r, uint64_t total) {
    return r < 1.f ? (uint64_t)(fmax((double)r, 0.0) * (double)total) + 1 : total;
}

// The token at which it does, by the sums of the runs.
template <class T>
__device__ __forceinline__ void row_draw(const Row<T>& row, Shared& s, uint64_t border, uint64_t want, int64_t* token) {
    using R = Row<T>;
    constexpr int kOwn = kMaxVocab / R::kRun / kThreads;
    const int tid = threadIdx.x, count = (row.vocab + R::kRun - 1) / R::kRun;
    uint64_t own[kOwn], sum = 0;
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
        own[j] = tid * kOwn + j < count ? s.runs[tid * kOwn + j] : 0;
        sum += own[j];
    }
    uint64_t all;
    if (tid == 0) s.bin = 0, s.rest = 1;  // a place in the row whatever the sums are
    uint64_t before = block_before(sum, s, &all);
    if (before < want && before + sum >= want)
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
            if (before < want && before + own[j] >= want) s.bin = tid * kOwn + j, s.rest = want - before;
            before += own[j];
        }
    __syncthreads();
    if (tid < kWave) {
        const int i = (int)s.bin * R::kRun + tid * R::kVec;
        float x[R::kVec];
        row.template neighbours<R::kVec>(i, x);
        uint64_t w[R::kVec], mine = 0;
#pragma unroll
        for (int j = 0; j < R::kVec; ++j) {
            w[j] = row.kept_units(i + j, x[j], border);
            mine += w[j];
        }
        uint64_t upto = wave_scan(mine) - mine;
        const uint64_t rest = s.rest;
#pragma unroll
        for (int j = 0; j < R::kVec; ++j) {
            if (upto < rest && upto + w[j] >= rest) *token = i + j;
            upto += w[j];
        }
    }
}

}  // namespace libred
