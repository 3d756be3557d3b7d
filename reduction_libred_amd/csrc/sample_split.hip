// Sampling: rows cut into chunks, in three or four launches (one more with
// probabilities).
//
//  1. bins: a block a chunk of 8192 logits, held in registers. Every logit
//     goes into a bin of an eighth of a power of two of its weight: with y = 8
//     log2(e) x / T the bin is floor(y), so the bins of all chunks line up
//     whatever their largest logits are, and a chunk needs no other's. A bin
//     has the number of its logits and the sum of their weights, relative to
//     the bin's upper edge, in whole numbers of 2^-36, as one 64-bit number of
//     the LDS. This is the only time that every weight is computed: by a
//     polynomial in the place in the bin, 2^((f - 1) / 8).
//  2. find: a block a row adds up the chunks' bins and finds those in which the
//     borders of top-k, top-p and min-p lie, as ranges of logits.
//  3. gather: the codes of the logits in these ranges, a few thousand; a
//     second read of the row, with two comparisons a logit. Few rows, or short
//     ones: in the launch before.
//  4. draw: a block a row finds the border among them, the chunk in which the
//     running sum of the kept weights passes its target, by the chunks' bins,
//     and the token in that chunk.
//  5. probabilities.
//
// Microseconds of bins / find / gather / draw (/ probabilities): one row of 32000
// float32, top-k 50 and top-p, 4.6 / 8.8 with the gathering / 10.2; 192 rows of 131071, top-p, 22.8 /
// 7.7 / 18.9 / 21.1; 224 rows of bfloat16, top-p and min-p, 25.4 / 8.2 / 13.7 / 16.7 /
// 34.2. The bins take turns at the read (the 100 MB alone 14), 22 vector
// instructions a logit, half of them float64 (two thirds of the cycles), and an LDS
// atomic each (two fifths): 17 instructions a logit took 23, blocks that go through
// several chunks with the next one's logits on their way 24 to 27. The gathering and
// the probabilities are bound by memory (5.4 and 5.3 TB/s); find and draw by their
// latency, a block a row, the draw by the longest list (6000 codes where 1000 are
// usual). Finding, gathering and drawing in one launch of a block a row: 55 instead
// of 47 for the 192 rows, 23 instead of 20 for the one.
//
// Where more logits than kList are near a border, or the border is further than 64
// powers of two below the largest weight, the block that draws goes through the whole
// row instead, once for every step of every border. That is rows of thousands of equal
// logits, and flat rows of distinct ones: logits of spread 1 and top-p 0.9 from 262144
// tokens at temperature 3 on (1 row 580 us, at temperature 2 47) and at 2^20 tokens from
// 0.7 on (2.2 ms at temperature 1, 48 us at 0.3); 64 rows take little longer than one.
#include "sample_common.hpp"

namespace libred {

namespace {

constexpr int kOwn = 32;                  // logits of a thread that holds a part of a row
constexpr int kGrid = kSampleGrid;       // bins: 64 powers of two
constexpr double kPerPower = 8.0;        // bins a power of two
// A bin adds up doubles 2^52 + v by their bits: v, the relative weight in units
// of 2^-36, in the low 52, and in the others 0x433 for each, modulo 2^12.
constexpr uint64_t kSumMask = ((uint64_t)1 << 52) - 1;
constexpr unsigned int kInverse = 1787;  // of 0x433, modulo 2^12
static_assert(0x433 * kInverse % 4096 == 1 && kSampleChunk <= 32768, "a bin's number can be told");

// How many were added: known modulo 2^12, at least the sum and at most 2^(1/8)
// times it, which leaves one number up to 32768.
__device__ __forceinline__ unsigned int count_of(uint64_t bin) {
    const uint64_t sum = bin & kSumMask;
    const unsigned int least = (unsigned int)((sum + ((1ull << 36) - 1)) >> 36), n = (unsigned int)(bin >> 52) * kInverse & 4095u;
    return least + ((n - least) & 4095u);
}

// What a logit is on the grid of a row.
struct Place {
    double scale;  // 8 log2(e) / T
    __device__ __forceinline__ double floor_of(float x) const { return __builtin_floor((double)x * scale); }
    // From the bin's lower edge, by the product before it is rounded.
    __device__ __forceinline__ double in_bin(float x, double floor) const { return __builtin_fma((double)x, scale, -floor); }
    // Whether the bins' numbers are small enough for all that is done with them: of
    // a row by its largest logit, and of a chunk, with room for any that is on the
    // grid of a row for which they are.
    __device__ __forceinline__ bool fits(float top) const { return __builtin_fabs((double)top * scale) < 0x1p26; }
    __device__ __forceinline__ bool chunk_fits(float top) const { return __builtin_fabs((double)top * scale) < 0x1p27; }
};

// 2^52 + 2^36 2^((f - 1) / 8) for the place f in its bin, rounded to a whole
// number. The polynomial interpolates at the Chebyshev points of the bin and is
// off by 2^-41 of the weight. Its coefficients are kept in scalar registers: as
// constants the compiler moves each into vector registers for each logit, as
// many instructions as the rest.
struct Relative {
    double c0 = 0x1p36 * 0.9170040432043982 + 0x1p52, c1 = 0x1p36 * 0.07945234590833129, c2 = 0x1p36 * 0.003442010367212629,
           c3 = 0x1p36 * 9.941014004467738e-05, c4 = 0x1p36 * 2.1514114906866102e-06, c5 = 0x1p36 * 3.896824607481367e-08;
    __device__ __forceinline__ Relative() { asm("" : "+s"(c0), "+s"(c1), "+s"(c2), "+s"(c3), "+s"(c4), "+v"(c5)); }
    __device__ __forceinline__ uint64_t units(double f) const {
        double r = __builtin_fma(c5, f, c4);
        r = __builtin_fma(r, f, c3);
        r = __builtin_fma(r, f, c2);
        r = __builtin_fma(r, f, c1);
        return __builtin_bit_cast(uint64_t, __builtin_fma(r, f, c0));
    }
};

template <class T, int THREADS>
struct Loads {
    using B = typename T::bits;
    static constexpr int kVec = 16 / sizeof(B), kCount = kOwn / kVec, kAll = THREADS * kOwn;
    typedef B Vector __attribute__((ext_vector_type(16 / sizeof(B)), aligned(sizeof(B))));
    Vector v[kCount];

    // kAll logits from number `first` on, those of thread tid: kVec neighbours
    // every THREADS * kVec. Behind the last: -inf. (A chunk
    // that the row ends in is read by vectors too, but for the one that the end
    // is in: element by element it took as long as all others, 26 us / 16 of 192
    // rows of 131071.)
    Loads() = default;
    __device__ __forceinline__ Loads(const B* p, int first, int vocab) {
        const int tid = threadIdx.x;
        auto place = [&](int u) { return first + (u * THREADS + tid) * kVec; };
#pragma unroll
        for (int u = 0; u < kCount; ++u) v[u] = *reinterpret_cast<const Vector*>(p + (place(u) + kVec <= vocab ? place(u) : 0));
        if (first + kAll > vocab)
#pragma unroll
            for (int u = 0; u < kCount; ++u)
                if (place(u) + kVec > vocab)
#pragma unroll
                    for (int j = 0; j < kVec; ++j) v[u][j] = place(u) + j < vocab ? p[place(u) + j] : T::narrow(kNone);
    }
    __device__ __forceinline__ float at(int n) const { return T::widen(v[n / kVec][n % kVec]); }
    __device__ __forceinline__ static int number(int n) { return (n / kVec * THREADS + threadIdx.x) * kVec + n % kVec; }
};

// Every logit of `x` into its bin: a logit below the grid goes to a place of its lane's behind it, without
// a branch. Bins go by their negative numbers, that rise from the first bin down.
template <class L>
__device__ __forceinline__ void fill_bins(const L& x, const Place& place, double peak, unsigned long long* bins) {
    const Relative relative;
    const double up = -place.scale, end = kGrid - peak;
    const int aside = (kGrid + (int)threadIdx.x % kWave) * 8, base = (int)peak * 8;
#pragma unroll
    for (int n = 0; n < kOwn; ++n) {
        const double v = (double)x.at(n), g = __builtin_ceil(v * up);
        const int to = g < end ? ((int)g << 3) + base : aside;
        atomicAdd(reinterpret_cast<unsigned long long*>(reinterpret_cast<char*>(bins) + to),
                  (unsigned long long)relative.units(__builtin_fma(v, place.scale, g)));
    }
}

// The probabilities of the logits that a thread holds, which begin at number
// `first` of the row.
template <class P, class T, int THREADS>
__device__ __forceinline__ void write_probs(const Row<T>& row, const Loads<T, THREADS>& x, int first, uint64_t border, double share,
                                            typename P::bits* probs) {
    using L = Loads<T, THREADS>;
    typedef typename P::bits Out __attribute__((ext_vector_type(L::kVec), aligned(sizeof(typename P::bits))));
#pragma unroll
    for (int u = 0; u < L::kCount; ++u) {
        const int i0 = first + L::number(u * L::kVec);
        Out v;
#pragma unroll
        for (int j = 0; j < L::kVec; ++j) {
            const float f = row.seen(x.v[u][j]);
            const bool kept = f != kNone && Code<T>::of(f, i0 + j) >= border;
            // A second rounding, from float32, moves a 16-bit one by 2^-16 of its step at most.
            float w = 0.f;
            if (__any(kept) && kept) w = (float)(power2<8>(((double)f - row.top) * row.scale) * share);
            v[j] = P::narrow(w);
        }
        if (i0 + L::kVec <= row.vocab) {
            *reinterpret_cast<Out*>(probs + i0) = v;
        } else {
#pragma unroll
            for (int j = 0; j < L::kVec; ++j)
                if (i0 + j < row.vocab) probs[i0 + j] = v[j];
        }
    }
}

// Running sum over the wave's lanes, this one's value included.
__device__ __forceinline__ unsigned int count_scan(unsigned int v) {
    v += dpp_move<0x111, 0xF>(0u, v);
    v += dpp_move<0x112, 0xF>(0u, v);
    v += dpp_move<0x114, 0xF>(0u, v);
    v += dpp_move<0x118, 0xF>(0u, v);
    v += dpp_move<0x142, 0xA>(0u, v);
    v += dpp_move<0x143, 0xC>(0u, v);
    return v;
}

// What the block that finds shares.
struct Found {
    unsigned long long mass[kGrid];  // weights of the bins up to one, in units
    unsigned int count[kGrid];       // their numbers
    unsigned long long part[kGrid / kWave];
    unsigned int parts[kGrid / kWave];
    int first[4];
    unsigned int edge[4], cut;
};

// The first bin for which `is` holds, kGrid if for none; slot `at` is used once.
__device__ __forceinline__ int first_bin(Found& s, int at, bool is) {
    const uint64_t yes = __ballot(is);
    if (threadIdx.x % kWave == 0 && yes) atomicMin(&s.first[at], (int)threadIdx.x + __ffsll((unsigned long long)yes) - 1);
    __syncthreads();
    return s.first[at];
}

// A bin's sum in units of the largest weight, whose own relative units are
// `largest`; norm: unit / largest; factor: 2^(-bin / 8). Where all of it are of
// that weight it is exact, so that a row of equal logits has exact sums.
__device__ __forceinline__ uint64_t scaled(uint64_t v, double norm, double factor, uint64_t largest, uint64_t unit, bool first) {
    const uint64_t sum = v & kSumMask;
    uint64_t of = (uint64_t)((double)sum * (norm * factor));
    if (first) {
        const unsigned int n = count_of(v);
        if (n * largest == sum) of = n * unit;
    }
    return of;
}

// Where the borders of a row are: its ranges of logits to be gathered, `most_held`
// of them at most, and what the draw needs to know of the bins, in `plan`. `sum`
// and `count` are those of bin tid.
template <class T>
__device__ __forceinline__ void find_ranges(const Row<T>& row, const Settings& set, const SampleHead& head, uint64_t sum, unsigned int count,
                                            unsigned int most_held, Found& s, SamplePlan& plan) {
    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const Place place{set.scale * kPerPower};
    const float top = row.top_logit;
    const double peak = place.floor_of(top);
    const uint64_t largest = Relative().units(place.in_bin(top, peak)) & kSumMask, unit = (uint64_t)row.unit;
    const double norm = row.unit / (double)largest;
    uint64_t mass = (uint64_t)((double)sum * (norm * power2<11>(-(double)tid / kPerPower)));
    if (tid == 0 && count * largest == sum) mass = count * unit;  // all of the largest weight: exact
    const unsigned int own_count = count;
    mass = wave_scan(mass);
    count = count_scan(count);
    __syncthreads();
    if (lane == kWave - 1) s.part[wave] = mass, s.parts[wave] = count;
    __syncthreads();
    for (int w = 0; w < wave; ++w) mass += s.part[w], count += s.parts[w];
    s.mass[tid] = mass, s.count[tid] = count;
    // The least logit that min-p keeps.
    if (wave == 0 && set.m > 0.0) {
        const uint32_t cut = Code<T>::first_key((uint32_t)(head.first >> 20), [&](float x) { return row.weight(x) >= set.m; });
        if (lane == 0) s.cut = cut;
    }
    __syncthreads();
    const uint64_t all = s.mass[kGrid - 1];
    int state = kRowCut;
    const bool has_k = set.k < head.count, has_p = set.p < 2.0;
    // Bins in which the borders lie: top-k's; from `low` to `high` those in which
    // top-p's may (its target is known to 2^-30, or as far as the bin of top-k's
    // border is unresolved).
    int kbin = kGrid, low = kGrid, high = -1;
    if (has_k) {
        kbin = first_bin(s, 0, count >= (unsigned int)set.k);
        if (kbin == kGrid) state = kRowWhole;
    }
    uint64_t before_k = 0;
    if (has_k && state == kRowCut) before_k = kbin > 0 ? s.mass[kbin - 1] : 0;
    if (has_p && state == kRowCut) {
        const double least = has_k ? (double)before_k : (double)all, most = has_k ? (double)s.mass[kbin] : (double)all;
        const double from = set.p * least * (1.0 - 0x1p-30), upto = set.p * most * (1.0 + 0x1p-30);
        low = first_bin(s, 1, (double)mass >= from && own_count > 0);
        high = first_bin(s, 2, (double)mass >= upto);
        if (has_k) low = min(low, kbin), high = min(high, kbin);
        if (low == kGrid || high == kGrid) state = kRowWhole;
    }
    if (!has_p && has_k) low = high = kbin;
    bool use_k = has_k, use_p = has_p;
    uint64_t cut = 0;
    if (state == kRowCut && set.m > 0.0) {
        cut = (uint64_t)s.cut << 20;
        const double d = peak - place.floor_of(Code<T>::logit(cut));
        const int mbin = d < (double)kGrid ? (int)d : kGrid;
        if (mbin < low || high < 0) {
            // min-p keeps fewer than the others, or is alone.
            if (mbin == kGrid) state = kRowWhole;
            low = high = mbin, use_k = use_p = false;
        }
    }
    // Ranges of bins: low .. high, and top-k's where that is below and needed.
    const bool second = use_p && use_k && kbin > high;
    int ranges = state != kRowCut || high < 0 ? 0 : second ? 2 : 1;
    if (ranges > 0) {
        unsigned int n = s.count[high] - (low > 0 ? s.count[low - 1] : 0);
        if (second) n += s.count[kbin] - s.count[kbin - 1];
        if (n > most_held) state = kRowWhole, ranges = 0;
    }
    // Their logits: from the first of the last bin to below the first of the bin
    // before the first.
    if (wave < 2 * ranges) {
        const int bin = wave == 0 ? high : wave == 1 ? low - 1 : wave == 2 ? kbin : kbin - 1;
        const uint32_t key = (uint32_t)(head.first >> 20);
        const uint32_t edge = bin < 0 ? key + 1 : Code<T>::first_key(key, [&](float x) { return peak - place.floor_of(x) <= (double)bin; });
        if (lane == 0) s.edge[wave] = edge;
    }
    __syncthreads();
    if (tid == 0) {
        plan.state = state, plan.ranges = ranges;
        plan.use_k = use_k && ranges > 0, plan.use_p = use_p && ranges > 0;
        plan.cut = cut;
        for (int r = 0; r < ranges; ++r) plan.from[r] = Code<T>::logit_of_key(s.edge[2 * r]), plan.upto[r] = Code<T>::logit_of_key(s.edge[2 * r + 1]);
        plan.low = low, plan.high = high;
        const int before = second ? kbin : low;  // bins before the range that has top-k's border
        plan.k_rest = use_k && ranges > 0 ? (uint64_t)set.k - (before > 0 ? s.count[before - 1] : 0) : 0;
        plan.k_before = before_k;
        plan.p_before = low > 0 && low < kGrid ? s.mass[low - 1] : 0;
        plan.all = all;
        plan.norm = norm, plan.largest = largest;
    }
}

// The least code of a logit.
template <class T>
__device__ __forceinline__ uint64_t first_code(float x) {
    return Code<T>::of(x, kMaxVocab - 1);
}

// The codes of a list: the first kFast of them with their weights in the LDS, the
// others in memory.
constexpr int kFast = 2 * kHeld;
template <class T>
struct List {
    const Row<T>& row;
    Shared& s;
    const unsigned long long* rest;
    int n;
    __device__ __forceinline__ uint64_t units(uint64_t c) const { return row.units(row.weight(Code<T>::logit(c))); }
    // f(code, weight) of all, weight() what it weighs.
    template <class F>
    __device__ __forceinline__ void each(F f) const {
        for (int i = threadIdx.x; i < min(n, kFast); i += kThreads) f(s.list[i], [&]() -> uint64_t { return s.list_own[i]; });
        if (n <= kFast) return;
        uint64_t next = rest[min(kFast + (int)threadIdx.x, n - 1)];
#pragma unroll 1
        for (int i = kFast + threadIdx.x; i < n; i += kThreads) {
            const uint64_t c = next;
            next = rest[min(i + kThreads, n - 1)];
            f(c, [&]() -> uint64_t { return units(c); });
        }
    }
};

// The code at which the running sum of the list's weights (`ones`: of ones), in
// the order of the codes, among those from `from` to below `upto`, reaches `want`,
// the last of them where it does not; ~0 where there are none. By bins of equal
// numbers of codes, 129 to 256 of them, and again in the border's bin, until a wave
// can take the rest. (Digits of 8 bits fell into few bins, one even, where the codes
// pass a power of two.) By the block.
template <class T>
__device__ __forceinline__ uint64_t list_border(const List<T>& list, uint64_t from, uint64_t upto, uint64_t want, bool ones) {
    if (from >= upto) return ~0ull;
    Shared& s = list.s;
    const int tid = threadIdx.x, lane = tid % kWave;
    unsigned int in = list.n;
    auto inside = [&](uint64_t c) { return c >= from && c < upto; };
    want = want > 0 ? want : 1;
    while (in > kWave) {
        const int bits = 64 - __builtin_clzll((upto - from - 1) | 1), to = bits > 8 ? bits - 8 : 0;
        clear_bins(s);
        list.each([&](uint64_t c, auto weight) {
            if (!inside(c)) return;
            const int d = (int)((c - from) >> to);
            atomicAdd(&s.mass[d], (unsigned long long)(ones ? 1 : weight()));
            atomicAdd(&s.count[d], 1u);
        });
        find_bin(s, want, true);
        if (s.bin >= kBins) return ~0ull;
        from += (uint64_t)s.bin << to;
        upto = upto - from < (1ull << to) ? upto : from + (1ull << to);
        want = s.rest, in = s.count[s.bin];
    }
    __syncthreads();
    if (tid == 0) s.held = 0;
    __syncthreads();
    list.each([&](uint64_t c, auto weight) {
        if (!inside(c)) return;
        const unsigned int at = atomicAdd(&s.held, 1u);
        if (at < kWave) s.few[at] = c, s.few_own[at] = ones ? 1 : weight();
    });
    __syncthreads();
    if (tid < kWave) {
        const int held = min((int)s.held, kWave);
        const uint64_t found = rank_border(lane < held ? s.few[lane] : 0, lane < held ? s.few_own[lane] : 0, held, want);
        if (lane == 0) s.found = found;
    }
    __syncthreads();
    return s.found;
}

// The border of a row from its plan: search(from, upto, want, ones) is the code at
// which a sum is reached, kept_sum(from, upto) the weights of the list's codes from
// `from` to below `upto`. above: the first code above those gathered for it.
template <class T, class F, class G>
__device__ __forceinline__ uint64_t border_of(const Settings& set, const SamplePlan& plan, uint64_t above, F search, G kept_sum) {
    const uint64_t from0 = first_code<T>(plan.from[0]);
    const bool two = plan.ranges == 2;
    const uint64_t k_from = two ? first_code<T>(plan.from[1]) : from0, k_upto = two ? first_code<T>(plan.upto[1]) : above;
    uint64_t border = 0;
    if (plan.use_k) border = search(k_from, k_upto, plan.k_rest, true);
    if (plan.use_p) {
        // What top-k keeps: bins above the last range, and of that what is above the
        // border.
        const uint64_t all = plan.use_k ? (two ? plan.k_before : plan.p_before) + kept_sum(border, k_upto) : plan.all;
        const uint64_t want = top_p_target(set.p, all), from = from0 > border ? from0 : border;
        const uint64_t found = want > plan.p_before ? search(from, above, want - plan.p_before, false) : above;
        border = found == ~0ull ? above : found > border ? found : border;
    }
    return plan.cut > border ? plan.cut : border;
}

// That border; what a wave can rank, one wave does for the block: with 16 at it each
// instruction takes four times as long.
template <class T>
__device__ __forceinline__ uint64_t cut_border(const List<T>& of, const Settings& set, const SamplePlan& plan, uint64_t above) {
    Shared& s = of.s;
    const int lane = threadIdx.x % kWave;
    if (of.n <= kWave) {
        if (threadIdx.x < kWave) {
            const uint64_t c = lane < of.n ? s.list[lane] : 0, w = lane < of.n ? s.list_own[lane] : 0;
            auto is = [&](uint64_t from, uint64_t upto) { return lane < of.n && c >= from && c < upto; };
            const uint64_t border = border_of<T>(
                set, plan, above,
                [&](uint64_t from, uint64_t upto, uint64_t want, bool ones) {
                    return rank_border(is(from, upto) ? c : 0, is(from, upto) ? ones ? 1 : w : 0, of.n, want);
                },
                [&](uint64_t from, uint64_t upto) { return group_combine<kWave>(is(from, upto) ? w : 0, AddU64()); });
            if (lane == 0) s.found = border;
        }
        __syncthreads();
        return s.found;
    }
    return border_of<T>(
        set, plan, above, [&](uint64_t from, uint64_t upto, uint64_t want, bool ones) { return list_border(of, from, upto, want, ones); },
        [&](uint64_t from, uint64_t upto) {
            uint64_t sum = 0;
            of.each([&](uint64_t c, auto weight) {
                if (c >= from && c < upto) sum += weight();
            });
            return block_combine(sum, s, AddU64());
        });
}

constexpr int kChunk = kSampleChunk, kChunkThreads = kChunk / kOwn;
static_assert(kChunkThreads == 256, "a block of four waves");
constexpr int kList = kSampleList;
template <class T>
using Chunk = Loads<T, kChunkThreads>;

template <class T>
__global__ __launch_bounds__(kChunkThreads) void sample_bins_kernel(Sample a) {
    constexpr int W = kChunkThreads / kWave;
    __shared__ __align__(16) unsigned long long bins[kGrid + kWave];
    __shared__ float tops[W];
    __shared__ int numbers[W], counts[W];
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int at = a.first_row + blockIdx.y, b = at / a.steps, step = at - b * a.steps, first = blockIdx.x * kChunk;
    const typename T::bits* p = static_cast<const typename T::bits*>(a.x) + b * a.batch_stride + step * a.step_stride;
    const Chunk<T> x(p, first, a.vocab);
    const Settings set(a, b);
    for (int i = tid; i < kGrid; i += kChunkThreads) bins[i] = 0;  // those behind are not read
    // The largest logit; a NaN is none. (A signalling one is made quiet first: of it the
    // hardware's maximum makes a quiet one in place of what came before it, and bins go
    // by their distance from the largest.)
    float top = kNone;
#pragma unroll
    for (int n = 0; n < kOwn; ++n) top = fmaxf(top, __builtin_canonicalizef(x.at(n)));
    top = group_combine<kWave>(top, [](float m, float n) { return fmaxf(m, n); });
    if (lane == 0) tops[wave] = top;
    __syncthreads();
    top = tops[0];
#pragma unroll
    for (int w = 1; w < W; ++w) top = fmaxf(top, tops[w]);
    const Place place{set.scale * kPerPower};
    const bool binned = set.k != 1 && place.chunk_fits(top);
    int number = kOwn, count = 0;
    if (binned) {
        fill_bins(x, place, place.floor_of(top), bins);
        if (set.k < a.vocab)
#pragma unroll
            for (int n = 0; n < kOwn; ++n) count += x.at(n) > kNone ? 1 : 0;
    }
    // The largest logit's first number.
#pragma unroll
    for (int n = kOwn - 1; n >= 0; --n) number = x.at(n) == top ? n : number;
    number = number < kOwn ? Chunk<T>::number(number) : kChunk;
    number = group_combine<kWave>(number, [](int m, int n) { return min(m, n); });
    count = group_combine<kWave>(count, [](int m, int n) { return m + n; });
    if (lane == 0) numbers[wave] = number, counts[wave] = count;
    __syncthreads();
    const int64_t chunk = (int64_t)blockIdx.y * a.chunks + blockIdx.x;
    if (tid == 0) {
        for (int w = 1; w < W; ++w) number = min(number, numbers[w]), count += counts[w];
        a.heads[chunk] = SampleHead{Code<T>::of(top + 0.f, first + (number < kChunk ? number : 0)), count};
        if (blockIdx.x == 0) a.plans[blockIdx.y].held = 0;
    }
    if (binned)
        for (int i = tid; i < kGrid / 2; i += kChunkThreads)
            reinterpret_cast<u32x4*>(a.bins + chunk * kGrid)[i] = reinterpret_cast<const u32x4*>(bins)[i];
}

__device__ __forceinline__ SampleHead row_head(const SampleHead* heads, int chunks, unsigned long long* lds, unsigned int* lds32) {
    const int waves = blockDim.x / kWave;
    uint64_t first = 0;
    int count = 0;
    for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
        const SampleHead h = heads[c];
        first = h.first > first ? h.first : first;
        count += h.count;
    }
    first = group_combine<kWave>(first, MaxU64());
    count = group_combine<kWave>(count, [](int m, int n) { return m + n; });
    if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = first, lds32[threadIdx.x / kWave] = (unsigned)count;
    __syncthreads();
    count = 0, first = 0;
    for (int w = 0; w < waves; ++w) first = lds[w] > first ? lds[w] : first, count += (int)lds32[w];
    return SampleHead{first, count};
}

// How far the bins of a chunk whose largest logit has this code are below the
// row's; kGrid and more: none of them counts.
template <class T>
__device__ __forceinline__ int chunk_shift(const Place& place, double peak, uint64_t code) {
    const float x = Code<T>::logit(code);
    const double d = x > kNone ? peak - place.floor_of(x) : (double)kGrid;
    return d < (double)kGrid ? (int)d : kGrid;
}

// The codes of the logits that a thread holds, which begin at number `first` of the
// row, and lie in the ranges of `plan`, go into the row's list.
template <class T, int THREADS>
__device__ __forceinline__ void gather(const Loads<T, THREADS>& x, int first, const SamplePlan& plan, const typename T::bits* p,
                                       unsigned int* held, unsigned long long* list) {
    constexpr int W = THREADS / kWave;
    __shared__ unsigned int counts[W], start;
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    uint32_t in = 0;
    static_assert(kOwn <= 32, "a bit a logit");
    const int ranges = plan.ranges;
    const float from0 = plan.from[0], upto0 = plan.upto[0], from1 = plan.from[1], upto1 = plan.upto[1];
    for (int r = 0; r < ranges; ++r) {
        const float from = r ? from1 : from0, upto = r ? upto1 : upto0;
#pragma unroll
        for (int n = 0; n < kOwn; ++n) {
            const float v = x.at(n);
            in |= v >= from && v < upto ? 1u << n : 0u;
        }
    }
    // Places in the list: this thread's behind those of the threads before.
    const unsigned int own = (unsigned)__popc(in), upto = count_scan(own);
    if (lane == kWave - 1) counts[wave] = upto;
    __syncthreads();
    unsigned int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        if (w == wave) before = all;
        all += counts[w];
    }
    if (all == 0) return;
    if (tid == 0) start = atomicAdd(held, all);
    __syncthreads();
    unsigned int to = start + before + upto - own;
    // Few have any: read again rather than chosen among registers.
    while (in) {
        const int n = __ffs(in) - 1, i = first + Loads<T, THREADS>::number(n);
        if (to < kList) list[to] = Code<T>::of(T::widen(p[i]) + 0.f, i);
        ++to, in &= in - 1;
    }
}

// The plan of a row, by one block; or by one for each 16384 logits, which then
// gathers from these.
template <class T>
__global__ __launch_bounds__(kGrid) void sample_find_kernel(Sample a, bool gathers) {
    using L = Loads<T, kGrid>;
    __shared__ Found s;
    __shared__ SamplePlan plan;
    __shared__ int shifts[kMaxVocab / kChunk];
    const int tid = threadIdx.x, first = blockIdx.x * L::kAll;
    const int at = a.first_row + blockIdx.y, b = at / a.steps, step = at - b * a.steps;
    Row<T> row(a, b, step);
    L x;
    if (gathers) x = L(row.p, first, a.vocab);  // before the plan is known: one trip
    const Settings set(a, b);
    const SampleHead* heads = a.heads + (int64_t)blockIdx.y * a.chunks;
    const SampleHead head = row_head(heads, a.chunks, s.part, s.parts);
    const float top = Code<T>::logit(head.first);
    const int state = top == kNone ? kRowNone : set.k == 1 ? kRowOne : !Place{set.scale * kPerPower}.fits(top) ? kRowWhole : kRowCut;
    if (tid < 4) s.first[tid] = kGrid;
    if (tid == 0) plan.first = head.first, plan.state = state, plan.ranges = 0;
    if (state == kRowCut) {
        row.settle(head.first, set.scale, a.shift);
        const Place place{set.scale * kPerPower};
        const double peak = place.floor_of(top);
        for (int c = tid; c < a.chunks; c += kGrid) shifts[c] = chunk_shift<T>(place, peak, heads[c].first);
        __syncthreads();
        // Bin tid of the row.
        uint64_t sum = 0;
        unsigned int count = 0;
        const unsigned long long* bins = a.bins + (int64_t)blockIdx.y * a.chunks * kGrid;
        for (int c0 = 0; c0 < a.chunks; c0 += 8) {
            uint64_t v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int c = min(c0 + u, a.chunks - 1), j = tid - shifts[c];
                v[u] = bins[(int64_t)c * kGrid + max(j, 0)];
                if (j < 0 || c0 + u >= a.chunks) v[u] = 0;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) sum += v[u] & kSumMask, count += count_of(v[u]);
        }
        find_ranges(row, set, head, sum, count, kList, s, plan);
    }
    __syncthreads();
    SamplePlan& to = a.plans[blockIdx.y];
    if (blockIdx.x == 0 && tid == 0) {
        to.first = plan.first, to.state = plan.state, to.ranges = plan.ranges, to.use_k = plan.use_k, to.use_p = plan.use_p, to.cut = plan.cut;
        for (int r = 0; r < 2; ++r) to.from[r] = plan.from[r], to.upto[r] = plan.upto[r];
        to.low = plan.low, to.high = plan.high, to.k_rest = plan.k_rest, to.k_before = plan.k_before, to.p_before = plan.p_before;
        to.all = plan.all, to.norm = plan.norm, to.largest = plan.largest;
    }
    if (gathers && plan.ranges > 0) gather<T, kGrid>(x, first, plan, row.p, &to.held, a.list + (int64_t)blockIdx.y * kList);
}

template <class T>
__global__ __launch_bounds__(kChunkThreads) void sample_gather_kernel(Sample a) {
    SamplePlan& plan = a.plans[blockIdx.y];
    const int at = a.first_row + blockIdx.y, b = at / a.steps, step = at - b * a.steps, first = blockIdx.x * kChunk;
    const typename T::bits* p = static_cast<const typename T::bits*>(a.x) + b * a.batch_stride + step * a.step_stride;
    const Chunk<T> x(p, first, a.vocab);  // before the plan is known: one trip
    if (plan.ranges > 0) gather<T, kChunkThreads>(x, first, plan, p, &plan.held, a.list + (int64_t)blockIdx.y * kList);
}

// A chunk's sum over the bins before `bin` of the row, from its own, of which
// this lane of a wave has those kWave apart. -> in lane 0.
__device__ __forceinline__ uint64_t chunk_sum(const uint64_t (&v)[kGrid / kWave], int shift, int bin, const SamplePlan& plan, uint64_t unit,
                                              const double* factors) {
    uint64_t sum = 0;
#pragma unroll
    for (int u = 0; u < kGrid / kWave; ++u) {
        const int j = u * kWave + threadIdx.x % kWave + shift;
        if (j < bin) sum += scaled(v[u], plan.norm, factors[min(j, kGrid - 1)], plan.largest, unit, u == 0 && j == 0);
    }
    return group_combine<kWave>(sum, AddU64());
}

template <class T>
__global__ __launch_bounds__(kThreads) void sample_draw_kernel(Sample a) {
    using R = Row<T>;
    constexpr int kPer = kGrid / kWave, kFirst = kFast / kThreads;
    __shared__ Shared s;
    __shared__ unsigned long long runs[kMaxVocab / kChunk];
    __shared__ double factors[kGrid];
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int at = a.first_row + blockIdx.x, b = at / a.steps, step = at - b * a.steps;
    const SampleHead* heads = a.heads + (int64_t)blockIdx.x * a.chunks;
    const unsigned long long* bins = a.bins + (int64_t)blockIdx.x * a.chunks * kGrid;
    const unsigned long long* list = a.list + (int64_t)blockIdx.x * kList;
    // All that does not wait for anything else is asked for at once: the list's
    // first codes whether there are so many or not, the bins of a chunk a wave.
    uint64_t codes[kFirst], v[kPer];
#pragma unroll
    for (int u = 0; u < kFirst; ++u) codes[u] = list[u * kThreads + tid];
    const int own_chunk = min(wave, a.chunks - 1);
#pragma unroll
    for (int u = 0; u < kPer; ++u) v[u] = bins[(int64_t)own_chunk * kGrid + u * kWave + lane];
    const uint64_t head = heads[own_chunk].first;
    const uint64_t chunk_first = heads[min(tid, a.chunks - 1)].first;
    const SamplePlan plan = a.plans[blockIdx.x];
    SamplePlan& to = a.plans[blockIdx.x];
    const float r = a.r ? a.r[at] : 0.f;
    const int state = plan.state;
    const Settings set(a, b);
    for (int i = tid; i < kGrid; i += kThreads) factors[i] = power2<11>(-(double)i / kPerPower);
    R row(a, b, step);
    const uint64_t first = row.settle(plan.first, set.scale, a.shift);
    if (state == kRowNone || state == kRowOne) {
        if (tid == 0) {
            to.border = state == kRowOne ? first : ~0ull;
            to.share = 1.0;
            if (a.tokens) a.tokens[at] = state == kRowOne ? R::C::token(first) : -1;
        }
        return;
    }
    if (state == kRowWhole) {
        const uint64_t border = row_border(row, s, set, first);
        const uint64_t total = row_total(row, s, border);
        if (tid == 0) to.border = border, to.share = row.unit / (double)total;
        if (a.tokens) row_draw(row, s, border, draw_target(r, total), a.tokens + at);
        return;
    }
    // The gathered codes: in the LDS, with their weights, as far as there is room.
    const int held = (int)min(plan.held, (unsigned)kList), ranges = plan.ranges;
    const List<T> of{row, s, list, held};
#pragma unroll
    for (int u = 0; u < kFirst; ++u) {
        const int i = u * kThreads + tid;
        if (i < held) s.list[i] = codes[u], s.list_own[i] = of.units(codes[u]);
    }
    __syncthreads();
    // The chunks' sums in the bins above those gathered, which are kept whole.
    const Place place{set.scale * kPerPower};
    const double peak = place.floor_of(row.top_logit);
    const int bin = ranges > 0 ? plan.low : kGrid;
    const uint64_t unit = (uint64_t)row.unit;
    if (wave < a.chunks) {
        const uint64_t sum = chunk_sum(v, chunk_shift<T>(place, peak, head), bin, plan, unit, factors);
        if (lane == 0) runs[wave] = sum;
    }
    for (int c = wave + kWaves; c < a.chunks; c += kWaves) {
#pragma unroll
        for (int u = 0; u < kPer; ++u) v[u] = bins[(int64_t)c * kGrid + u * kWave + lane];
        const uint64_t sum = chunk_sum(v, chunk_shift<T>(place, peak, heads[c].first), bin, plan, unit, factors);
        if (lane == 0) runs[c] = sum;
    }
    // The border among the gathered codes.
    const uint64_t above = ranges > 0 ? first_code<T>(plan.upto[0]) : 0;
    const uint64_t border = cut_border(of, set, plan, above);
    // What is kept of the list joins its chunks.
    __syncthreads();
    if (ranges > 0)
        of.each([&](uint64_t c, auto weight) {
            // The gathering left a chunk's codes side by side: a wave has mostly those of
            // one, and adds them up first.
            const int chunk = R::C::token(c) / kChunk, one = __builtin_amdgcn_readfirstlane(chunk);
            uint64_t w = c >= border && c < above ? weight() : 0;
            if (__ballot(true) == ~0ull && __all(chunk == one)) {
                w = group_combine<kWave>(w, AddU64());
                if (lane == 0 && w) atomicAdd(&runs[one], (unsigned long long)w);
            } else if (w) {
                atomicAdd(&runs[chunk], (unsigned long long)w);
            }
        });
    __syncthreads();
    const uint64_t own = tid < a.chunks ? runs[tid] : 0;
    uint64_t total;
    uint64_t before = block_before(own, s, &total);
    if (tid == 0) to.border = border, to.share = row.unit / (double)total;
    if (!a.tokens) return;
    // The chunk: the last that begins below the target, of those in which a weight counts
    // by itself. (Its first code tells. The sums by bins hold weights of less than half a
    // unit as well, where they are many, and are cut off to whole units.) Where that is
    // none, the token is the first of the first of those; for r of 1, the last of the last.
    const uint64_t want = draw_target(r, total);
    const bool last = !(r < 1.f);
    const bool counts = tid < a.chunks && chunk_first >= border && row.units(row.weight(R::C::logit(chunk_first))) > 0;
    const uint64_t all = __ballot(counts), below = __ballot(counts && (last || before < want));
    if (tid < a.chunks) runs[tid] = want - before;
    if (tid < 2 * kWave && lane == 0) s.few[wave] = all, s.few_own[wave] = below;
    __syncthreads();
    static_assert(kMaxVocab / kChunk <= 2 * kWave, "chunks are told by two words");
    const bool first_one = (s.few_own[0] | s.few_own[1]) == 0;
    const int chunk = s.few_own[1] ? 127 - __clzll(s.few_own[1]) : s.few_own[0] ? 63 - __clzll(s.few_own[0])
                      : s.few[0]   ? __ffsll(s.few[0]) - 1
                                   : s.few[1] ? __ffsll(s.few[1]) + 63 : 0;
    // Its token. Sums by weights may fall short of those by bins.
    constexpr int kEach = kChunk / kThreads;
    const int i0 = chunk * kChunk + tid * kEach;
    const uint64_t rest = first_one ? 1 : last ? ~0ull : runs[chunk];
    float x[kEach];
    row.template neighbours<kEach>(i0, x);
    uint64_t w[kEach], mine = 0, whole;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        w[j] = row.kept_units(i0 + j, x[j], border);
        mine += w[j];
    }
    before = block_before(mine, s, &whole);
    const uint64_t goal = rest < whole ? rest : whole;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        if (before < goal && before + w[j] >= goal) a.tokens[at] = i0 + j;
        before += w[j];
    }
}

template <class T, class P>
__global__ __launch_bounds__(kChunkThreads) void sample_probs_kernel(Sample a) {
    using L = Chunk<T>;
    const SamplePlan& plan = a.plans[blockIdx.y];
    const int at = a.first_row + blockIdx.y, b = at / a.steps, step = at - b * a.steps, first = blockIdx.x * kChunk;
    const Settings set(a, b);
    Row<T> row(a, b, step);
    const L x(row.p, first, a.vocab);
    typename P::bits* probs = static_cast<typename P::bits*>(a.probs) + b * a.probs_batch + step * a.probs_step;
    const uint64_t border = plan.border;
    const double share = plan.share;
    row.settle(plan.first, set.scale, a.shift);
    write_probs<P>(row, x, first, border, share, probs);
}

template <class T>
hipError_t split(int probs_type, const Sample& a, unsigned int rows, hipStream_t stream) {
    const dim3 grid((unsigned)a.chunks, rows);
    sample_bins_kernel<T><<<grid, kChunkThreads, 0, stream>>>(a);
    hipError_t e = hipGetLastError();
    // Where few blocks would gather, each makes the row's plan itself, which saves a
    // launch. (Microseconds of the whole call, top-p, gathering apart / by the blocks
    // that find: 1 row of 32000 float32 25.1 / 24.1, 16 rows of 131071 (128 blocks) 27.9 /
    // 27.8, 64 rows of 65536 (256 blocks) 28.0 / 30.2, 192 rows of 131071 61 / 75. With
    // one block a row it saves 1 to 3 whatever the rows: 1900 rows of 16000 153 / 149.)
    const unsigned int blocks = (a.vocab + Loads<T, kGrid>::kAll - 1) / Loads<T, kGrid>::kAll;
    const bool few = a.filtered && (blocks == 1 || blocks * rows <= 128);
    if (e == hipSuccess) sample_find_kernel<T><<<dim3(few ? blocks : 1, rows), kGrid, 0, stream>>>(a, few), e = hipGetLastError();
    if (e == hipSuccess && a.filtered && !few) sample_gather_kernel<T><<<grid, kChunkThreads, 0, stream>>>(a), e = hipGetLastError();
    if (e == hipSuccess) sample_draw_kernel<T><<<rows, kThreads, 0, stream>>>(a), e = hipGetLastError();
    if (e != hipSuccess || !a.probs) return e;
    if (probs_type == RED_F16) sample_probs_kernel<T, F16><<<grid, kChunkThreads, 0, stream>>>(a);
    else if (probs_type == RED_BF16) sample_probs_kernel<T, BF16><<<grid, kChunkThreads, 0, stream>>>(a);
    else sample_probs_kernel<T, F32><<<grid, kChunkThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_sample_split(int type, int probs_type, const Sample& a, unsigned int rows, hipStream_t stream) {
    return type == RED_F32   ? split<F32>(probs_type, a, rows, stream)
           : type == RED_F16 ? split<F16>(probs_type, a, rows, stream)
                             : split<BF16>(probs_type, a, rows, stream);
}

}  // namespace libred
