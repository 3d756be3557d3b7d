// Sampling: rows cut into chunks, in four launches (five with probabilities).
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
//     second read of the row, with two comparisons a logit.
//  4. draw: a block a row finds the border among them, the chunk in which the
//     running sum of the kept weights passes its target, by the chunks' bins,
//     and the token in that chunk.
//  5. probabilities.
//
// Where more logits than kList are near a border (thousands of equal ones), or
// the border is further than 64 powers of two below the largest weight, the
// block that draws goes through the whole row instead.
#include "sample_common.hpp"

namespace libred {

namespace {

constexpr int kChunk = kSampleChunk, kChunkThreads = 256, kOwn = kChunk / kChunkThreads;
constexpr int kGrid = kSampleGrid;       // bins: 64 powers of two
constexpr double kPerPower = 8.0;        // bins a power of two
constexpr int kList = kSampleList;
constexpr int kCountAt = 50;             // a bin's number is above this bit, its sum below, in units of 2^-36
constexpr uint64_t kSumMask = (1ull << kCountAt) - 1;
static_assert(kChunk <= 1 << (64 - kCountAt - 1) && kChunk <= 1 << (kCountAt - 37), "a chunk's sums have room");

// What a logit is on the grid of a row.
struct Place {
    double scale;  // 8 log2(e) / T
    __device__ __forceinline__ double y(float x) const { return (double)x * scale; }
    __device__ __forceinline__ double floor_of(float x) const { return __builtin_floor(y(x)); }
};

// 2^36 2^((f - 1) / 8) for the place f in its bin, as the low bits of 2^52 more.
// Coefficients: (log(2) / 8)^n / n! times 2^36 2^(-1/16), around f = 1/2; what
// is left out is below 2^-44 of the whole.
__device__ __forceinline__ uint64_t relative_units(double f) {
    constexpr double l = 0.69314718055994530942 / 8.0, c = 0x1p36 * 0.95760328069857364694;  // 2^(-1/16)
    const double t = f - 0.5;
    double r = c * l * l * l * l * l * l / 720.0;
    r = __builtin_fma(r, t, c * l * l * l * l * l / 120.0);
    r = __builtin_fma(r, t, c * l * l * l * l / 24.0);
    r = __builtin_fma(r, t, c * l * l * l / 6.0);
    r = __builtin_fma(r, t, c * l * l / 2.0);
    r = __builtin_fma(r, t, c * l);
    r = __builtin_fma(r, t, c + 0x1p52);
    return __builtin_bit_cast(uint64_t, r) & 0xFFFFFFFFFFFFFull;
}

template <class T>
struct Loads {
    using B = typename T::bits;
    static constexpr int kVec = 16 / sizeof(B), kCount = kOwn / kVec;
    typedef B Vector __attribute__((ext_vector_type(16 / sizeof(B)), aligned(sizeof(B))));
    Vector v[kCount];

    // The chunk's logits from number `first` on, those of thread tid: kVec
    // neighbours every kChunkThreads * kVec. Behind the last: -inf.
    __device__ __forceinline__ Loads(const B* p, int first, int vocab) {
        const int tid = threadIdx.x;
        if (first + kChunk <= vocab) {
#pragma unroll
            for (int u = 0; u < kCount; ++u) v[u] = *reinterpret_cast<const Vector*>(p + first + (u * kChunkThreads + tid) * kVec);
        } else {
#pragma unroll
            for (int u = 0; u < kCount; ++u)
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    const int i = first + (u * kChunkThreads + tid) * kVec + j;
                    v[u][j] = i < vocab ? p[i] : T::narrow(kNone);
                }
        }
    }
    __device__ __forceinline__ float at(int n) const { return T::widen(v[n / kVec][n % kVec]); }
    __device__ __forceinline__ static int number(int n) { return (n / kVec * kChunkThreads + threadIdx.x) * kVec + n % kVec; }
};

template <class T>
__global__ __launch_bounds__(kChunkThreads) void sample_bins_kernel(Sample a) {
    constexpr int W = kChunkThreads / kWave;
    __shared__ __align__(16) unsigned long long bins[kGrid];
    __shared__ float tops[W];
    __shared__ int numbers[W], counts[W];
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int at = a.first_row + blockIdx.y, b = at / a.steps, step = at - b * a.steps, first = blockIdx.x * kChunk;
    const typename T::bits* p = static_cast<const typename T::bits*>(a.x) + b * a.batch_stride + step * a.step_stride;
    const Loads<T> x(p, first, a.vocab);
    const Settings set(a, b);
    for (int i = tid; i < kGrid; i += kChunkThreads) bins[i] = 0;
    // The largest logit; a NaN is none.
    float top = kNone;
#pragma unroll
    for (int n = 0; n < kOwn; ++n) top = fmaxf(top, x.at(n));
    top = group_combine<kWave>(top, [](float m, float n) { return fmaxf(m, n); });
    if (lane == 0) tops[wave] = top;
    __syncthreads();
    top = tops[0];
#pragma unroll
    for (int w = 1; w < W; ++w) top = fmaxf(top, tops[w]);
    // Its first number, how many logits there are above -inf, and the bins.
    const Place place{set.scale * kPerPower};
    const double peak = place.floor_of(top);
    const bool binned = set.k != 1 && top < __builtin_inff();
    int number = kChunk, count = 0;
#pragma unroll
    for (int n = 0; n < kOwn; ++n) {
        const float v = x.at(n);
        if (v == top) number = min(number, Loads<T>::number(n));
        if (binned && v > kNone) {
            ++count;
            const double y = place.y(v), g = __builtin_floor(y), d = peak - g;
            if (d < (double)kGrid) atomicAdd(&bins[(int)d], (unsigned long long)(relative_units(y - g) + (1ull << kCountAt)));
        }
    }
    number = group_combine<kWave>(number, [](int m, int n) { return min(m, n); });
    count = group_combine<kWave>(count, [](int m, int n) { return m + n; });
    if (lane == 0) numbers[wave] = number, counts[wave] = count;
    __syncthreads();
    const int64_t chunk = (int64_t)blockIdx.y * a.chunks + blockIdx.x;
    if (tid == 0) {
        for (int w = 1; w < W; ++w) number = min(number, numbers[w]), count += counts[w];
        a.heads[chunk] = SampleHead{code_of(top + 0.f, first + (number < kChunk ? number : 0)), count};
    }
    if (binned)
        for (int i = tid; i < kGrid / 2; i += kChunkThreads)
            reinterpret_cast<u32x4*>(a.bins + chunk * kGrid)[i] = reinterpret_cast<const u32x4*>(bins)[i];
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
__device__ __forceinline__ int chunk_shift(const Place& place, double peak, uint64_t code) {
    const float x = logit_of(code);
    const double d = x > kNone ? peak - place.floor_of(x) : (double)kGrid;
    return d < (double)kGrid ? (int)d : kGrid;
}

template <class T>
__global__ __launch_bounds__(kGrid) void sample_find_kernel(Sample a) {
    __shared__ Found s;
    __shared__ int shifts[kMaxVocab / kChunk];
    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int at = a.first_row + blockIdx.x, b = at / a.steps, step = at - b * a.steps;
    const Settings set(a, b);
    const SampleHead* heads = a.heads + (int64_t)blockIdx.x * a.chunks;
    SamplePlan& plan = a.plans[blockIdx.x];
    const SampleHead head = row_head(heads, a.chunks, s.part, s.parts);
    const float top = logit_of(head.first);
    int state = top == kNone ? kRowNone : set.k == 1 ? kRowOne : top == __builtin_inff() ? kRowWhole : kRowCut;
    if (tid < 4) s.first[tid] = kGrid;
    if (tid == 0) plan.first = head.first, plan.held = 0, plan.state = state, plan.ranges = 0;
    if (state != kRowCut) return;

    Row<T> row(a, b, step);
    row.settle(head.first, set.scale, a.shift);
    const Place place{set.scale * kPerPower};
    const double peak = place.floor_of(top);
    for (int c = tid; c < a.chunks; c += kGrid) shifts[c] = chunk_shift(place, peak, heads[c].first);
    __syncthreads();
    // Bin tid of the row.
    uint64_t sum = 0;
    unsigned int count = 0;
    const unsigned long long* bins = a.bins + (int64_t)blockIdx.x * a.chunks * kGrid;
    for (int c = 0; c < a.chunks; ++c) {
        const int j = tid - shifts[c];
        if (j >= 0) {
            const uint64_t v = bins[(int64_t)c * kGrid + j];
            sum += v & kSumMask, count += (unsigned int)(v >> kCountAt);
        }
    }
    // In units of the largest weight: bin 0's upper edge is 2^((peak + 1 - y) / 8) of it.
    const double norm = row.unit * 0x1p-36 * exp2((peak + 1.0 - place.y(top)) / kPerPower);
    uint64_t mass = (uint64_t)((double)sum * (norm * exp2(-(double)tid / kPerPower)));
    const unsigned int own_count = count;
    mass = wave_scan(mass);
    count += dpp_move<0x111, 0xF>(0u, count);
    count += dpp_move<0x112, 0xF>(0u, count);
    count += dpp_move<0x114, 0xF>(0u, count);
    count += dpp_move<0x118, 0xF>(0u, count);
    count += dpp_move<0x142, 0xA>(0u, count);
    count += dpp_move<0x143, 0xC>(0u, count);
    __syncthreads();
    if (lane == kWave - 1) s.part[wave] = mass, s.parts[wave] = count;
    __syncthreads();
    for (int w = 0; w < wave; ++w) mass += s.part[w], count += s.parts[w];
    s.mass[tid] = mass, s.count[tid] = count;
    // The least logit that min-p keeps.
    if (wave == 0 && set.m > 0.0) {
        const uint32_t cut = first_key((uint32_t)(head.first >> 20), [&](float x) { return row.weight(x) >= set.m; });
        if (lane == 0) s.cut = cut;
    }
    __syncthreads();
    const uint64_t all = s.mass[kGrid - 1];
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
        const double d = peak - place.floor_of(logit_of(cut));
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
        if (n > kList) state = kRowWhole, ranges = 0;
    }
    // Their logits: from the first of the last bin to below the first of the bin
    // before the first.
    if (wave < 2 * ranges) {
        const int bin = wave == 0 ? high : wave == 1 ? low - 1 : wave == 2 ? kbin : kbin - 1;
        const uint32_t key = (uint32_t)(head.first >> 20);
        const uint32_t edge = bin < 0 ? key + 1 : first_key(key, [&](float x) { return peak - place.floor_of(x) <= (double)bin; });
        if (lane == 0) s.edge[wave] = edge;
    }
    __syncthreads();
    if (tid == 0) {
        plan.state = state, plan.ranges = ranges;
        plan.use_k = use_k && ranges > 0, plan.use_p = use_p && ranges > 0;
        plan.cut = cut;
        for (int r = 0; r < ranges; ++r) plan.from[r] = logit_of_key(s.edge[2 * r]), plan.upto[r] = logit_of_key(s.edge[2 * r + 1]);
        plan.low = low, plan.high = high;
        const int before = second ? kbin : low;  // bins before the range that has top-k's border
        plan.k_rest = use_k && ranges > 0 ? (uint64_t)set.k - (before > 0 ? s.count[before - 1] : 0) : 0;
        plan.k_before = before_k;
        plan.p_before = low > 0 && low < kGrid ? s.mass[low - 1] : 0;
        plan.all = all;
        plan.norm = norm;
    }
}

template <class T>
__global__ __launch_bounds__(kChunkThreads) void sample_gather_kernel(Sample a) {
    constexpr int W = kChunkThreads / kWave;
    __shared__ unsigned int counts[W], start;
    SamplePlan& plan = a.plans[blockIdx.y];
    if (plan.ranges == 0) return;
    const float from0 = plan.from[0], upto0 = plan.upto[0];
    const bool two = plan.ranges == 2;
    const float from1 = two ? plan.from[1] : 1.f, upto1 = two ? plan.upto[1] : 0.f;
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int at = a.first_row + blockIdx.y, b = at / a.steps, step = at - b * a.steps, first = blockIdx.x * kChunk;
    const typename T::bits* p = static_cast<const typename T::bits*>(a.x) + b * a.batch_stride + step * a.step_stride;
    const Loads<T> x(p, first, a.vocab);
    uint32_t in = 0;
    static_assert(kOwn <= 32, "a bit a logit");
#pragma unroll
    for (int n = 0; n < kOwn; ++n) {
        const float v = x.at(n);
        if ((v >= from0 && v < upto0) || (v >= from1 && v < upto1)) in |= 1u << n;
    }
    // Places in the list: this thread's behind those of the threads before.
    unsigned int own = (unsigned)__popc(in), upto = own;
    upto += dpp_move<0x111, 0xF>(0u, upto);
    upto += dpp_move<0x112, 0xF>(0u, upto);
    upto += dpp_move<0x114, 0xF>(0u, upto);
    upto += dpp_move<0x118, 0xF>(0u, upto);
    upto += dpp_move<0x142, 0xA>(0u, upto);
    upto += dpp_move<0x143, 0xC>(0u, upto);
    if (lane == kWave - 1) counts[wave] = upto;
    __syncthreads();
    unsigned int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        if (w == wave) before = all;
        all += counts[w];
    }
    if (all == 0) return;
    if (tid == 0) start = atomicAdd(&plan.held, all);
    __syncthreads();
    unsigned int to = start + before + upto - own;
    unsigned long long* list = a.list + (int64_t)blockIdx.y * kList;
#pragma unroll
    for (int n = 0; n < kOwn; ++n)
        if (in >> n & 1) {
            if (to < kList) list[to] = code_of(x.at(n) + 0.f, first + Loads<T>::number(n));
            ++to;
        }
}

// The code at which the running sum of value(code), in the order of the codes
// of the list, among those from `from` to below `upto`, reaches `want`; the last of
// them where it does not, ~0 where there are none.
template <class V>
__device__ __forceinline__ uint64_t list_border(Shared& s, const unsigned long long* list, int n, uint64_t from, uint64_t upto,
                                                uint64_t want, V value) {
    __syncthreads();
    if (threadIdx.x == 0) s.found = 0, s.held = 0, s.rest = ~0ull;
    __syncthreads();
    uint64_t least = ~0ull, most = 0, sum = 0;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const uint64_t c = list[i];
        if (c >= from && c < upto) {
            least = c < least ? c : least, most = c > most ? c : most;
            sum += value(c);
        }
    }
    sum = block_combine(sum, s, AddU64());
    most = block_combine(most, s, MaxU64());
    least = ~block_combine(~least, s, MaxU64());
    if (most == 0) return ~0ull;
    if (want >= sum) return least;  // also where roundings leave the sum short
    if (want == 0) want = 1;
    int down = bytes_of(least ^ most) * 8;
    uint64_t prefix = most >> down;
    while (down > 0) {
        const int to = down - 8;
        clear_bins(s);
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const uint64_t c = list[i];
            if (c >= from && c < upto && c >> down == prefix) atomicAdd(&s.mass[c >> to & 255], (unsigned long long)value(c));
        }
        find_bin(s, want, true);
        prefix = prefix << 8 | s.bin;
        want = s.rest;
        down = to;
    }
    return prefix;
}

template <class T>
__global__ __launch_bounds__(kThreads) void sample_draw_kernel(Sample a) {
    using R = Row<T>;
    __shared__ Shared s;
    __shared__ unsigned long long runs[kMaxVocab / R::kRun];
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int at = a.first_row + blockIdx.x, b = at / a.steps, step = at - b * a.steps;
    SamplePlan& plan = a.plans[blockIdx.x];
    const int state = plan.state;
    const Settings set(a, b);
    R row(a, b, step);
    const uint64_t first = row.settle(plan.first, set.scale, a.shift);
    if (state == kRowNone || state == kRowOne) {
        if (tid == 0) {
            plan.border = state == kRowOne ? first : ~0ull;
            plan.share = 1.0;
            if (a.tokens) a.tokens[at] = state == kRowOne ? token_of(first) : -1;
        }
        return;
    }
    if (state == kRowWhole) {
        const uint64_t border = row_border(row, s, set, first);
        const uint64_t total = row_total(row, s, runs, border);
        if (tid == 0) plan.border = border, plan.share = row.unit / (double)total;
        if (a.tokens) row_draw(row, s, runs, border, draw_target(a.r[at], total), a.tokens + at);
        return;
    }
    // The border among the gathered codes.
    const unsigned long long* list = a.list + (int64_t)blockIdx.x * kList;
    const int held = (int)min(plan.held, (unsigned)kList), ranges = plan.ranges;
    auto key = [](float x) { return code_of(x, kMaxVocab - 1); };  // the last code of a logit
    uint64_t border = 0;
    auto units = [&](uint64_t c) { return row.units(row.weight(logit_of(c))); };
    if (plan.use_k) {
        const int r = ranges - 1;
        border = list_border(s, list, held, key(plan.from[r]), key(plan.upto[r]), plan.k_rest, [](uint64_t) -> uint64_t { return 1; });
    }
    if (plan.use_p) {
        uint64_t all = plan.all;
        if (plan.use_k) {
            // Those of the bin of top-k's border that are kept.
            const uint64_t from = border, upto = key(plan.upto[ranges - 1]);
            uint64_t sum = 0;
            for (int i = tid; i < held; i += kThreads)
                if (list[i] >= from && list[i] < upto) sum += units(list[i]);
            sum = block_combine(sum, s, AddU64());
            // of the last range's first bin on: with one range what lies between is counted with it
            all = (ranges == 2 ? plan.k_before : plan.p_before) + sum;
        }
        const uint64_t want = top_p_target(set.p, all);
        uint64_t from = key(plan.from[0]);
        from = from > border ? from : border;
        const uint64_t upto = key(plan.upto[0]);
        const uint64_t found = want > plan.p_before ? list_border(s, list, held, from, upto, want - plan.p_before, units) : upto;
        border = found > border ? found : border;
        if (found == ~0ull) border = upto;
    }
    border = plan.cut > border ? plan.cut : border;
    // The sums of the chunks: bins above the list's by what the chunks have of
    // them, and what is kept of the list.
    const Place place{set.scale * kPerPower};
    const double peak = place.floor_of(row.top_logit);
    const int bin = ranges > 0 ? plan.low : kGrid;                    // bins before this one are kept whole
    const uint64_t above = ranges > 0 ? key(plan.upto[0]) : 0;  // their codes, from here on
    const SampleHead* heads = a.heads + (int64_t)blockIdx.x * a.chunks;
    const unsigned long long* bins = a.bins + (int64_t)blockIdx.x * a.chunks * kGrid;
    __syncthreads();
    for (int c = wave; c < a.chunks; c += kWaves) {
        const int shift = chunk_shift(place, peak, heads[c].first);
        uint64_t sum = 0;
        for (int j = lane; j < kGrid; j += kWave)
            if (j + shift < bin) {
                const uint64_t v = bins[(int64_t)c * kGrid + j] & kSumMask;
                sum += (uint64_t)((double)v * (plan.norm * exp2(-(double)(j + shift) / kPerPower)));
            }
        sum = group_combine<kWave>(sum, AddU64());
        if (lane == 0) runs[c] = sum;
    }
    __syncthreads();
    if (ranges > 0)
        for (int i = tid; i < held; i += kThreads) {
            const uint64_t c = list[i];
            if (c >= border && c < above) atomicAdd(&runs[token_of(c) / kChunk], (unsigned long long)units(c));
        }
    __syncthreads();
    uint64_t own = tid < a.chunks ? runs[tid] : 0;
    const uint64_t total = block_combine(own, s, AddU64());
    if (tid == 0) plan.border = border, plan.share = row.unit / (double)total;
    if (!a.tokens) return;
    const uint64_t want = draw_target(a.r[at], total);
    uint64_t before = block_before(own, s);
    if (own > 0 && before < want && before + own >= want) s.bin = tid, s.rest = want - before;
    __syncthreads();
    // The chunk, in which sums by weights may fall short of those by bins.
    constexpr int kEach = kChunk / kThreads;
    const int i0 = (int)s.bin * kChunk + tid * kEach;
    const uint64_t rest = s.rest;
    uint64_t w[kEach], mine = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        w[j] = i0 + j < a.vocab ? row.kept_units(i0 + j, row.seen(row.p[i0 + j]), border) : 0;
        mine += w[j];
    }
    before = block_before(mine, s);
    const uint64_t whole = block_combine(mine, s, AddU64());
    const uint64_t goal = rest < whole ? rest : whole;
    if (whole == 0 && tid == 0) a.tokens[at] = token_of(first);  // weights that are less than a unit each
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        if (before < goal && before + w[j] >= goal) a.tokens[at] = i0 + j;
        before += w[j];
    }
}

template <class T, class P>
__global__ __launch_bounds__(kChunkThreads) void sample_probs_kernel(Sample a) {
    using L = Loads<T>;
    const SamplePlan& plan = a.plans[blockIdx.y];
    const int at = a.first_row + blockIdx.y, b = at / a.steps, step = at - b * a.steps, first = blockIdx.x * kChunk;
    const Settings set(a, b);
    Row<T> row(a, b, step);
    const L x(row.p, first, a.vocab);
    typename P::bits* probs = static_cast<typename P::bits*>(a.probs) + b * a.probs_batch + step * a.probs_step;
    const uint64_t border = plan.border;
    const double share = plan.share;
    row.settle(plan.first, set.scale, a.shift);
    typedef typename P::bits Out __attribute__((ext_vector_type(L::kVec), aligned(sizeof(typename P::bits))));
#pragma unroll
    for (int u = 0; u < L::kCount; ++u) {
        const int i0 = first + L::number(u * L::kVec);
        Out v;
#pragma unroll
        for (int j = 0; j < L::kVec; ++j) {
            const float f = row.seen(x.v[u][j]);
            const bool kept = f != kNone && code_of(f, i0 + j) >= border;
            // A second rounding, from float32, moves a 16-bit one by 2^-16 of its step at most.
            v[j] = P::narrow(kept ? (float)(row.weight(f) * share) : 0.f);
        }
        if (i0 + L::kVec <= a.vocab) {
            *reinterpret_cast<Out*>(probs + i0) = v;
        } else {
#pragma unroll
            for (int j = 0; j < L::kVec; ++j)
                if (i0 + j < a.vocab) probs[i0 + j] = v[j];
        }
    }
}

template <class T>
hipError_t split(int probs_type, const Sample& a, unsigned int rows, hipStream_t stream) {
    const dim3 grid((unsigned)a.chunks, rows);
    sample_bins_kernel<T><<<grid, kChunkThreads, 0, stream>>>(a);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess) sample_find_kernel<T><<<rows, kGrid, 0, stream>>>(a), e = hipGetLastError();
    if (e == hipSuccess && a.filtered) sample_gather_kernel<T><<<grid, kChunkThreads, 0, stream>>>(a), e = hipGetLastError();
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
