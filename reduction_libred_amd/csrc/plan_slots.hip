// Pages and slots for the next tokens of a batch of sequences.
//
// Running sums over the sequences say everything: of the pages given back,
// where each lies on the stack; of the pages wanted, who gets any and which;
// of the tokens, their numbers. Then three things are independent for each
// element: a page of the stack's changed part goes to `fresh` or onto the stack
// (its place on the stack tells where it comes from: the stack itself or a row
// given back), a new page of a row comes from `fresh`, and a token's slot from
// its row's page, old or fresh. The order of the sums is that of the sequences.
//
// Latency bounds it: a page of bytes, four trips to memory one after another
// (lengths, stack, searches, table). So a small step is one launch of one block:
// 6.2 us for 32 sequences of 9 tokens. Where tokens are many they go through a
// launch of their own, and so do pages (the borders are beside the launch): 256
// prompts of 130000 tokens in all, 2100 pages taken and 16000 given back, 9.7 us for
// the sums and pages and 6 for the tokens. Pages given back in a step of few tokens go
// through the one block, however many: 2.5 ns each.
#include "decode_common.hpp"
#include "serve.hpp"

namespace libred {

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / kWave;

// Running sum over the block's threads, this one's value included; *total is
// the whole. Fixed order (whole numbers, so any order would do).
template <class V>
__device__ __forceinline__ V block_scan(V v, V* lds, V* total) {
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    v += dpp_move<0x111, 0xF>((V)0, v);
    v += dpp_move<0x112, 0xF>((V)0, v);
    v += dpp_move<0x114, 0xF>((V)0, v);
    v += dpp_move<0x118, 0xF>((V)0, v);
    v += dpp_move<0x142, 0xA>((V)0, v);
    v += dpp_move<0x143, 0xC>((V)0, v);
    __syncthreads();
    if (lane == kWave - 1) lds[wave] = v;
    __syncthreads();
    V before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w == wave) before = all;
        all += lds[w];
    }
    *total = all;
    return before + v;
}

__device__ __forceinline__ int clamped(int v, int top) { return min(max(v, 0), top); }

// The last of n + 1 numbers, none smaller than the one before it, that is not
// above v; the first is not.
__device__ __forceinline__ int last_upto(const int* x, int n, int v) {
    int low = 0, high = n;
    while (low < high) {
        const int mid = (low + high + 1) >> 1;
        if (x[mid] <= v) low = mid;
        else high = mid - 1;
    }
    return low;
}

// The sums (a block). What a sequence brings is asked for at once; with more than
// kThreads of them it is asked for again for the second sums.
__device__ __forceinline__ void plan_sums(const PlanSlots& a) {
    __shared__ int64_t lds[kWaves];
    __shared__ int lds32[kWaves], taken;
    struct Sequence {
        int count, len, held, done;
    };
    const int tid = threadIdx.x;
    auto sequence = [&](int b) {
        Sequence q = {0, 0, 0, 0};
        if (b < a.batch) q = Sequence{a.counts[b], a.lens[b], a.held[b], a.done ? a.done[b] : 0};
        return Sequence{max(q.count, 0), max(q.len, 0), clamped(q.held, a.cols), q.done};
    };
    Sequence q = sequence(tid);
    const int height = clamped(a.height[0], a.pages);
    int given = 0;
    if (a.done) {
        for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
            if (b0 > 0) q = sequence(b0 + tid);
            const int b = b0 + tid, own = q.done ? q.held : 0;
            int all;
            const int upto = given + block_scan(own, lds32, &all);
            if (b < a.batch) a.back[b] = upto - own;
            given += all;
        }
    }
    const int now = (int)min((int64_t)height + given, (int64_t)a.pages);
    if (tid == 0) taken = 0;
    int64_t tokens = 0;
    int wants = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
        if (a.batch > kThreads) q = sequence(b0 + tid);
        const int b = b0 + tid, n = q.count, have = q.done ? 0 : q.held;
        int64_t all;
        const int64_t upto = tokens + block_scan((int64_t)n, lds, &all);
        const int64_t need = ((int64_t)q.len + n + a.places - 1) / a.places;
        const bool fits = n > 0 && upto <= a.tokens && need <= a.cols;
        const int want = fits ? max((int)need - have, 0) : 0;
        int all32;
        const int cum = wants + block_scan(want, lds32, &all32);
        const bool good = fits && (want == 0 || cum <= now);
        if (b < a.batch) {
            a.starts[b] = (int)min(upto - n, (int64_t)a.tokens);
            a.granted[b] = good ? n : 0;
            a.have[b] = have;
            a.before[b] = cum - want;
            a.held[b] = have + (good ? want : 0);
            if (good && want > 0) atomicMax(&taken, cum);
        }
        tokens += all;
        wants += all32;
    }
    __syncthreads();
    if (tid == 0) {
        a.starts[a.batch] = (int)min(tokens, (int64_t)a.tokens);
        a.back[a.batch] = given;
        a.before[a.batch] = wants;
        a.sums[0] = height, a.sums[1] = now, a.sums[2] = now - taken;
        a.height[0] = now - taken;
    }
}

// The stack and the pages taken from it, `stride` threads at a time.
__device__ __forceinline__ void plan_pages(const PlanSlots& a, int64_t at, int64_t stride) {
    const int height = a.sums[0], now = a.sums[1], base = a.sums[2];
    for (int64_t i = min(base, height) + at; i < now; i += stride) {
        int page;
        if (i < height) {
            page = a.stack[i];
        } else {
            const int o = (int)i - height, b = last_upto(a.back, a.batch, o);
            page = a.table[b * a.table_stride + o - a.back[b]];
        }
        if (i >= base) a.fresh[i - base] = page;
        a.stack[i] = i >= base ? -1 : page;
    }
}

// The rows' new pages, and the tokens.
__device__ __forceinline__ void plan_tokens(const PlanSlots& a, int64_t at, int64_t stride) {
    const int taken = a.sums[1] - a.sums[2], all = a.starts[a.batch];
    for (int64_t o = at; o < taken; o += stride) {
        const int b = last_upto(a.before, a.batch, (int)o);
        a.table[b * a.table_stride + a.have[b] + o - a.before[b]] = a.fresh[o];
    }
    for (int64_t t = at; t < a.tokens; t += stride) {
        int64_t slot = -1, pos = 0;
        if (t < all) {
            const int b = last_upto(a.starts, a.batch, (int)t);
            const uint32_t p = (uint32_t)max(a.lens[b], 0) + (uint32_t)(t - a.starts[b]);
            pos = p;
            if (a.granted[b]) {
                const uint32_t j = p / (uint32_t)a.places;
                const int have = a.have[b];
                const int page = (int)j < have ? a.table[b * a.table_stride + j] : a.fresh[a.before[b] + (int)j - have];
                slot = (int64_t)page * a.places + (p - j * (uint32_t)a.places);
            }
        }
        a.slots[t] = slot;
        a.pos[t] = pos;
    }
}

__global__ __launch_bounds__(kThreads) void plan_one_kernel(PlanSlots a) {
    plan_sums(a);
    __syncthreads();
    plan_pages(a, threadIdx.x, kThreads);
    __syncthreads();
    plan_tokens(a, threadIdx.x, kThreads);
}

__global__ __launch_bounds__(kThreads) void plan_sums_kernel(PlanSlots a, int few) {
    plan_sums(a);
    if (!few) return;
    __syncthreads();
    plan_pages(a, threadIdx.x, kThreads);
}

constexpr int kWide = 256;
__global__ __launch_bounds__(kWide) void plan_pages_kernel(PlanSlots a) {
    plan_pages(a, (int64_t)blockIdx.x * kWide + threadIdx.x, (int64_t)gridDim.x * kWide);
}
__global__ __launch_bounds__(kWide) void plan_tokens_kernel(PlanSlots a) {
    plan_tokens(a, (int64_t)blockIdx.x * kWide + threadIdx.x, (int64_t)gridDim.x * kWide);
}

}  // namespace

hipError_t launch_plan_slots(const PlanSlots& a, int blocks, bool few, hipStream_t stream) {
    if (blocks == 0) {
        plan_one_kernel<<<1, kThreads, 0, stream>>>(a);
        return hipGetLastError();
    }
    plan_sums_kernel<<<1, kThreads, 0, stream>>>(a, few);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && !few) plan_pages_kernel<<<blocks, kWide, 0, stream>>>(a), e = hipGetLastError();
    if (e == hipSuccess) plan_tokens_kernel<<<blocks, kWide, 0, stream>>>(a), e = hipGetLastError();
    return e;
}

}  // namespace libred
