// Sampling: a block a row, in one launch, and the choice of the kernel by types.
// A row goes through the block once for its largest logit, once or twice more for
// each border and twice for the token. It is for short rows, where latency is all
// there is: 4000 logits, top-p, 16.5 us for 1 row, 18.4 for 192 (see kSampleRow).
#include "sample_common.hpp"

namespace libred {

namespace {

template <class T, class P>
__global__ __launch_bounds__(kThreads) void sample_row_kernel(Sample a) {
    using R = Row<T>;
    __shared__ Shared s;
    const int at = a.first_row + blockIdx.x, b = at / a.steps, step = at - b * a.steps, tid = threadIdx.x;
    const Settings set(a, b);
    R row(a, b, step);
    typename P::bits* probs = a.probs ? static_cast<typename P::bits*>(a.probs) + b * a.probs_batch + step * a.probs_step : nullptr;

    uint64_t first = 0;
    row.each([&](int i, float x) {
        const uint64_t c = R::C::of(x, i);
        first = c > first ? c : first;
    });
    first = block_combine(first, s, MaxU64());
    if (R::C::logit(first) == kNone) {
        if (a.tokens && tid == 0) a.tokens[at] = -1;
        if (probs)
            for (int i = tid; i < a.vocab; i += kThreads) probs[i] = P::narrow(0.f);
        return;
    }
    first = row.settle(first, set.scale, a.shift);
    const uint64_t border = row_border(row, s, set, first);
    const uint64_t total = row_total(row, s, border);
    if (a.tokens) row_draw(row, s, border, draw_target(a.r[at], total), a.tokens + at);
    if (probs) {
        const double share = row.unit / (double)total;
        row.tiles([&](int i, const float(&x)[R::kVec]) {
            typename P::bits v[R::kVec];
            // A second rounding, from float32, moves a 16-bit one by 2^-16 of its step at most.
#pragma unroll
            for (int j = 0; j < R::kVec; ++j)
                v[j] = P::narrow(x[j] == kNone || R::C::of(x[j], i + j) < border ? 0.f : (float)(row.weight(x[j]) * share));
            for (int j = 0; j < R::kVec; ++j)
                if (i + j < a.vocab) probs[i + j] = v[j];
        });
    }
}

template <class T, class P>
hipError_t launch_row(const Sample& a, unsigned int rows, hipStream_t stream) {
    sample_row_kernel<T, P><<<rows, kThreads, 0, stream>>>(a);
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
