// The verification's kernels on the host (SOURCE: verify_drafts.hip up to its
// launches): one sequence without drafts, `vocab` tokens of weight 1, so that r
// draws token floor(r * vocab). Arguments: one launch (1) or two (0), vocab, r,
// the wave that is late. Prints the token.
#include <stdio.h>
#include <stdlib.h>

#include SOURCE

int main(int, char** argv) {
    using namespace libred;
    const bool one = atoi(argv[1]) != 0;
    const int64_t vocab = atoll(argv[2]);
    const float r = (float)atof(argv[3]);
    emulated::late_wave = atoi(argv[4]);
    std::vector<float> p(vocab, 1.f);
    Verify a = {};
    int32_t accepted = -1;
    int64_t token = -2;
    double sums[kVerifyMaxSegs];
    a.p = p.data(), a.r = &r, a.accepted = &accepted, a.tokens = &token, a.sums = sums;
    a.vocab = vocab, a.seg = 1024, a.segs = (int)((vocab + 1023) / 1024), a.batch = 1;
    if (one) {
        emulated::run_block(kThreadsOne, 1, 0, 0, [&] { verify_one_kernel<F32>(a); });
    } else {
        for (int b = 0; b < (a.segs + 3) / 4; ++b)
            emulated::run_block(kThreads, (a.segs + 3) / 4, b, 0, [&] { verify_sum_kernel<F32>(a); });
        emulated::run_block(kThreads, 1, 0, 0, [&] { verify_pick_kernel<F32>(a); });
    }
    printf("%d %lld\n", accepted, (long long)token);
    return 0;
}
