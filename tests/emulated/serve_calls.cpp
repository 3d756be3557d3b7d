// The entry points of libred_serve.h (serve.cpp, compiled for the host) over
// launchers that note what they are asked for and do nothing.
#include <vector>

#include "serve.cpp"

namespace {

std::vector<size_t> scratch;  // bytes asked for

// What a launch was asked for: blocks of its largest grid and their threads,
// items (sequences, rows), and where its lengths and its output begin.
struct Launch {
    int64_t blocks, threads, items, in, out;
};
std::vector<Launch> launches;

int64_t at(const void* p) { return (int64_t)(uintptr_t)p; }

}  // namespace

namespace libred {

red_status host_fail(hipError_t, red_status code) { return code; }
red_status host_compute_units(int* dev, int* cu_count) {
    *dev = 0, *cu_count = 256;
    return RED_OK;
}
red_status host_scratch(int, hipStream_t, size_t bytes, void** out) {
    scratch.push_back(bytes);
    *out = reinterpret_cast<void*>((uintptr_t)1 << 50);
    return RED_OK;
}

hipError_t launch_plan_slots(const PlanSlots& a, int blocks, bool, hipStream_t) {
    launches.push_back({blocks < 1 ? 1 : blocks, 1024, a.tokens, at(a.lens), at(a.slots)});
    return hipSuccess;
}
hipError_t launch_page_bounds(int, int, int, int, const PageBounds& a, unsigned int blocks, unsigned int batch, hipStream_t) {
    launches.push_back({(int64_t)blocks * batch, kBoundsWaves * 64, batch, at(a.lens), at(a.table)});
    return hipSuccess;
}
hipError_t launch_select_pages(int, int, int, const SelectPages& a, hipStream_t) {
    const int64_t scores = (int64_t)(a.most + a.share - 1) / a.share * a.heads * a.batch * 256, chooses = (int64_t)a.heads * a.batch * 1024;
    launches.push_back({scores > chooses ? scores : chooses, 1, a.batch, at(a.lens), at(a.selected)});
    return hipSuccess;
}
hipError_t launch_sample(int, int, const Sample& a, unsigned int rows, hipStream_t) {
    const int64_t chunks = (int64_t)rows * a.chunks * 256, whole = (int64_t)rows * 1024;
    launches.push_back({chunks > whole ? chunks : whole, 1, rows, a.first_row, at(a.plans) + (int64_t)(rows * sizeof(SamplePlan))});
    return hipSuccess;
}

}  // namespace libred

extern "C" {

void forget() { scratch.clear(), launches.clear(); }

// The launches since forget(), 5 numbers each; -> how many.
int launched(int64_t* to, int most) {
    for (int i = 0; i < most && i < (int)launches.size(); ++i) {
        const Launch& l = launches[i];
        for (const int64_t v : {l.blocks, l.threads, l.items, l.in, l.out}) *to++ = v;
    }
    return (int)launches.size();
}

// Bytes of scratch that the calls since forget() asked for, at most.
size_t scratch_asked() {
    size_t most = 0;
    for (const size_t s : scratch) most = s > most ? s : most;
    return most;
}
int64_t scratch_at() { return (int64_t)1 << 50; }
}
