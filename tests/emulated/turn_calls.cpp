// Calls of several host threads on one stream: decode.cpp and serve.cpp (compiled
// for the host beside this file) over launchers that look whether another call
// has asked for the stream's buffers since their own did.
#include <atomic>
#include <chrono>
#include <map>
#include <mutex>
#include <thread>
#include <vector>

#include "serve.hpp"

namespace {

using std::this_thread::get_id;
std::mutex guard;
std::map<hipStream_t, std::thread::id> owner;  // the call that asked for the buffers of a stream last
std::atomic<int> mixed, entered, met;
thread_local bool meets = false;  // this thread's next launch waits for another thread's

void pause() { std::this_thread::sleep_for(std::chrono::microseconds(200)); }

// A launch that hands something on through the buffers.
hipError_t launch(hipStream_t s) {
    auto look = [&] {
        const std::lock_guard<std::mutex> lock(guard);
        if (owner[s] != get_id()) ++mixed;
    };
    look();
    if (meets) {  // 5 s at most
        meets = false, ++entered;
        for (int i = 0; i < 25000 && entered < 2; ++i) pause();
        met += entered == 2;
    }
    pause();
    look();
    return hipSuccess;
}

}  // namespace

namespace libred {

red_status host_fail(hipError_t, red_status code) { return code; }
red_status host_compute_units(int* dev, int* cu_count) {
    *dev = 0, *cu_count = 256;
    return RED_OK;
}
red_status host_scratch(int, hipStream_t s, size_t, void** out) {
    {
        const std::lock_guard<std::mutex> lock(guard);
        owner[s] = get_id();
    }
    pause();
    *out = reinterpret_cast<void*>((uintptr_t)1 << 50);
    return RED_OK;
}

hipError_t launch_qk_norm_f32(int, int, const QkNorm&, bool, int, hipStream_t s) { return launch(s); }
hipError_t launch_qk_norm_f16(int, int, const QkNorm&, bool, int, hipStream_t s) { return launch(s); }
hipError_t launch_qk_norm_bf16(int, int, const QkNorm&, bool, int, hipStream_t s) { return launch(s); }
hipError_t launch_qk_norm_weights(const float*, int, int, float*, float*, hipStream_t s) { return launch(s); }
hipError_t launch_cache_write(int, int, int, int, const CacheRows&, unsigned int, hipStream_t) { return hipSuccess; }
hipError_t launch_cache_read(int, int, int, int, const CacheRows&, unsigned int, hipStream_t) { return hipSuccess; }
hipError_t launch_tree_attention(int, int, const TreeAttention&, hipStream_t s) { return launch(s); }
hipError_t launch_attention_combine(int, const TreeAttention&, int, hipStream_t s) { return launch(s); }
hipError_t launch_verify(int, const Verify&, hipStream_t s) { return launch(s); }
hipError_t launch_plan_slots(const PlanSlots&, int, bool, hipStream_t s) { return launch(s); }
hipError_t launch_page_bounds(int, int, int, int, const PageBounds&, unsigned int, unsigned int, hipStream_t) { return hipSuccess; }
hipError_t launch_select_pages(int, int, int, const SelectPages&, hipStream_t s) { return launch(s); }
hipError_t launch_sample(int, int, const Sample&, unsigned int, hipStream_t s) { return launch(s); }

}  // namespace libred

namespace {

// One of the calls whose launches share buffers, by its number.
struct Call {
    int what;
    const void *a, *dq, *dk;
    red_status operator()(hipStream_t s) const {
        switch (what) {
            case 0: return red_plan_slots(static_cast<const red_plan_slots_args*>(a), s);
            case 1: return red_select_pages(static_cast<const red_select_pages_args*>(a), s);
            case 2: return red_sample(static_cast<const red_sample_args*>(a), s);
            case 3: return red_tree_attention(static_cast<const red_tree_attention_args*>(a), s);
            case 4: return red_verify_drafts(static_cast<const red_verify_drafts_args*>(a), s);
            default: return red_qk_norm_rope_backward(static_cast<const red_qk_norm_rope_args*>(a), static_cast<const red_heads*>(dq),
                                                      static_cast<const red_heads*>(dk), nullptr, nullptr, s);
        }
    }
};

hipStream_t stream_of(int n) { return reinterpret_cast<hipStream_t>((uintptr_t)(n + 1) << 8); }

}  // namespace

extern "C" {

// `threads` host threads that make the call `times` each, on one stream. -> how
// often a launch met another call's buffers, -1 where a call failed.
int on_one_stream(int what, const void* a, const void* dq, const void* dk, int threads, int times) {
    const Call call{what, a, dq, dk};
    mixed = 0;
    std::atomic<bool> fine{true};
    std::vector<std::thread> all;
    for (int t = 0; t < threads; ++t)
        all.emplace_back([&] {
            for (int i = 0; i < times; ++i)
                if (call(stream_of(0)) != RED_OK) fine = false;
        });
    for (std::thread& t : all) t.join();
    return fine ? mixed.load() : -1;
}

// Two host threads that make the call once, on a stream each. -> how many were in
// their first launch at the same time.
int on_two_streams(int what, const void* a, const void* dq, const void* dk) {
    const Call call{what, a, dq, dk};
    entered = met = 0;
    std::thread one([&] { meets = true, call(stream_of(1)); }), two([&] { meets = true, call(stream_of(2)); });
    one.join(), two.join();
    return met;
}
}
