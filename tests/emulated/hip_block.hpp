// A block of GPU threads as host threads: what the kernels of libred need to be
// compiled for the host and run there, one thread a lane, so that a test can
// hold one wave back at every barrier and see what the others do meanwhile.
// Stands in for hip/hip_runtime.h.
#pragma once

#include <pthread.h>
#include <stddef.h>
#include <stdint.h>
#include <string.h>
#include <time.h>

#include <algorithm>
#include <cmath>
#include <functional>
#include <thread>
#include <vector>

#define __device__
#define __host__
#define __global__
#define __forceinline__ inline
#define __shared__ static
#define __launch_bounds__(...)
#define __align__(n) alignas(n)

typedef int hipError_t;
typedef void* hipStream_t;
constexpr hipError_t hipSuccess = 0;
struct float2 {
    float x, y;
};
inline float2 make_float2(float x, float y) { return float2{x, y}; }
using std::max;
using std::min;

namespace emulated {

struct Index {
    unsigned x, y, z;
};
inline thread_local Index thread_index, block_index;
inline Index grid_size{1, 1, 1};
inline pthread_barrier_t block_barrier;
inline std::vector<pthread_barrier_t> wave_barriers;
inline std::vector<uint64_t> lanes;  // what the lanes of every wave hand each other
inline int late_wave = -1;           // the wave that is held back after every barrier

inline unsigned wave() { return thread_index.x / 64; }
inline unsigned lane() { return thread_index.x % 64; }

inline void block_sync() {
    pthread_barrier_wait(&block_barrier);
    if ((int)wave() == late_wave) {
        timespec t = {0, 5000000};
        nanosleep(&t, nullptr);
    }
}

// Every lane of the wave hands over `v`; -> what get(values of the 64) makes of it.
template <class F>
inline auto exchange(uint64_t v, F get) {
    uint64_t* own = &lanes[wave() * 64];
    own[lane()] = v;
    pthread_barrier_wait(&wave_barriers[wave()]);
    auto r = get(own);
    pthread_barrier_wait(&wave_barriers[wave()]);
    return r;
}

inline int dpp(int old, int src, int ctrl, int row_mask) {
    const int l = (int)lane(), row = l / 16;
    int from = -1;
    if (ctrl < 0x100) from = l / 4 * 4 + (ctrl >> (2 * (l % 4)) & 3);                      // quad_perm
    else if (ctrl >= 0x111 && ctrl <= 0x11F) from = l % 16 >= ctrl - 0x110 ? l - (ctrl - 0x110) : -1;  // row_shr
    else if (ctrl == 0x140) from = row * 16 + 15 - l % 16;                                 // row_mirror
    else if (ctrl == 0x141) from = l / 8 * 8 + 7 - l % 8;                                  // row_half_mirror
    else if (ctrl == 0x142) from = row > 0 ? row * 16 - 1 : -1;                            // row_bcast:15
    else if (ctrl == 0x143) from = row > 1 ? 31 : -1;                                      // row_bcast:31
    const int got = exchange((uint32_t)src, [&](const uint64_t* x) { return from < 0 ? 0 : (int)(uint32_t)x[from]; });
    return from < 0 || !(row_mask >> row & 1) ? old : got;
}

template <class T>
inline T shuffle(T v, int from) {
    uint64_t w = 0;
    memcpy(&w, &v, sizeof(T));
    w = exchange(w, [&](const uint64_t* x) { return x[from]; });
    memcpy(&v, &w, sizeof(T));
    return v;
}

// Run body() as a block of `threads` lanes, block (x, y) of a grid of `grid_x`.
inline void run_block(int threads, unsigned grid_x, unsigned x, unsigned y, const std::function<void()>& body) {
    grid_size.x = grid_x;
    lanes.assign(threads, 0);
    pthread_barrier_init(&block_barrier, nullptr, threads);
    wave_barriers.resize(threads / 64);
    for (auto& b : wave_barriers) pthread_barrier_init(&b, nullptr, 64);
    std::vector<std::thread> all;
    for (int t = 0; t < threads; ++t)
        all.emplace_back([&, t] {
            thread_index = {(unsigned)t, 0, 0};
            block_index = {x, y, 0};
            body();
        });
    for (auto& t : all) t.join();
}

}  // namespace emulated

#define threadIdx emulated::thread_index
#define blockIdx emulated::block_index
#define gridDim emulated::grid_size
#define __syncthreads emulated::block_sync
#define __ballot(is)                                                                \
    emulated::exchange((is) ? 1 : 0, [](const uint64_t* x) {                        \
        uint64_t m = 0;                                                             \
        for (int i = 0; i < 64; ++i) m |= x[i] << i;                                \
        return m;                                                                   \
    })
#define __ffsll __builtin_ffsll
#define __clzll __builtin_clzll
#define __shfl_xor(v, o) emulated::shuffle(v, (int)emulated::lane() ^ (o))
#define __builtin_amdgcn_update_dpp(old, src, ctrl, rows, banks, bound) emulated::dpp(old, src, ctrl, rows)
#define __builtin_amdgcn_readlane(v, l) emulated::shuffle(v, l)
#define __builtin_amdgcn_readfirstlane(v) emulated::shuffle((int)(v), 0)
#define __builtin_amdgcn_fence(...)
#define __builtin_amdgcn_wave_barrier()
