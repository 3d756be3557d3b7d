// host.hpp -- what the C entry points share on the host: argument checks,
// device facts, the per-(device, stream) scratch and the last HIP error.
// Defined in libred.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <map>
#include <mutex>
#include <utility>

#include "libred.h"

namespace libred {

// Record `e` as the calling thread's last HIP error and return `code`.
red_status host_fail(hipError_t e, red_status code);
// Number of compute units of the current device.
red_status host_compute_units(int* dev, int* cu_count);
// Calls on one stream take turns: held by a call from before it asks for the
// buffers of (dev, stream) until its last launch is enqueued. The launches of a
// call hand each other results through these buffers, so those of two host
// threads that use the same stream must not come between each other. Streams have
// a lock each, since an enqueue may block until another stream gets on. (Looking it
// up and taking it: 40 ns.)
class StreamTurn {
public:
    StreamTurn(int dev, hipStream_t stream) : lock_(of(dev, stream)) {}

private:
    static std::mutex& of(int dev, hipStream_t stream) {
        static std::mutex guard;
        static std::map<std::pair<int, hipStream_t>, std::mutex> turns;  // a node stays where it is
        const std::lock_guard<std::mutex> lock(guard);
        return turns[std::make_pair(dev, stream)];
    }
    std::lock_guard<std::mutex> lock_;
};
// The scratch buffer of (dev, stream), at least `bytes` long. The caller has the
// stream's turn.
red_status host_scratch(int dev, hipStream_t stream, size_t bytes, void** out);

inline bool is_aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

}  // namespace libred
