// The entry points of libred_decode.h (decode.cpp, compiled for the host) over
// launchers that note what they are asked for and do nothing.
#include <vector>

#include "decode.cpp"

namespace {

std::vector<size_t> scratch;  // bytes asked for
std::vector<libred::CacheRows> cache_launches;

// What a launch was asked for: blocks (in x) of 256 threads, tokens or
// sequences, and where its first input, first output and positions, slots or
// lengths begin.
struct Launch {
    int64_t blocks, items, in, out, by;
};
std::vector<Launch> launches;

int64_t at(const void* p) { return (int64_t)(uintptr_t)p; }

hipError_t note(const libred::QkNorm& a, int blocks) {
    launches.push_back({blocks, a.tokens, at(a.q.p), at(a.q_out.p), at(a.pos)});
    return hipSuccess;
}
hipError_t note(const libred::CacheRows& a, unsigned groups) {
    cache_launches.push_back(a);
    launches.push_back({groups, a.tokens, at(a.k.p), at(a.v.p), at(a.slots)});
    return hipSuccess;
}

}  // namespace

namespace libred {

red_status host_fail(hipError_t, red_status code) { return code; }
red_status host_compute_units(int* dev, int* cu_count) {
    *dev = 0, *cu_count = 256;
    return RED_OK;
}
red_status host_scratch(int, hipStream_t, size_t bytes, void** out) {
    scratch.push_back(bytes);
    *out = reinterpret_cast<void*>((uintptr_t)1 << 40);
    return RED_OK;
}

hipError_t launch_qk_norm_f32(int, int, const QkNorm& a, bool, int blocks, hipStream_t) { return note(a, blocks); }
hipError_t launch_qk_norm_f16(int, int, const QkNorm& a, bool, int blocks, hipStream_t) { return note(a, blocks); }
hipError_t launch_qk_norm_bf16(int, int, const QkNorm& a, bool, int blocks, hipStream_t) { return note(a, blocks); }
hipError_t launch_qk_norm_weights(const float*, int, int, float*, float*, hipStream_t) { return hipSuccess; }
hipError_t launch_cache_write(int, int, int, int, const CacheRows& a, unsigned int n, hipStream_t) { return note(a, n); }
hipError_t launch_cache_read(int, int, int, int, const CacheRows& a, unsigned int n, hipStream_t) { return note(a, n); }
hipError_t launch_attention_combine(int, const TreeAttention&, int, hipStream_t) { return hipSuccess; }
hipError_t launch_tree_attention(int, int, const TreeAttention& a, hipStream_t) {
    const int64_t segments = (int64_t)a.batch * a.cache.heads * a.row_blocks;
    launches.push_back({a.blocks ? a.blocks : segments, a.batch, at(a.q), at(a.out), at(a.lens)});
    return hipSuccess;
}
hipError_t launch_verify(int, const Verify&, hipStream_t) { return hipSuccess; }

}  // namespace libred

extern "C" {

void forget() { scratch.clear(), cache_launches.clear(), launches.clear(); }

// The launches since forget(), 5 numbers each; -> how many.
int launched(int64_t* to, int most) {
    for (int i = 0; i < most && i < (int)launches.size(); ++i) {
        const Launch& l = launches[i];
        for (const int64_t v : {l.blocks, l.items, l.in, l.out, l.by}) *to++ = v;
    }
    return (int)launches.size();
}

// Bytes from `base` on that the last launch on a cache loads for a token whose
// slot lies outside the cache: of elements (what 0) or scales (what 1). Such a
// token's loads are those of the cache's first row of every head.
int64_t outside_reads(const void* base, int what) {
    const libred::CacheRows& a = cache_launches.back();
    const libred::PagedCache& c = a.cache;
    int64_t end = 0;
    for (const void* p : {static_cast<const void*>(what ? c.k_scales : c.k), static_cast<const void*>(what ? c.v_scales : c.v)}) {
        const int64_t last = (c.heads - 1) * (what ? c.scale_head_stride : c.head_stride);
        const int64_t bytes = what ? 4 * (last + 1) : 2 * (last + c.dim);  // elements of at most 2 bytes
        const int64_t e = (int64_t)((uintptr_t)p - (uintptr_t)base) + bytes;
        if (e > end) end = e;
    }
    return end;
}
}

// Bytes of scratch that the calls since forget() asked for, at most.
extern "C" size_t scratch_asked() {
    size_t most = 0;
    for (const size_t s : scratch) most = s > most ? s : most;
    return most;
}

extern "C" int share_size(int all, int blocks) { return libred::share_size(all, blocks); }
extern "C" int share_begin(int all, int per, int share) { return libred::share_begin(all, per, share); }
