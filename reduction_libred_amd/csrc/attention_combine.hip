// Attention of drafted tokens over a shared-out cache: joins the pieces of a
// row,
//     out = sum_c 2^(M_c - M) O_c / sum_c 2^(M_c - M) l_c,  M = max M_c,
// in their order, and the choice of the kernel by types.
#include "decode_common.hpp"

namespace libred {

namespace {

constexpr int kThreads = 256;

struct MaxOp {
    __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct AddOp {
    __device__ float operator()(float a, float b) const { return a + b; }
};

// A row is joined by WAVES waves of the block. Its pieces are taken 64 at a
// time: their weights first, then their sums, LANES lanes with 4 neighbouring
// columns each. Latency bounds it: one trip for the plan, one for weights and
// sums together (32 sequences x 256 rows of 128, 2 pieces a row, 12 MB: 6.8 us;
// 32 rows of 64 pieces: 4.0 us).
template <class T, int LANES, int WAVES>
__global__ __launch_bounds__(kThreads) void combine_kernel(TreeAttention a, int rows_a_block) {
    constexpr int kRowsHere = kThreads / kWave / WAVES, kSlices = WAVES * kWave / LANES;
    __shared__ f32x4 sums[WAVES > 1 ? kThreads : 1];
    asm volatile("" ::"s"(a.out), "s"(a.out_batch), "s"(a.cache.dim), "s"(a.lens), "s"(a.plan));  // one of every 64-byte line
    const int D = a.cache.dim, group = a.group, M = a.nodes * group, heads = a.cache.heads;
    const int tid = threadIdx.x % (WAVES * kWave), wl = threadIdx.x % kWave;
    const int rw = blockIdx.x * kRowsHere + __builtin_amdgcn_readfirstlane(threadIdx.x / (WAVES * kWave)), h = blockIdx.y, b = blockIdx.z;
    if (rw >= M) return;  // whole waves; with several waves a row, whole blocks
    const int node = rw / group, g = rw - node * group;
    int count;
    sequence_tokens(a, b, &count);
    const int per = a.plan[a.batch + 1], start = a.plan[b], seg_tiles = a.plan[b + 1] - start, per_seq = heads * a.row_blocks;
    const int rb = rw / rows_a_block, seg = h * a.row_blocks + rb;
    const int first = start * per_seq + seg * seg_tiles;
    int pieces = 0;
    int64_t slot = 0;
    if (node < count && seg_tiles > 0) {
        const int w0 = first / per, w1 = (first + seg_tiles - 1) / per;
        pieces = w1 - w0 + 1;
        slot = w0 + (int64_t)b * per_seq + seg;
    }
    const int64_t row0 = slot * rows_a_block + (rw - rb * rows_a_block);
    const int lane = tid % LANES, slice = tid / LANES, c = lane * 4;
    float m = -__builtin_inff(), l = 0.f;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    for (int k0 = 0; k0 < pieces; k0 += kWave) {
        const int here = min(pieces - k0, kWave);
        // The first sums are asked for together with the weights.
        f32x4 x[4];
        auto load = [&](int k1) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int k = k0 + min(k1 + u * kSlices + slice, here - 1);
                x[u] = *reinterpret_cast<const f32x4*>(a.part_o + (row0 + (int64_t)k * rows_a_block) * D + (c < D ? c : 0));
            }
        };
        float2 ml = a.part_ml[row0 + (int64_t)(k0 + min(wl, here - 1)) * rows_a_block];
        load(0);
        if (wl >= here) ml = make_float2(-__builtin_inff(), 0.f);
        const float to = fmaxf(m, group_combine<kWave>(ml.x, MaxOp()));
        // Powers of 2 in halves: with 8-bit values a sum may be as far above
        // its 2^M as their scales are apart.
        const float hf = m == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(0.5f * (m - to)), f = hf * hf;
        const float hw = ml.x == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(0.5f * (ml.x - to)), w = hw * hw;
        l = l * hf * hf + group_combine<kWave>(ml.y * hw * hw, AddOp());
        v *= f;
        m = to;
        for (int k1 = 0; k1 < here; k1 += 4 * kSlices) {
            if (k1 > 0) load(k1);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int k = k1 + u * kSlices + slice;
                const float wk = __shfl(w, min(k, here - 1));
                if (k < here) v += wk * x[u];
            }
        }
    }
    // Slices: those of a wave, then those of the block's waves.
    if constexpr (LANES < kWave) {
#pragma unroll
        for (int o = LANES; o < kWave; o <<= 1)
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] += __shfl_xor(v[j], o);
    }
    if constexpr (WAVES > 1) {
        sums[threadIdx.x] = v;
        __syncthreads();
        if (tid >= LANES) return;
#pragma unroll
        for (int w = 1; w < WAVES; ++w) v += sums[w * kWave + lane];
    }
    if (tid < LANES && c < D) {
        const bool empty = l == 0.f;
        const float inv = empty ? 0.f : 1.f / l;
        typename Vec<T, 4>::type out;
#pragma unroll
        for (int j = 0; j < 4; ++j) out[j] = empty ? (typename T::bits)0 : T::narrow(v[j] * inv);
        *reinterpret_cast<typename Vec<T, 4>::type*>(static_cast<typename T::bits*>(a.out) + b * a.out_batch +
                                                     node * a.out_node + (h * group + g) * a.out_head + c) = out;
        if (lane == 0)
            a.lse[((int64_t)b * a.nodes + node) * (heads * group) + h * group + g] =
                empty ? -__builtin_inff() : (m + __builtin_amdgcn_logf(l)) * 0.69314718055994531f;
    }
}

template <class T, int LANES>
hipError_t combine_lanes(const TreeAttention& a, int rows_a_block, hipStream_t stream) {
    const int64_t rows = (int64_t)a.batch * a.cache.heads * a.nodes * a.group;
    const unsigned int M = (unsigned)(a.nodes * a.group);
    // A block a row, or a wave: 32 rows of 64 pieces 4.0 us / 5.0, 1024 rows of
    // 16 pieces 4.5 / 4.2, 8192 rows of 2 pieces 19.8 / 6.8.
    const bool few = rows < 512;
    const dim3 grid(few ? M : (M + 3) / 4, (unsigned)a.cache.heads, (unsigned)a.batch);
    if (few)
        combine_kernel<T, LANES, 4><<<grid, kThreads, 0, stream>>>(a, rows_a_block);
    else
        combine_kernel<T, LANES, 1><<<grid, kThreads, 0, stream>>>(a, rows_a_block);
    return hipGetLastError();
}

template <class T>
hipError_t combine(const TreeAttention& a, int rows_a_block, hipStream_t stream) {
    if (a.cache.dim <= 64) return combine_lanes<T, 16>(a, rows_a_block, stream);
    if (a.cache.dim <= 128) return combine_lanes<T, 32>(a, rows_a_block, stream);
    return combine_lanes<T, 64>(a, rows_a_block, stream);
}

}  // namespace

hipError_t launch_attention_combine(int type, const TreeAttention& a, int rows_a_block, hipStream_t stream) {
    return type == RED_F16 ? combine<F16>(a, rows_a_block, stream) : combine<BF16>(a, rows_a_block, stream);
}

hipError_t launch_tree_attention(int type, int cache_type, const TreeAttention& a, hipStream_t stream) {
    if (type == RED_F16)
        return cache_type == RED_I8     ? launch_attention_f16_i8(a, stream)
               : cache_type == RED_E4M3 ? launch_attention_f16_e4m3(a, stream)
                                        : launch_attention_f16_16(a, stream);
    return cache_type == RED_I8     ? launch_attention_bf16_i8(a, stream)
           : cache_type == RED_E4M3 ? launch_attention_bf16_e4m3(a, stream)
                                    : launch_attention_bf16_16(a, stream);
}

}  // namespace libred
