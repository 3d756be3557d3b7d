// Attention of drafted tokens over a split cache: joins the chunks of a row,
//     out = sum_c 2^(M_c - M) O_c / sum_c 2^(M_c - M) l_c,  M = max M_c,
// in the order of the chunks, and the choice of the kernel by types.
#include "decode_common.hpp"

namespace libred {

namespace {

constexpr int kThreads = 256;

struct MaxOp {
    __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
};

// One block a row: first the weight of every chunk, then the chunks in
// kThreads / LANES slices, each lane with 4 neighbouring columns.
template <class T, int LANES>
__global__ __launch_bounds__(kThreads) void combine_kernel(TreeAttention a) {
    constexpr int kSlices = kThreads / LANES;
    __shared__ float weight[kAttentionMaxSplits], red[2][kThreads / kWave];
    __shared__ f32x4 sums[kThreads];
    const int D = a.cache.dim, group = a.group, M = a.nodes * group, heads = a.cache.heads;
    const int tid = threadIdx.x, rw = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    const int node = rw / group, g = rw - node * group;
    const int count = a.count ? min(max(a.count[b], 0), a.nodes) : a.nodes;
    const int64_t lenb = max(a.lens[b], 0);
    const int total = (int)min(lenb + count, (int64_t)a.max_tokens);
    const int chunks = node < count ? (total + a.chunk - 1) / a.chunk : 0;
    const int64_t row0 = ((int64_t)b * heads + h) * a.splits * M + rw;  // of chunk c: + c * M
    float2 ml = make_float2(-__builtin_inff(), 0.f);
    if (tid < chunks) ml = a.part_ml[row0 + (int64_t)tid * M];
    float m = group_combine<kWave>(ml.x, MaxOp());
    if (tid % kWave == 0) red[0][tid / kWave] = m;
    __syncthreads();
    m = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    const float w = ml.x == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(ml.x - m);
    weight[tid] = w;
    const float lw = group_sum<kWave>(w * ml.y);
    if (tid % kWave == 0) red[1][tid / kWave] = lw;
    __syncthreads();
    const float l = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
    const int lane = tid % LANES, slice = tid / LANES, c = lane * 4;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (c < D)
        for (int k = slice; k < chunks; k += kSlices)
            v += weight[k] * *reinterpret_cast<const f32x4*>(a.part_o + (row0 + (int64_t)k * M) * D + c);
    sums[tid] = v;
    __syncthreads();
    if (slice == 0 && c < D) {
#pragma unroll
        for (int s = 1; s < kSlices; ++s) v += sums[s * LANES + lane];
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

template <class T>
hipError_t combine(const TreeAttention& a, hipStream_t stream) {
    const dim3 grid((unsigned)(a.nodes * a.group), (unsigned)a.cache.heads, (unsigned)a.batch);
    if (a.cache.dim <= 64)
        combine_kernel<T, 16><<<grid, kThreads, 0, stream>>>(a);
    else if (a.cache.dim <= 128)
        combine_kernel<T, 32><<<grid, kThreads, 0, stream>>>(a);
    else
        combine_kernel<T, 64><<<grid, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attention_combine(int type, const TreeAttention& a, hipStream_t stream) {
    return type == RED_F16 ? combine<F16>(a, stream) : combine<BF16>(a, stream);
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
