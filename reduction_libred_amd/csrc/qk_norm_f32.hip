// Norms of heads with the rotation: float32, and the sum of the backward
// pass's weight partials.
#include "qk_norm.hpp"

namespace libred {

hipError_t launch_qk_norm_f32(int vec, int lanes, const QkNorm& a, bool back, int blocks, hipStream_t stream) {
    return launch_qk_norm_type<F32>(vec, lanes, a, back, blocks, stream);
}

// A block adds up 16 columns: a wave takes 4 rows of partials at a time, its 16
// waves every 16th group of 4, 8 loads a lane in flight (the sum is short and
// all latency: 1536 rows of 256 columns took 10.7 us with 64 columns a block,
// 4 blocks in all). float64, in a fixed order.
constexpr int kWeightWaves = 16, kWeightCols = 16;
__global__ __launch_bounds__(kWeightWaves* kWave) void qk_norm_weights_kernel(const float* partials, int blocks,
                                                                              int dim, float* dq, float* dk) {
    constexpr int U = 8, S = kWeightWaves * kWave / kWeightCols;  // rows at a time
    __shared__ double sums[kWeightWaves][kWeightCols];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, n = 2 * dim;
    const int col = blockIdx.x * kWeightCols + lane % kWeightCols, at = min(col, n - 1);
    double s = 0.0;
    for (int b0 = threadIdx.x / kWeightCols; b0 < blocks; b0 += S * U) {
        float x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = partials[(size_t)min(b0 + u * S, blocks - 1) * n + at];
#pragma unroll
        for (int u = 0; u < U; ++u) s += b0 + u * S < blocks ? (double)x[u] : 0.0;
    }
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if (lane < kWeightCols) sums[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && lane < kWeightCols && col < n) {
#pragma unroll
        for (int w = 1; w < kWeightWaves; ++w) s += sums[w][lane];
        float* out = col < dim ? dq : dk;
        if (out != nullptr) out[col < dim ? col : col - dim] = (float)s;
    }
}

hipError_t launch_qk_norm_weights(const float* partials, int blocks, int dim, float* dq_weight, float* dk_weight,
                                  hipStream_t stream) {
    qk_norm_weights_kernel<<<(2 * dim + kWeightCols - 1) / kWeightCols, kWeightWaves * kWave, 0, stream>>>(
        partials, blocks, dim, dq_weight, dk_weight);
    return hipGetLastError();
}

}  // namespace libred
