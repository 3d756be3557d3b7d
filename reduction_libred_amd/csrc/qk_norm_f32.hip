// Norms of heads with the rotation: float32, and the sum of the backward
// pass's weight partials.
#include "qk_norm.hpp"

namespace libred {

hipError_t launch_qk_norm_f32(int vec, int lanes, const QkNorm& a, bool back, int blocks, hipStream_t stream) {
    return launch_qk_norm_type<F32>(vec, lanes, a, back, blocks, stream);
}

// One column a lane, 16 waves that each take every 16th block's row of
// partials; float64, in a fixed order.
constexpr int kWeightWaves = 16;
__global__ __launch_bounds__(kWeightWaves* kWave) void qk_norm_weights_kernel(const float* partials, int blocks,
                                                                              int dim, float* dq, float* dk) {
    __shared__ double sums[kWeightWaves][kWave];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int col = blockIdx.x * kWave + lane;
    double s = 0.0;
    if (col < 2 * dim) {
        // 16 loads in flight: the sum is short and all latency.
        constexpr int U = 16;
        for (int b0 = wave; b0 < blocks; b0 += kWeightWaves * U) {
            float x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int b = b0 + u * kWeightWaves;
                x[u] = partials[(size_t)min(b, blocks - 1) * 2 * dim + col];
            }
#pragma unroll
            for (int u = 0; u < U; ++u) s += b0 + u * kWeightWaves < blocks ? (double)x[u] : 0.0;
        }
    }
    sums[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && col < 2 * dim) {
        for (int w = 1; w < kWeightWaves; ++w) s += sums[w][lane];
        float* out = col < dim ? dq : dk;
        if (out != nullptr) out[col < dim ? col : col - dim] = (float)s;
    }
}

hipError_t launch_qk_norm_weights(const float* partials, int blocks, int dim, float* dq_weight, float* dk_weight,
                                  hipStream_t stream) {
    qk_norm_weights_kernel<<<(2 * dim + kWave - 1) / kWave, kWeightWaves * kWave, 0, stream>>>(partials, blocks, dim,
                                                                                          dq_weight, dk_weight);
    return hipGetLastError();
}

}  // namespace libred
