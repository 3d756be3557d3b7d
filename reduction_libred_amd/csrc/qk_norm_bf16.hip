// Norms of heads with the rotation: bfloat16.
#include "qk_norm.hpp"

namespace libred {

hipError_t launch_qk_norm_bf16(int vec, int lanes, const QkNorm& a, bool back, int blocks, hipStream_t stream) {
    return launch_qk_norm_type<BF16>(vec, lanes, a, back, blocks, stream);
}

}  // namespace libred
