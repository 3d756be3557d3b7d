// Attention of drafted tokens: f16 queries over a cache of the same type.
#include "tree_attention.hpp"

namespace libred {

hipError_t launch_attention_f16_16(const TreeAttention& a, hipStream_t stream) {
    return launch_attention<F16, Cached16>(a, stream);
}

}  // namespace libred
