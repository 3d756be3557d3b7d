// Attention of drafted tokens: bf16 queries over a cache of i8.
#include "tree_attention.hpp"

namespace libred {

hipError_t launch_attention_bf16_i8(const TreeAttention& a, hipStream_t stream) {
    return launch_attention<BF16, CachedI8>(a, stream);
}

}  // namespace libred
