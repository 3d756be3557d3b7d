// Attention of drafted tokens: bf16 queries over a cache of e4m3.
#include "tree_attention.hpp"

namespace libred {

hipError_t launch_attention_bf16_e4m3(const TreeAttention& a, hipStream_t stream) {
    return launch_attention<BF16, CachedE4M3>(a, stream);
}

}  // namespace libred
