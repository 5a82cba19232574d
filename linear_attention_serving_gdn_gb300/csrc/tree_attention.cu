// Attention of trees of drafted tokens over the paged K/V cache (paged_attention.cuh with kTree).
#include "paged_attention.cuh"

namespace gdn {

cudaError_t launch_tree_attention(const PagedAttentionArgs &a, cudaStream_t stream) {
    return launch_attention<true>(a, stream);
}

}  // namespace gdn
