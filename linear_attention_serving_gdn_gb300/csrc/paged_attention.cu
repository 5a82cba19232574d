// Attention of new tokens over the paged K/V cache, each token behind the one before it (paged_attention.cuh).
#include "paged_attention.cuh"

namespace gdn {

size_t paged_attention_workspace(int32_t h_q, int32_t h_kv, int32_t d, int32_t num_reqs, int64_t num_tokens,
                                 int64_t max_kv_len) {
    return workspace_at(nullptr, h_q, h_kv, d, num_reqs, num_tokens, max_kv_len).bytes;
}

cudaError_t launch_paged_attention(const PagedAttentionArgs &a, cudaStream_t stream) {
    return launch_attention<false>(a, stream);
}

}  // namespace gdn
