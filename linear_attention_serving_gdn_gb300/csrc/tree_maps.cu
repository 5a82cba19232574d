// The maps of a step's trees of drafted tokens: each node's word (itself and
// the nodes above it) and its position, from the nodes' parents.
//
// A warp takes a request; words are joined along doubled pointers: after round
// r a node's word holds the 2^r nodes up from it and its pointer stands 2^r
// levels up, so 64 nodes in any shape take six rounds, and a chain no more than
// a bush.  16 bytes a token: bound by latency (cu_seqlens, the parents, the
// rounds, the writes; 8 requests 2.2 us on the GPU, 512 of up to 64 nodes 3.0)
// and, called alone, by the host's 5.1 us.
#include "paged.cuh"

namespace gdn {
namespace {

constexpr int kMapsWarps = 4;

__global__ void __launch_bounds__(kMapsWarps * 32) tree_maps_kernel(const TreeMapsArgs a) {
    __shared__ uint64_t s_word[kMapsWarps][kTreeNodes];
    __shared__ int32_t s_up[kMapsWarps][kTreeNodes];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t *word = s_word[warp];
    int32_t *up = s_up[warp];
    int32_t end = a.num_reqs > 0 ? a.cu_seqlens[a.num_reqs] : 0;  // of the tokens that requests may have
    if (end < 0 || end > a.num_tokens) end = static_cast<int32_t>(a.num_tokens);
    const int64_t warps = static_cast<int64_t>(gridDim.x) * kMapsWarps;
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * kMapsWarps + warp; r < a.num_reqs; r += warps) {
        const int32_t b = a.cu_seqlens[r], e = a.cu_seqlens[r + 1], kv = a.kv_lens[r];
        const bool range = b >= 0 && b <= e && e <= end;
        const int32_t m = range ? e - b : 0;
        const bool tree = m <= kTreeNodes, keys = kv >= m;
        if (lane == 0 && (!range || !tree || !keys)) report(a.dev_status, GDN_DEV_BAD_LENGTH);
        if (!tree) {
            for (int32_t u = lane; u < m; u += 32) {
                a.masks[b + u] = 0;
                a.positions[b + u] = 0;
            }
            continue;
        }
        for (int32_t u = lane; u < m; u += 32) {
            int32_t p = a.parents[b + u];
            if (p < -1 || p >= u) {
                report(a.dev_status, GDN_DEV_BAD_PARENT);
                p = -1;
            }
            word[u] = 1ull << u;
            up[u] = p;
        }
        __syncwarp();
        for (int32_t reach = 1; reach < m; reach *= 2) {
            uint64_t w[2];
            int32_t p[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int32_t u = lane + 32 * i;
                if (u >= m) continue;
                p[i] = up[u];
                w[i] = word[u];
                if (p[i] >= 0) {
                    w[i] |= word[p[i]];
                    p[i] = up[p[i]];
                }
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int32_t u = lane + 32 * i;
                if (u >= m) continue;
                word[u] = w[i];
                up[u] = p[i];
            }
            __syncwarp();
        }
        for (int32_t u = lane; u < m; u += 32) {
            a.masks[b + u] = word[u];
            a.positions[b + u] = keys ? kv - m + __popcll(word[u]) - 1 : 0;
        }
        __syncwarp();
    }
    for (int64_t t = end + static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; t < a.num_tokens;
         t += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        a.masks[t] = 0;
        a.positions[t] = 0;
    }
}

}  // namespace

cudaError_t launch_tree_maps(const TreeMapsArgs &a, cudaStream_t stream) {
    int dev = 0, sms = 0;
    if (!current_device(&dev, &sms)) return cudaErrorInvalidDevice;
    int64_t blocks = (static_cast<int64_t>(a.num_reqs) + kMapsWarps - 1) / kMapsWarps;
    const int64_t most = static_cast<int64_t>(sms) * 8;
    if (blocks > most) blocks = most;
    if (blocks < 1) blocks = 1;
    tree_maps_kernel<<<static_cast<unsigned>(blocks), kMapsWarps * 32, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace gdn
