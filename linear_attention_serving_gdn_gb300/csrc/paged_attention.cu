// Attention of a chunk of new tokens over the paged K/V cache.
//
// One warp per (token, query head): lane l holds d/32 elements of q and of the
// output; the keys the token sees are walked in order with a running maximum
// and sum (one pass over K and V, softmax statistics in fp32).
#include "paged.cuh"

#include <cuda_fp16.h>

namespace gdn {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float to_float(uint16_t b, bool fp16) {
    return fp16 ? __half2float(__ushort_as_half(b)) : bf16_bits_to_float(b);
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) attention_rows_kernel(const PagedAttentionArgs a) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (row >= a.num_tokens * a.h_q) return;
    const int64_t t = row / a.h_q;
    const int head = static_cast<int>(row - t * a.h_q);
    const gdn_paged_cache_t &c = a.cache;
    const bool fp16 = c.dtype == GDN_FP16;
    const int kvh = head / (a.h_q / c.h_kv);
    float q[E], o[E] = {};
    float m = -INFINITY, l = 0.f;
    // request of token t: the last r whose range [cu[r], cu[r + 1]) holds it
    int r = -1;
    for (int base = 0; base < a.num_reqs; base += 32) {
        const int i = base + lane;
        const bool in = i < a.num_reqs && a.cu_seqlens[i] <= t && t < a.cu_seqlens[i + 1];
        const unsigned hit = __ballot_sync(0xffffffffu, in);
        if (hit) {
            r = base + __ffs(hit) - 1;
            break;
        }
    }
    int64_t lo = 0, hi = 0;
    if (r >= 0) {
        const int32_t first = a.cu_seqlens[r], last = a.cu_seqlens[r + 1], kv = a.kv_lens[r];
        if (first < 0 || last > a.num_tokens || kv < 0 || kv > a.max_kv_len) {
            if (lane == 0) report(a.dev_status, GDN_DEV_BAD_LENGTH);
        } else {
            hi = static_cast<int64_t>(kv) - last + t + 1;
            lo = a.window > 0 && hi > a.window ? hi - a.window : 0;
        }
    }
    const float sc = a.scale * 1.4426950408889634f;
#pragma unroll
    for (int e = 0; e < E; ++e)
        q[e] = to_float(a.q[t * a.q_token_stride + static_cast<int64_t>(head) * D + e * 32 + lane], fp16);
    for (int64_t j = lo; j < hi; ++j) {
        const int64_t idx = j / c.page_size, in = j - idx * c.page_size;
        const int32_t page = a.block_table[r * a.table_stride + idx];
        const bool good = page >= 0 && page < c.num_pages;
        if (!good && lane == 0) report(a.dev_status, GDN_DEV_BAD_SLOT);
        const uint16_t *k = static_cast<const uint16_t *>(c.k) + page * c.k_page_stride + in * c.k_slot_stride +
                            kvh * c.k_head_stride;
        const uint16_t *v = static_cast<const uint16_t *>(c.v) + page * c.v_page_stride + in * c.v_slot_stride +
                            kvh * c.v_head_stride;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(q[e], good ? to_float(k[e * 32 + lane], fp16) : 0.f, s);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= sc;
        const float mn = fmaxf(m, s);
        const float f = mn == -INFINITY ? 1.f : exp2f(m - mn), p = mn == -INFINITY ? 0.f : exp2f(s - mn);
        m = mn;
        l = l * f + p;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(p, good ? to_float(v[e * 32 + lane], fp16) : 0.f, o[e] * f);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float x = l == 0.f ? 0.f : o[e] * inv;
        a.o[row * D + e * 32 + lane] = fp16 ? __half_as_ushort(__float2half_rn(x)) : float_to_bf16_bits(x);
    }
}

}  // namespace

size_t paged_attention_workspace(int32_t, int32_t, int32_t, int32_t, int64_t, int64_t) { return 0; }

cudaError_t launch_paged_attention(const PagedAttentionArgs &a, cudaStream_t stream) {
    const unsigned blocks = static_cast<unsigned>((a.num_tokens * a.h_q + kWarps - 1) / kWarps);
    switch (a.cache.d) {
        case 64: attention_rows_kernel<64><<<blocks, kWarps * 32, 0, stream>>>(a); break;
        case 128: attention_rows_kernel<128><<<blocks, kWarps * 32, 0, stream>>>(a); break;
        default: attention_rows_kernel<256><<<blocks, kWarps * 32, 0, stream>>>(a); break;
    }
    return cudaGetLastError();
}

}  // namespace gdn
