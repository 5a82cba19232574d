// Arguments of the paged K/V cache calls (maps of a step, K/V write, attention).
#pragma once

#include "gdn_internal.cuh"

namespace gdn {

struct PagedMapsArgs {
    int32_t num_reqs, page_size;
    int64_t num_pages;
    const int32_t *context_lens, *new_lens;
    int32_t *block_table;
    int32_t table_width;
    int64_t table_stride;
    const int32_t *free_pages;  // null: the table already covers the new tokens
    int32_t num_free;
    const int32_t *free_head;
    int32_t *free_head_out;
    int32_t *cu_seqlens, *kv_lens;
    int64_t token_capacity;
    int32_t *slot_map, *positions;
    bool aligned;  // slot_map and positions start at 16-byte boundaries
    int32_t *dev_status;
};

// One side (K or V) of the write: rows of [h][d] 16-bit elements into a cache.
struct PagedWriteSide {
    const uint16_t *src;
    int64_t token_stride, head_stride;
    uint16_t *dst;
    int64_t page_stride, slot_stride, dst_head_stride;
};

struct PagedWriteArgs {
    PagedWriteSide side[2];
    int64_t num_tokens;
    int32_t h, d, page_size;
    int64_t num_pages;
    const int32_t *slot_map;
    int32_t *dev_status;
};

struct PagedAttentionArgs {
    gdn_paged_cache_t cache;
    int32_t num_reqs, h_q, window;
    int64_t num_tokens;
    float scale;
    int64_t max_kv_len;
    const uint16_t *q;
    int64_t q_token_stride;
    const int32_t *block_table;
    int64_t table_stride;
    const int32_t *cu_seqlens, *kv_lens;
    uint16_t *o;
    void *workspace;
    int32_t *dev_status;
};

cudaError_t launch_paged_maps(const PagedMapsArgs &a, cudaStream_t stream);
cudaError_t launch_paged_write(const PagedWriteArgs &a, cudaStream_t stream);
cudaError_t launch_paged_attention(const PagedAttentionArgs &a, cudaStream_t stream);
// Device scratch of launch_paged_attention; arguments validated by the caller.
size_t paged_attention_workspace(int32_t h_q, int32_t h_kv, int32_t d, int32_t num_reqs, int64_t num_tokens,
                                 int64_t max_kv_len);

}  // namespace gdn
