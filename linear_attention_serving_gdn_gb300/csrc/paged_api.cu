// C ABI of the paged K/V cache calls: host-side validation, then launches on
// the caller's stream.  See include/gdn.h for the contract of each entry point.
#include <limits.h>
#include <math.h>

#include "paged.cuh"

namespace {

constexpr int64_t kMaxStride = int64_t{1} << 39;  // elements: a tensor map's strides are under 2^40 bytes
constexpr int64_t kMaxKeys = int64_t{1} << 30;    // keys of a request: key indices stay inside int32
constexpr int32_t kMaxHeads = 65536;              // K/V heads: pieces of a token stay inside int32
constexpr int32_t kMaxGroup = 128;  // query heads per K/V head: one token's heads fit a 128-row tile

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// A stride matters only where its dimension has more than one entry; an unused
// one is replaced by the row length, so that tensor maps always see a valid value.
bool stride_ok(int64_t *stride, int64_t entries, int64_t row) {
    if (entries <= 1) *stride = row;
    return *stride > 0 && *stride % 8 == 0 && *stride < kMaxStride;
}

// Checks a cache description and fills unused strides of the copy.
gdn_status_t cache_ok(const gdn_paged_cache_t *in, gdn_paged_cache_t *c) {
    if (!in) return GDN_ERR_INVALID_ARG;
    *c = *in;
    if (c->h_kv <= 0 || c->d <= 0 || c->page_size <= 0 || c->num_pages <= 0) return GDN_ERR_INVALID_ARG;
    if (c->dtype != GDN_BF16 && c->dtype != GDN_FP16) return GDN_ERR_UNSUPPORTED;
    if (c->d != 64 && c->d != 128 && c->d != 256) return GDN_ERR_UNSUPPORTED;
    if (c->page_size % 16 != 0 || c->h_kv > kMaxHeads) return GDN_ERR_UNSUPPORTED;
    if (c->num_pages > INT_MAX / c->page_size) return GDN_ERR_UNSUPPORTED;
    if (!c->k || !c->v) return GDN_ERR_INVALID_ARG;
    if (!aligned16(c->k) || !aligned16(c->v)) return GDN_ERR_INVALID_ARG;
    if (!stride_ok(&c->k_page_stride, c->num_pages, c->d) || !stride_ok(&c->v_page_stride, c->num_pages, c->d) ||
        !stride_ok(&c->k_slot_stride, c->page_size, c->d) || !stride_ok(&c->v_slot_stride, c->page_size, c->d) ||
        !stride_ok(&c->k_head_stride, c->h_kv, c->d) || !stride_ok(&c->v_head_stride, c->h_kv, c->d))
        return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status_t gdn_paged_maps(int32_t num_reqs, int32_t page_size, int64_t num_pages, const int32_t *context_lens,
                            const int32_t *new_lens, int32_t *block_table, int32_t table_width,
                            int64_t table_stride, const int32_t *free_pages, int32_t num_free,
                            const int32_t *free_head, int32_t *free_head_out, int32_t *cu_seqlens,
                            int32_t *kv_lens, int64_t token_capacity, int32_t *slot_map, int32_t *positions,
                            int32_t *dev_status, void *stream) {
    if (num_reqs < 0 || page_size <= 0 || num_pages < 0 || table_width < 0 || token_capacity < 0 || num_free < 0)
        return GDN_ERR_INVALID_ARG;
    if (num_pages > INT_MAX / page_size || token_capacity > INT_MAX) return GDN_ERR_UNSUPPORTED;
    if (!cu_seqlens || (token_capacity > 0 && (!slot_map || !positions))) return GDN_ERR_INVALID_ARG;
    if (num_reqs > 0 && (!context_lens || !new_lens || !kv_lens)) return GDN_ERR_INVALID_ARG;
    if (num_reqs > 0 && table_width > 0 && (!block_table || table_stride < table_width)) return GDN_ERR_INVALID_ARG;
    if (free_pages && (!free_head || !free_head_out)) return GDN_ERR_INVALID_ARG;
    gdn::PagedMapsArgs a{};
    a.num_reqs = num_reqs;
    a.page_size = page_size;
    a.num_pages = num_pages;
    a.context_lens = context_lens;
    a.new_lens = new_lens;
    a.block_table = block_table;
    a.table_width = table_width;
    a.table_stride = table_stride;
    a.free_pages = free_pages;
    a.num_free = num_free;
    a.free_head = free_head;
    a.free_head_out = free_head_out;
    a.cu_seqlens = cu_seqlens;
    a.kv_lens = kv_lens;
    a.token_capacity = token_capacity;
    a.slot_map = slot_map;
    a.positions = positions;
    a.dev_status = dev_status;
    return gdn::launch_paged_maps(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status_t gdn_paged_kv_write(const gdn_paged_cache_t *cache, int64_t num_tokens, const void *k,
                                int64_t k_token_stride, int64_t k_head_stride, const void *v,
                                int64_t v_token_stride, int64_t v_head_stride, const int32_t *slot_map,
                                int32_t *dev_status, void *stream) {
    gdn_paged_cache_t c;
    const gdn_status_t s = cache_ok(cache, &c);
    if (s != GDN_OK) return s;
    if (num_tokens < 0) return GDN_ERR_INVALID_ARG;
    if (num_tokens > INT_MAX) return GDN_ERR_UNSUPPORTED;
    if (num_tokens == 0) return GDN_OK;
    if (!k || !v || !slot_map || !aligned16(k) || !aligned16(v)) return GDN_ERR_INVALID_ARG;
    if (!stride_ok(&k_token_stride, num_tokens, c.d) || !stride_ok(&v_token_stride, num_tokens, c.d) ||
        !stride_ok(&k_head_stride, c.h_kv, c.d) || !stride_ok(&v_head_stride, c.h_kv, c.d))
        return GDN_ERR_INVALID_ARG;
    gdn::PagedWriteArgs a{};
    a.side[0] = {static_cast<const uint16_t *>(k), k_token_stride, k_head_stride, static_cast<uint16_t *>(c.k),
                 c.k_page_stride, c.k_slot_stride, c.k_head_stride};
    a.side[1] = {static_cast<const uint16_t *>(v), v_token_stride, v_head_stride, static_cast<uint16_t *>(c.v),
                 c.v_page_stride, c.v_slot_stride, c.v_head_stride};
    a.num_tokens = num_tokens;
    a.h = c.h_kv;
    a.d = c.d;
    a.page_size = c.page_size;
    a.num_pages = c.num_pages;
    a.slot_map = slot_map;
    a.dev_status = dev_status;
    return gdn::launch_paged_write(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_paged_attention_workspace_bytes(int32_t h_q, int32_t h_kv, int32_t d, int32_t num_reqs,
                                           int64_t num_tokens, int64_t max_kv_len) {
    if (h_q <= 0 || h_kv <= 0 || h_q % h_kv != 0 || h_q / h_kv > kMaxGroup || (d != 64 && d != 128 && d != 256) ||
        num_reqs < 0 || num_tokens < 0 || num_tokens > INT_MAX || max_kv_len < 0 || max_kv_len > kMaxKeys)
        return static_cast<size_t>(-1);
    // The call takes 0 for what its block table holds, which is not known here: enough for any table.
    return gdn::paged_attention_workspace(h_q, h_kv, d, num_reqs, num_tokens, max_kv_len > 0 ? max_kv_len : kMaxKeys);
}

gdn_status_t gdn_paged_attention(const gdn_paged_cache_t *cache, int32_t num_reqs, int64_t num_tokens, int32_t h_q,
                                 float scale, int32_t window, int64_t max_kv_len, const void *q,
                                 int64_t q_token_stride, const int32_t *block_table, int32_t table_width,
                                 int64_t table_stride, const int32_t *cu_seqlens, const int32_t *kv_lens, void *o,
                                 void *workspace, size_t workspace_bytes, int32_t *dev_status, void *stream) {
    gdn::PagedAttentionArgs a{};
    const gdn_status_t s = cache_ok(cache, &a.cache);
    if (s != GDN_OK) return s;
    const gdn_paged_cache_t &c = a.cache;
    if (num_reqs < 0 || num_tokens < 0 || h_q <= 0 || h_q % c.h_kv != 0 || window < 0 || table_width < 0)
        return GDN_ERR_INVALID_ARG;
    if (!(scale >= 0.f) || isinf(scale)) return GDN_ERR_INVALID_ARG;
    if (h_q / c.h_kv > kMaxGroup || num_tokens > INT_MAX || num_tokens > INT_MAX / h_q) return GDN_ERR_UNSUPPORTED;
    const int64_t table_tokens = static_cast<int64_t>(table_width) * c.page_size;
    if (max_kv_len < 0 || max_kv_len > table_tokens) return GDN_ERR_INVALID_ARG;
    if (max_kv_len == 0) max_kv_len = table_tokens < kMaxKeys ? table_tokens : kMaxKeys;
    if (max_kv_len > kMaxKeys) return GDN_ERR_UNSUPPORTED;
    if (num_tokens == 0) return GDN_OK;
    if (!q || !o || !cu_seqlens || !aligned16(q) || !aligned16(o)) return GDN_ERR_INVALID_ARG;
    if (num_reqs > 0 && (!kv_lens || (table_width > 0 && (!block_table || table_stride < table_width))))
        return GDN_ERR_INVALID_ARG;
    const int64_t q_row = static_cast<int64_t>(h_q) * c.d;
    if (!stride_ok(&q_token_stride, num_tokens, q_row) || q_token_stride < q_row) return GDN_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return GDN_ERR_WORKSPACE;
    const size_t need = gdn::paged_attention_workspace(h_q, c.h_kv, c.d, num_reqs, num_tokens, max_kv_len);
    if (need > 0 && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
    a.num_reqs = num_reqs;
    a.h_q = h_q;
    a.window = window;
    a.num_tokens = num_tokens;
    a.scale = scale;
    a.max_kv_len = max_kv_len;
    a.q = static_cast<const uint16_t *>(q);
    a.q_token_stride = q_token_stride;
    a.block_table = block_table;
    a.table_stride = table_stride;
    a.cu_seqlens = cu_seqlens;
    a.kv_lens = kv_lens;
    a.o = static_cast<uint16_t *>(o);
    a.workspace = workspace;
    a.dev_status = dev_status;
    return gdn::launch_paged_attention(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
