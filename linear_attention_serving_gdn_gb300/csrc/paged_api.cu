// C ABI of the paged K/V cache calls, the maps of trees and the rotary positions: host-side validation, then launches on
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
bool aligned8(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

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

// gdn_paged_attention, or with `tree` gdn_tree_attention.
gdn_status_t attention_impl(const gdn_paged_cache_t *cache, int32_t num_reqs, int64_t num_tokens, int32_t h_q, float scale,
                            int32_t window, int64_t max_kv_len, const void *q, int64_t q_token_stride,
                            const int32_t *block_table, int32_t table_width, int64_t table_stride,
                            const int32_t *cu_seqlens, const int32_t *kv_lens, bool tree, const uint64_t *masks, void *o,
                            void *workspace, size_t workspace_bytes, int32_t *dev_status, cudaStream_t stream) {
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
    if (tree && (!masks || !aligned8(masks))) return GDN_ERR_INVALID_ARG;
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
    a.masks = masks;
    a.o = static_cast<uint16_t *>(o);
    a.workspace = workspace;
    a.dev_status = dev_status;
    const cudaError_t e = tree ? gdn::launch_tree_attention(a, stream) : gdn::launch_paged_attention(a, stream);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

constexpr int32_t kMaxRotaryDim = 1024;
constexpr int64_t kMaxRotaryStride = int64_t{1} << 39;

// Whether no two of the rows of d elements at t * token_stride + h * head_stride share one; strides of d to kMaxRotaryStride.
// Rows h heads apart meet those of a token whose distance is nearest to theirs, or none.  (The products stay under 2^56.)
bool rows_apart(int64_t tokens, int64_t token_stride, int64_t heads, int64_t head_stride, int64_t d) {
    if (tokens <= 1 || heads <= 1 || token_stride >= (heads - 1) * head_stride + d) return true;
    if ((head_stride - d) / token_stride >= tokens - 1) return true;
    for (int64_t h = 1; h < heads; ++h) {
        const int64_t far = h * head_stride, t = far / token_stride;  // t tokens are that far or nearer, t + 1 farther
        if ((t > 0 && t < tokens && far - t * token_stride < d) || (t + 1 < tokens && (t + 1) * token_stride - far < d))
            return false;
    }
    return true;
}

// One side of a rotation; strides that matter only.
gdn_status_t rotary_side_ok(const gdn_rotary_side_t &in, int64_t num_tokens, int32_t d, gdn::RotarySide *out) {
    if (in.heads < 0) return GDN_ERR_INVALID_ARG;
    if (in.heads > kMaxHeads) return GDN_ERR_UNSUPPORTED;
    if (in.heads == 0 || num_tokens == 0) return GDN_OK;
    if (!in.x || !in.out) return GDN_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(in.x) | reinterpret_cast<uintptr_t>(in.out)) & 1u) return GDN_ERR_INVALID_ARG;
    gdn::RotarySide s = {static_cast<const uint16_t *>(in.x), in.x_token_stride, in.x_head_stride,
                         static_cast<uint16_t *>(in.out), in.out_token_stride, in.out_head_stride, in.heads};
    // (an unused stride must not decide on the access width)
    if (num_tokens == 1) s.token_stride = s.dst_token_stride = 0;
    if (in.heads == 1) s.head_stride = s.dst_head_stride = 0;
    auto bad = [](int64_t stride, int64_t entries, int64_t least) {
        return entries > 1 && (stride < least || stride > kMaxRotaryStride);
    };
    // Inputs may be shared by tokens or heads (stride 0); outputs may not.
    if (bad(s.token_stride, num_tokens, 0) || bad(s.head_stride, in.heads, 0) || bad(s.dst_token_stride, num_tokens, d) ||
        bad(s.dst_head_stride, in.heads, d) || !rows_apart(num_tokens, s.dst_token_stride, in.heads, s.dst_head_stride, d))
        return GDN_ERR_INVALID_ARG;
    if (s.src == s.dst && (s.token_stride != s.dst_token_stride || s.head_stride != s.dst_head_stride))
        return GDN_ERR_INVALID_ARG;
    *out = s;
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
    return attention_impl(cache, num_reqs, num_tokens, h_q, scale, window, max_kv_len, q, q_token_stride, block_table,
                          table_width, table_stride, cu_seqlens, kv_lens, false, nullptr, o, workspace, workspace_bytes,
                          dev_status, static_cast<cudaStream_t>(stream));
}

gdn_status_t gdn_tree_attention(const gdn_paged_cache_t *cache, int32_t num_reqs, int64_t num_tokens, int32_t h_q,
                                float scale, int64_t max_kv_len, const void *q, int64_t q_token_stride,
                                const int32_t *block_table, int32_t table_width, int64_t table_stride,
                                const int32_t *cu_seqlens, const int32_t *kv_lens, const uint64_t *masks, void *o,
                                void *workspace, size_t workspace_bytes, int32_t *dev_status, void *stream) {
    return attention_impl(cache, num_reqs, num_tokens, h_q, scale, 0, max_kv_len, q, q_token_stride, block_table,
                          table_width, table_stride, cu_seqlens, kv_lens, true, masks, o, workspace, workspace_bytes,
                          dev_status, static_cast<cudaStream_t>(stream));
}

gdn_status_t gdn_tree_maps(int32_t num_reqs, int64_t num_tokens, const int32_t *parents, const int32_t *cu_seqlens,
                           const int32_t *kv_lens, uint64_t *masks, int32_t *positions, int32_t *dev_status,
                           void *stream) {
    if (num_reqs < 0 || num_tokens < 0) return GDN_ERR_INVALID_ARG;
    if (num_tokens > INT_MAX) return GDN_ERR_UNSUPPORTED;
    if (num_tokens == 0) return GDN_OK;
    if (!parents || !masks || !positions || (num_reqs > 0 && (!cu_seqlens || !kv_lens))) return GDN_ERR_INVALID_ARG;
    if (!aligned8(masks)) return GDN_ERR_INVALID_ARG;
    gdn::TreeMapsArgs a{};
    a.num_reqs = num_reqs;
    a.num_tokens = num_tokens;
    a.parents = parents;
    a.cu_seqlens = cu_seqlens;
    a.kv_lens = kv_lens;
    a.masks = masks;
    a.positions = positions;
    a.dev_status = dev_status;
    return gdn::launch_tree_maps(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status_t gdn_rotary(int32_t dtype, int64_t num_tokens, int32_t d, int32_t rotary_dim, int32_t interleaved,
                        float magnitude, const int32_t *positions, const uint64_t *frequencies,
                        const gdn_rotary_side_t *q, const gdn_rotary_side_t *k, void *stream) {
    if (num_tokens < 0 || d <= 0 || rotary_dim <= 0 || rotary_dim > d || rotary_dim % 2 != 0 || !isfinite(magnitude))
        return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_BF16 && dtype != GDN_FP16) return GDN_ERR_UNSUPPORTED;
    if (num_tokens > INT_MAX || d > kMaxRotaryDim) return GDN_ERR_UNSUPPORTED;
    gdn::RotaryArgs a{};
    const gdn_rotary_side_t *const sides[2] = {q, k};
    for (int i = 0; i < 2; ++i)
        if (sides[i]) {
            const gdn_status_t s = rotary_side_ok(*sides[i], num_tokens, d, &a.side[i]);
            if (s != GDN_OK) return s;
        }
    if (a.side[0].h + a.side[1].h == 0) return q || k ? GDN_OK : GDN_ERR_INVALID_ARG;
    if (num_tokens == 0) return GDN_OK;
    if (!positions || !frequencies || !aligned8(frequencies)) return GDN_ERR_INVALID_ARG;
    a.num_tokens = num_tokens;
    a.d = d;
    a.rot = rotary_dim;
    a.dtype = dtype;
    a.interleaved = interleaved != 0;
    a.magnitude = magnitude;
    a.positions = positions;
    a.frequencies = frequencies;
    return gdn::launch_rotary(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status_t gdn_rotary_frequencies(int32_t rotary_dim, double base, int32_t scaling, double factor,
                                    int64_t original_length, double beta_fast, double beta_slow, uint64_t *out) {
    constexpr double kTwoPi = 6.283185307179586476925;
    if (rotary_dim <= 0 || rotary_dim % 2 != 0 || !out || !(base > 1.) || !isfinite(base)) return GDN_ERR_INVALID_ARG;
    if (scaling < GDN_ROTARY_NONE || scaling > GDN_ROTARY_YARN) return GDN_ERR_UNSUPPORTED;
    if (scaling != GDN_ROTARY_NONE && (!(factor >= 1.) || !isfinite(factor))) return GDN_ERR_INVALID_ARG;
    const double rot = rotary_dim;
    double lo = 0., hi = 0., slow = 0.;  // ends of the ramp; the pair that makes beta_slow turns
    if (scaling == GDN_ROTARY_NTK) {
        if (rotary_dim <= 2) return GDN_ERR_INVALID_ARG;
        base *= pow(factor, rot / (rot - 2.));
    } else if (scaling == GDN_ROTARY_YARN) {
        if (original_length <= 0 || !(beta_slow > 0.) || !(beta_fast >= beta_slow) || !isfinite(beta_fast))
            return GDN_ERR_INVALID_ARG;
        // The pair that makes `turns` turns over the original length.
        auto pair = [&](double turns) { return rot * log(static_cast<double>(original_length) / (turns * kTwoPi)) / (2. * log(base)); };
        lo = fmax(floor(pair(beta_fast)), 0.);
        slow = pair(beta_slow);
        hi = fmin(ceil(slow), rot - 1.);
    }
    for (int32_t i = 0; i < rotary_dim / 2; ++i) {
        double f = pow(base, -2. * i / rot);
        if (scaling == GDN_ROTARY_LINEAR) f /= factor;
        if (scaling == GDN_ROTARY_YARN) {
            // (slow < 0: all pairs turn less, pair 0 too, which the clamped ramp begins with)
            const double ramp = slow < 0. ? 1. : fmin(fmax((i - lo) / fmax(hi - lo, 0.001), 0.), 1.);
            f = f * (1. - ramp) + f / factor * ramp;
        }
        out[i] = static_cast<uint64_t>(nearbyint(ldexp(f / kTwoPi, 64)));  // (at most a sixth of a turn)
    }
    return GDN_OK;
}

}  // extern "C"
