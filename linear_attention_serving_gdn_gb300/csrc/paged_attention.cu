// Attention of a chunk of new tokens over the paged K/V cache.
//
// For query row (token u, head) of a request, with s_j = scale q.K_j over the
// keys j it sees:  o = sum_j exp(s_j - m) V_j / sum_j exp(s_j - m).  One pass
// over the keys in tiles of 128: with running maximum m, sum l and
// accumulator O, a tile adds  P = exp2(c S - c m),  l += sum P,  O += P V
// (c = scale log2 e), and when m grows, l and O are multiplied by
// exp2(c (m_old - m)).
//
// Rows.  The h_q / h_kv query heads of a K/V head share its keys, so a tile of
// 128 rows holds 128 / (h_q / h_kv) tokens times those heads: every K/V tile
// is read once for all of them, and a single token's heads ride in one tile.
//
// Work items.  (request, K/V head, row tile, range of key tiles).  Where a
// request's own row tiles cannot fill the GPU, its keys are cut into splits,
// whose partial (O, m, l) a second kernel joins in split order.  The cut
// depends on the request's lengths alone (plan_request), never on the batch,
// so a request's bits do not change with what else is in the step.  A
// persistent grid (one block per SM) takes the items round robin; lengths are
// read on the device, so a captured call replays for others.
//
// One block, eight warps:
//   load   TMA boxes of K and V (one per page piece) into a ring of stages
//          128 keys x up to 128 columns, running ahead over item borders
//   mma    S = Q K^T (two TMEM buffers, so that the next tile's scores are
//          computed while this one's weights are), O += P V with P from TMEM
//   sched  walks the requests, cutting them into items
//   spare  TMEM allocation, zeros for padding tokens
//   4 softmax warps, one row per thread: S from TMEM, masks, maximum, exp2,
//          P back to TMEM over S; at the end O from TMEM to memory
//
// The running maximum only moves when it grows by more than 2^8: weights are
// then at most 2^8, exact in the sums, and O is rarely touched.  The rule is
// per row, so a row's bits do not depend on its neighbours.
//
// Every wait is bounded: one that runs out sets GDN_DEV_TIMEOUT and a flag
// that ends all the others; before the block leaves, its MMAs and copies in
// flight are waited for and TMEM is freed.
#include "paged.cuh"
#include "tc_ptx.cuh"

#include <cuda.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>
#include <limits.h>

#ifndef GDN_WAIT_CYCLES
#define GDN_WAIT_CYCLES 2000000000LL
#endif

namespace gdn {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();  // prefill.cu

namespace {

// A tensor of 16-bit elements, dims and strides (bytes, from dimension 1 on)
// innermost first; boxes land in the 128-byte-swizzled layout.
bool encode_tiles(CUtensorMap *m, const void *base, int dtype, int rank, const cuuint64_t *dims,
                  const cuuint64_t *strides, const cuuint32_t *box) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint32_t one[4] = {1, 1, 1, 1};
    return enc(m, dtype == GDN_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
               static_cast<cuuint32_t>(rank), const_cast<void *>(base), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kThreads = 256;
constexpr int kRows = 128;   // query rows of a tile (TMEM lanes)
constexpr int kKeys = 128;   // keys of a tile
constexpr int kPanel = 16384;  // 128 rows of 64 16-bit elements
constexpr int kItems = 4;    // items between the scheduler and the other warps
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 256;  // O after the two S buffers

// Splits.  A request alone should fill kSplitUnits SMs; the constant stands in
// for the SM count so that results do not depend on the device.
constexpr int kSplitUnits = 152;
constexpr int kMaxSplits = 64;
constexpr int kMinSplitTiles = 2;

struct Plan {
    int32_t row_tiles;    // tiles of query rows
    int32_t tile_tokens;  // tokens of one
    int32_t split_tiles;  // key tiles of a split
    int32_t split0, splits;
    int64_t items;
    int64_t partials;  // (token, split) pairs that leave partial results
};

__host__ __device__ __forceinline__ int32_t ceil_div(int32_t a, int32_t b) { return (a + b - 1) / b; }

// Key tiles [lo, hi) that tokens [u, u + n) of a request see together.
__device__ __forceinline__ void key_tiles(int32_t kv, int32_t m, int32_t u, int32_t n, int32_t window, int32_t *lo,
                                          int32_t *hi) {
    const int32_t first = kv - m + u, last = first + n;  // positions [first, last)
    *hi = last > 0 ? ceil_div(last, kKeys) : 0;
    *lo = window > 0 && first >= window ? (first - window + 1) / kKeys : 0;
    if (*lo > *hi) *lo = *hi;
}

// How a request of m new tokens and kv keys is cut; depends on nothing else of the batch.
__device__ __forceinline__ Plan plan_request(int32_t kv, int32_t m, int32_t group, int32_t h_kv, int32_t window) {
    Plan p;
    p.tile_tokens = kRows / group;
    p.row_tiles = ceil_div(m, p.tile_tokens);
    int32_t lo, hi;
    key_tiles(kv, m, 0, m, window, &lo, &hi);
    p.split_tiles = INT_MAX;
    p.split0 = 0;
    p.splits = 1;
    const int64_t units = static_cast<int64_t>(p.row_tiles) * h_kv;
    if (m > 0 && units * 2 <= kSplitUnits) {
        int32_t want = kSplitUnits / static_cast<int32_t>(units);
        if (want > kMaxSplits) want = kMaxSplits;
        const int32_t even = ceil_div(hi - lo, want);
        p.split_tiles = even > kMinSplitTiles ? even : kMinSplitTiles;
        p.split0 = lo / p.split_tiles;
        p.splits = hi > lo ? (hi - 1) / p.split_tiles - p.split0 + 1 : 1;
    }
    p.items = units * p.splits;
    p.partials = p.splits > 1 ? static_cast<int64_t>(m) * p.splits : 0;
    return p;
}

// Bound of `partials` over the requests of a call: at most `want` splits and
// one more where a window starts inside one, and never more than the longest
// context has.
int64_t partials_bound(int32_t group, int32_t h_kv, int32_t num_reqs, int64_t num_tokens, int64_t max_kv_len) {
    const int64_t tiles = (max_kv_len + kKeys - 1) / kKeys;
    if (h_kv * 2 > kSplitUnits || tiles <= kMinSplitTiles || num_tokens == 0 || num_reqs == 0) return 0;
    const int32_t want = kSplitUnits / h_kv < kMaxSplits ? kSplitUnits / h_kv : kMaxSplits;
    const int64_t by_length = (tiles + kMinSplitTiles - 1) / kMinSplitTiles;
    const int64_t splits = want < by_length ? want : by_length;
    // m tokens make at least m / tile_tokens row tiles, so m * want <= tile_tokens * kSplitUnits / h_kv
    const int64_t by_request = static_cast<int64_t>(num_reqs) * (kRows / group) * ceil_div(kSplitUnits, h_kv);
    const int64_t by_token = num_tokens * splits;
    return (by_token < by_request ? by_token : by_request) + num_tokens;
}

// Workspace: first partial of each request, then (m, l) and O of the partials.
struct Workspace {
    int64_t *base;
    float2 *ml;
    float *o;
    size_t bytes;
};
Workspace workspace_at(void *ws, int32_t num_reqs, int64_t partials, int32_t h_q, int32_t d) {
    auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
    Workspace w;
    char *p = static_cast<char *>(ws);
    const size_t rows = static_cast<size_t>(partials) * h_q;
    w.base = reinterpret_cast<int64_t *>(p);
    size_t at = up(static_cast<size_t>(num_reqs) * sizeof(int64_t));
    w.ml = reinterpret_cast<float2 *>(p + at);
    at += up(rows * sizeof(float2));
    w.o = reinterpret_cast<float *>(p + at);
    w.bytes = at + rows * d * sizeof(float);
    return w;
}

struct AttentionLaunch {
    CUtensorMap tm_q;      // [T][h_q][d]: boxes of a full tile's tokens x group x 64
    CUtensorMap tm_q_one;  // the same, one token
    CUtensorMap tm_k, tm_v;  // [page][head][row][d]: boxes of box_rows x 64
    PagedAttentionArgs a;
    Workspace ws;       // o null: no request of this call can be split
    int64_t partials;   // that the workspace holds
    int32_t group, box_rows;
    float c;  // scale * log2(e)
};

struct Item {
    int32_t stop;
    int32_t req, head;  // request, K/V head
    int32_t tok, n;     // first token (row of q) and tokens of the row tile
    int32_t pos;        // position of the first token
    int32_t lo, hi;     // key tiles
    int32_t splits;     // of the request
    int64_t partial;    // first token's partial, or -1: the item gives the final result
};

template <int D>
struct Shape {
    static constexpr int kCols = D < 128 ? D : 128;  // columns of a stage
    static constexpr int kHalves = D / kCols;        // stages of a K or V tile
    static constexpr int kPanels = kCols / 64;
    static constexpr uint32_t kStage = kPanels * kPanel;
    static constexpr uint32_t kQ = D / 64 * kPanel;
    // As many stages as 227 KB hold beside Q and 1.5 KB of barriers and items.
    static constexpr int kStages = (227 * 1024 - 1024 - 1536 - static_cast<int>(kQ)) / static_cast<int>(kStage);
    static constexpr uint32_t kSmem = 1024 + kQ + kStages * kStage + 1536;
};

template <int D>
struct Control {
    uint64_t kv_full[Shape<D>::kStages], kv_empty[Shape<D>::kStages];
    uint64_t q_full, q_empty;
    uint64_t s_full[2], p_full[2];
    uint64_t o_done, o_free;
    uint64_t item_full[kItems], item_empty[kItems];
    uint64_t drain;
    Item items[kItems];
    uint32_t tmem;
    int fail;
};

constexpr long long kWaitCycles = GDN_WAIT_CYCLES;
constexpr long long kDrainCycles = 2000000000LL;

// Bounded wait for the phase of `bar` with the given parity; gives up as soon
// as any thread has flagged a failure, and flags one when it runs out.
struct Waiter {
    int *fail;
    int32_t *status;
    __device__ __forceinline__ bool operator()(uint64_t *bar, uint32_t parity) const {
        if (tc::mbar_try_wait(bar, parity)) return true;
        const long long start = clock64();
        while (!tc::mbar_try_wait(bar, parity)) {
            if (*reinterpret_cast<volatile int *>(fail)) return false;
            if (clock64() - start > kWaitCycles) {
                atomicExch(fail, 1);
                report(status, GDN_DEV_TIMEOUT);
                return false;
            }
        }
        return true;
    }
    // The same for a whole warp: true for all lanes or for none.
    __device__ __forceinline__ bool all(uint64_t *bar, uint32_t parity) const {
        return __all_sync(0xffffffffu, (*this)(bar, parity));
    }
};
__device__ __forceinline__ void drain_bar(uint64_t *bar, uint32_t parity) {
    const long long start = clock64();
    while (!tc::mbar_try_wait(bar, parity))
        if (clock64() - start > kDrainCycles) return;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <bool kHalf>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    if (kHalf)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// ---- the scheduler: requests into items -----------------------------------------

struct Request {
    int32_t first, m, kv;
};
// Lengths of request r; m = 0 (nothing to do) where its token range is bad, kv = 0 (no keys) where its length is.
__device__ __forceinline__ Request load_request(const PagedAttentionArgs &a, int64_t r, bool tell) {
    Request q = {0, 0, 0};
    if (r < a.num_reqs) {
        const int32_t b = a.cu_seqlens[r], e = a.cu_seqlens[r + 1], kv = a.kv_lens[r];
        const bool range = b >= 0 && b <= e && e <= a.num_tokens, len = kv >= 0 && kv <= a.max_kv_len;
        if (range) q = {b, e - b, len ? kv : 0};
        if (tell && (!range || !len)) report(a.dev_status, GDN_DEV_BAD_LENGTH);
    }
    return q;
}

template <int D>
__device__ void schedule(const AttentionLaunch &L, Control<D> *ctl, const Waiter &wait) {
    const PagedAttentionArgs &a = L.a;
    const int lane = threadIdx.x & 31;
    const bool first_block = blockIdx.x == 0;
    uint32_t n = 0;
    auto publish = [&](const Item &it) {
        const uint32_t s = n % kItems;
        if (!wait.all(ctl->item_empty + s, (n / kItems & 1) ^ 1)) return false;
        if (lane == 0) {
            ctl->items[s] = it;
            tc::mbar_arrive(ctl->item_full + s);
        }
        ++n;
        __syncwarp();
        return true;
    };
    int64_t next = blockIdx.x, items0 = 0, partials0 = 0;
    for (int64_t base = 0; base < a.num_reqs; base += 32) {
        const Request q = load_request(a, base + lane, first_block);
        const Plan p = plan_request(q.kv, q.m, L.group, a.cache.h_kv, a.window);
        int64_t items = p.items, partials = p.partials;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, items, o), y = __shfl_up_sync(0xffffffffu, partials, o);
            if (lane >= o) {
                items += x;
                partials += y;
            }
        }
        if (first_block && L.ws.o && base + lane < a.num_reqs) L.ws.base[base + lane] = partials0 + partials - p.partials;
        const int64_t group_items = __shfl_sync(0xffffffffu, items, 31);
        while (next < items0 + group_items) {
            const int src = __ffs(__ballot_sync(0xffffffffu, items0 + items > next)) - 1;
            // Items of a request: row tiles of one (split, head) next to each other, longest first.
            const int64_t local = next - items0 - __shfl_sync(0xffffffffu, items - p.items, src);
            const int32_t m = __shfl_sync(0xffffffffu, q.m, src), kv = __shfl_sync(0xffffffffu, q.kv, src);
            const int32_t row_tiles = __shfl_sync(0xffffffffu, p.row_tiles, src);
            const int32_t split_tiles = __shfl_sync(0xffffffffu, p.split_tiles, src);
            const int32_t split0 = __shfl_sync(0xffffffffu, p.split0, src);
            const int32_t splits = __shfl_sync(0xffffffffu, p.splits, src);
            const int32_t first = __shfl_sync(0xffffffffu, q.first, src);
            const int64_t pbase = partials0 + __shfl_sync(0xffffffffu, partials - p.partials, src);
            const int32_t tile = row_tiles - 1 - static_cast<int32_t>(local % row_tiles);
            const int32_t rest = static_cast<int32_t>(local / row_tiles);
            const int32_t head = rest % a.cache.h_kv, split = split0 + rest / a.cache.h_kv;
            Item it;
            it.stop = 0;
            it.req = static_cast<int32_t>(base) + src;
            it.head = head;
            const int32_t u = tile * p.tile_tokens;
            it.n = m - u < p.tile_tokens ? m - u : p.tile_tokens;
            it.tok = first + u;
            it.pos = kv - m + u;
            it.splits = splits;
            int32_t lo, hi;
            key_tiles(kv, m, u, it.n, a.window, &lo, &hi);
            const bool whole = hi == lo || lo / split_tiles == (hi - 1) / split_tiles;
            const int64_t s_lo = static_cast<int64_t>(split) * split_tiles, s_hi = s_lo + split_tiles;
            it.lo = s_lo > lo ? static_cast<int32_t>(s_lo) : lo;
            it.hi = s_hi < hi ? static_cast<int32_t>(s_hi) : hi;
            it.partial = whole ? -1 : pbase + static_cast<int64_t>(u) * splits + (split - split0);
            // Token ranges that overlap can ask for more partials than there are tokens for.
            if (!whole && pbase + static_cast<int64_t>(m) * splits > L.partials) {
                if (lane == 0) report(a.dev_status, GDN_DEV_BAD_LENGTH);
                next += gridDim.x;
                continue;
            }
            // A split past what the tile sees has nothing to do; a tile that sees nothing is written by the first.
            if (it.lo < it.hi || (lo == hi && split == split0)) {
                if (it.lo >= it.hi) it.lo = it.hi = 0;
                if (!publish(it)) return;
            }
            next += gridDim.x;
        }
        items0 += group_items;
        partials0 += __shfl_sync(0xffffffffu, partials, 31);
    }
    Item end = {};
    end.stop = 1;
    publish(end);
}

// Key rows [*lo, *hi) that some token of the item sees (over all splits).
__device__ __forceinline__ void visible_rows(const Item &it, int32_t window, int32_t *lo, int32_t *hi) {
    *hi = it.pos + it.n;
    *lo = window > 0 && it.pos >= window ? it.pos - window + 1 : 0;
}

// ---- the load warp -------------------------------------------------------------------

template <int D>
__device__ void load_tiles(const AttentionLaunch &L, Control<D> *ctl, uint32_t q_smem, uint32_t ring, const Waiter &wait) {
    using Sh = Shape<D>;
    const PagedAttentionArgs &a = L.a;
    const int lane = threadIdx.x & 31;
    const int boxes = kKeys / L.box_rows;
    const int box = lane % boxes, panel = lane / boxes;
    const uint32_t dst = panel * kPanel + box * L.box_rows * 128;
    uint32_t stage = 0, phase = 0, filled = 0, q_loads = 0;
    // One stage: columns [half * kCols, + kCols) of a tile, one box per lane.
    auto fill = [&](const CUtensorMap *map, int32_t page, int32_t row, int32_t head, int half) {
        if (!wait.all(ctl->kv_empty + stage, phase ^ 1)) return false;
        if (lane == 0) tc::mbar_expect_tx(ctl->kv_full + stage, Sh::kStage);
        __syncwarp();
        if (panel < Sh::kPanels)
            tc::tma_load_4d(ring + stage * Sh::kStage + dst, map, half * Sh::kCols + panel * 64, row, head, page,
                            ctl->kv_full + stage);
        ++filled;
        if (++stage == Sh::kStages) {
            stage = 0;
            phase ^= 1;
        }
        return true;
    };
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
        const uint32_t s = n % kItems;
        if (!wait.all(ctl->item_full + s, n / kItems & 1)) break;
        const Item it = ctl->items[s];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(ctl->item_empty + s);
        if (it.stop) break;
        if (it.lo >= it.hi) continue;
        if (!wait.all(&ctl->q_empty, (q_loads & 1) ^ 1)) break;
        // Few tokens: a box per token and panel, one per lane, instead of the full tile's.
        constexpr int kQPanels = D / 64;
        const bool few = it.n * kQPanels <= 32 && it.n < kRows / L.group;
        const uint32_t token_bytes = L.group * 128u;
        if (lane == 0)
            tc::mbar_expect_tx(&ctl->q_full, kQPanels * token_bytes * static_cast<uint32_t>(few ? it.n : kRows / L.group));
        __syncwarp();
        if (few) {
            if (lane < it.n * kQPanels)
                tc::tma_load_3d(q_smem + lane % kQPanels * kPanel + lane / kQPanels * token_bytes, &L.tm_q_one,
                                lane % kQPanels * 64, it.head * L.group, it.tok + lane / kQPanels, &ctl->q_full);
        } else if (lane < kQPanels) {
            tc::tma_load_3d(q_smem + lane * kPanel, &L.tm_q, lane * 64, it.head * L.group, it.tok, &ctl->q_full);
        }
        ++q_loads;
        int32_t row_lo, row_hi;
        visible_rows(it, a.window, &row_lo, &row_hi);
        // Page and row of this lane's box of a tile.  A box that no token sees, or whose page id is bad, is loaded
        // from past the last page: TMA fills it with zeros.
        const int32_t none = static_cast<int32_t>(a.cache.num_pages);
        auto lookup = [&](int32_t tile, int32_t *page, int32_t *row) {
            const int32_t key = tile * kKeys + box * L.box_rows;
            *page = none;
            *row = 0;
            if (tile < it.hi && key < row_hi && key + L.box_rows > row_lo) {
                const int32_t idx = key / a.cache.page_size;
                const int32_t id = a.block_table[it.req * a.table_stride + idx];
                if (id >= 0 && id < none) {
                    *page = id;
                    *row = key - idx * a.cache.page_size;
                } else {
                    report(a.dev_status, GDN_DEV_BAD_SLOT);
                }
            }
        };
        int32_t k_page, k_row, v_page = none, v_row = 0;
        lookup(it.lo, &k_page, &k_row);
        for (int32_t t = it.lo; ok && t <= it.hi; ++t) {  // K of tile t, then V of tile t - 1
            int32_t next_page, next_row;
            lookup(t + 1, &next_page, &next_row);
            if (t < it.hi)
                for (int h = 0; ok && h < Sh::kHalves; ++h) ok = fill(&L.tm_k, k_page, k_row, it.head, h);
            if (t > it.lo)
                for (int h = 0; ok && h < Sh::kHalves; ++h) ok = fill(&L.tm_v, v_page, v_row, it.head, h);
            v_page = k_page;
            v_row = k_row;
            k_page = next_page;
            k_row = next_row;
        }
    }
    // Copies still in flight land before the block may leave.
    if (q_loads > 0) drain_bar(&ctl->q_full, (q_loads - 1) & 1);
    for (uint32_t i = 0; i < Sh::kStages && i < filled; ++i) {
        const uint32_t f = filled - 1 - i;
        drain_bar(ctl->kv_full + f % Sh::kStages, f / Sh::kStages & 1);
    }
}

// ---- the MMA warp (one thread) -----------------------------------------------------------

template <int D, bool kHalf>
__device__ void issue_products(Control<D> *ctl, uint32_t q_smem, uint32_t ring, uint32_t tmem, const Waiter &wait) {
    using Sh = Shape<D>;
    constexpr uint32_t kType = kHalf ? 0u : tc::kIdescBf16;
    constexpr uint32_t kIdescS = tc::idesc_f16_f32acc(kRows, kKeys) | kType;
    constexpr uint32_t kIdescO = tc::idesc_f16_f32acc(kRows, Sh::kCols) | kType | tc::kIdescBmn;
    uint32_t stage = 0, phase = 0, tile = 0, n_items = 0;
    auto next_stage = [&]() {
        tc::mma_commit(ctl->kv_empty + stage);
        if (++stage == Sh::kStages) {
            stage = 0;
            phase ^= 1;
        }
    };
    // O (+)= P V of the tile whose number is g
    auto weights = [&](uint32_t g, bool first) {
        if (!wait(ctl->p_full + (g & 1), g >> 1 & 1)) return false;
        if (first && !wait(&ctl->o_free, (n_items & 1) ^ 1)) return false;
        for (int h = 0; h < Sh::kHalves; ++h) {
            if (!wait(ctl->kv_full + stage, phase)) return false;
            tc::fence_after_sync();
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k)
                tc::mma_f16_ta(tmem + kTmemO + h * Sh::kCols, tmem + (g & 1) * kKeys + k * 8,
                               tc::desc_mn_sw128(ring + stage * Sh::kStage + k * 2048, kPanel), kIdescO,
                               !first || k > 0);
            next_stage();
        }
        tc::mma_commit(&ctl->o_done);
        return true;
    };
    for (uint32_t n = 0;; ++n) {
        const uint32_t s = n % kItems;
        if (!wait(ctl->item_full + s, n / kItems & 1)) break;
        const int32_t stop = ctl->items[s].stop, tiles = ctl->items[s].hi - ctl->items[s].lo;
        tc::mbar_arrive(ctl->item_empty + s);
        if (stop) break;
        if (tiles <= 0) continue;
        bool ok = wait(&ctl->q_full, n_items & 1);
        for (int32_t i = 0; ok && i < tiles; ++i, ++tile) {
            // S of tile i; its buffer's last reader, the product with P of tile i - 2, is ahead in the queue
            for (int h = 0; ok && h < Sh::kHalves; ++h) {
                ok = wait(ctl->kv_full + stage, phase);
                if (!ok) break;
                tc::fence_after_sync();
#pragma unroll
                for (int k = 0; k < Sh::kCols / 16; ++k)
                    tc::mma_f16(tmem + (tile & 1) * kKeys,
                                tc::desc_k_sw128(q_smem + (h * Sh::kPanels + k / 4) * kPanel) + (k % 4) * 2,
                                tc::desc_k_sw128(ring + stage * Sh::kStage + k / 4 * kPanel) + (k % 4) * 2, kIdescS,
                                h > 0 || k > 0);
                next_stage();
            }
            if (!ok) break;
            tc::mma_commit(ctl->s_full + (tile & 1));
            if (i + 1 == tiles) tc::mma_commit(&ctl->q_empty);
            if (i > 0) ok = weights(tile - 1, i == 1);
        }
        if (!ok || !weights(tile - 1, tiles == 1)) break;
        ++n_items;
    }
    tc::mma_commit(&ctl->drain);
    drain_bar(&ctl->drain, 0);
}

// ---- the softmax warps ----------------------------------------------------------------------

template <int D, bool kHalf>
__device__ void softmax_rows(const AttentionLaunch &L, Control<D> *ctl, uint8_t *ring, uint32_t tmem, const Waiter &wait) {
    using Sh = Shape<D>;
    const PagedAttentionArgs &a = L.a;
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3;
    const int row = warp * 32 + lane;
    const int32_t u = row / L.group, g = row - u * L.group;
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;  // this warp's TMEM lanes
    const uint32_t t_o = tmem + kTmemO + lanes;
    const float c = L.c;
    uint32_t tile = 0, stages = 0;  // tiles and stages of the items before
    for (uint32_t n = 0;; ++n) {
        const uint32_t s = n % kItems;
        if (!wait.all(ctl->item_full + s, n / kItems & 1)) return;
        const Item it = ctl->items[s];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(ctl->item_empty + s);
        if (it.stop) return;
        const bool valid = u < it.n;
        const bool any_row = warp * 32 < it.n * L.group;
        const int32_t tiles = it.hi - it.lo;
        const int32_t key_hi = it.pos + u + 1;
        const int32_t key_lo = a.window > 0 && key_hi > a.window ? key_hi - a.window : 0;
        int32_t row_lo, row_hi;
        visible_rows(it, a.window, &row_lo, &row_hi);
        float m = -INFINITY, l = 0.f;
        for (int32_t i = 0; i < tiles; ++i, ++tile) {
            const int32_t k0 = (it.lo + i) * kKeys;
            if (!wait.all(ctl->s_full + (tile & 1), tile >> 1 & 1)) return;
            tc::fence_after_sync();
            if (any_row) {
                const uint32_t t_s = tmem + (tile & 1) * kKeys + lanes;
                uint32_t sb[kKeys];
                tc::tmem_ld128(t_s, sb);
                float x[kKeys];
#pragma unroll
                for (int j = 0; j < kKeys; ++j) x[j] = __uint_as_float(sb[j]);
                if (__any_sync(0xffffffffu, valid && (k0 + kKeys > key_hi || k0 < key_lo))) {
                    const int32_t hi = key_hi - k0, lo = key_lo - k0;
#pragma unroll
                    for (int j = 0; j < kKeys; ++j) x[j] = (j < hi && j >= lo) ? x[j] : -INFINITY;
                }
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int j = 0; j < kKeys; ++j) top[j & 3] = fmaxf(top[j & 3], x[j]);
                float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                mx = valid ? fmaxf(m, mx) : -INFINITY;
                const bool move = (m == -INFINITY && mx > -INFINITY) || (mx - m) * c > 8.f;
                if (__any_sync(0xffffffffu, move)) {
                    const float f = move ? ex2((m - mx) * c) : 1.f;  // 0 from the empty maximum
                    if (move) m = mx;
                    l *= f;
                    if (i > 0) {
                        if (!wait.all(&ctl->o_done, (tile - 1) & 1)) return;
                        tc::fence_after_sync();
#pragma unroll 1
                        for (int q = 0; q < D / 16; ++q) {
                            uint32_t o[16];
                            tc::tmem_ld16(t_o + q * 16, o);
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                            tc::tmem_st16(t_o + q * 16, o);
                        }
                    }
                }
                const float mc = m == -INFINITY ? 0.f : m * c;
                float sum[4] = {};
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t pw[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const float p0 = ex2(fmaf(x[q * 64 + 2 * j], c, -mc)), p1 = ex2(fmaf(x[q * 64 + 2 * j + 1], c, -mc));
                        sum[j & 1] += p0;
                        sum[2 + (j & 1)] += p1;
                        pw[j] = pack2<kHalf>(p0, p1);
                    }
                    tc::tmem_st32(t_s + q * 32, pw);
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            }
            // Value rows that no token sees may hold anything (0 x NaN): zero them before the product.
            if (k0 + kKeys > row_hi || k0 < row_lo) {
                const uint32_t before = stages + Sh::kHalves * static_cast<uint32_t>((i + 2 < tiles ? i + 2 : tiles) + i);
                const bool dead = k0 + row >= row_hi || k0 + row < row_lo;
                for (uint32_t v = before; v < before + Sh::kHalves; ++v) {
                    const uint32_t st = v % Sh::kStages;
                    if (!wait.all(ctl->kv_full + st, v / Sh::kStages & 1)) return;
                    if (dead) {
#pragma unroll
                        for (int p = 0; p < Sh::kPanels * 8; ++p)
                            *reinterpret_cast<uint4 *>(ring + st * Sh::kStage + (p >> 3) * kPanel + row * 128 + (p & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                    }
                }
                tc::fence_proxy_async_smem();
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(ctl->p_full + (tile & 1));
        }
        stages += 2 * Sh::kHalves * static_cast<uint32_t>(tiles > 0 ? tiles : 0);
        // O to memory: the result, or this split's part of it.
        // (the last two products in turn: S of the last tile only told that the third-last is done, and a parity
        // tells two phases apart)
        if (tiles > 0) {
            if (tiles > 1 && !wait.all(&ctl->o_done, tile & 1)) return;
            if (!wait.all(&ctl->o_done, (tile - 1) & 1)) return;
            tc::fence_after_sync();
        }
        if (any_row) {
            const int64_t head = static_cast<int64_t>(it.head) * L.group + g;
            const bool part = it.partial >= 0;
            const int64_t prow = (it.partial + static_cast<int64_t>(u) * it.splits) * a.h_q + head;
            const float f = part ? 1.f : l == 0.f ? 0.f : 1.f / l;
            uint16_t *out = a.o + ((static_cast<int64_t>(it.tok) + u) * a.h_q + head) * D;
            float *pout = L.ws.o + prow * D;
            if (part && valid) L.ws.ml[prow] = make_float2(m * c, l);
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
                uint32_t o[32];
                if (tiles > 0)
                    tc::tmem_ld32(t_o + q * 32, o);
                if (valid) {
                    if (part) {
#pragma unroll
                        for (int j = 0; j < 32; j += 4)
                            *reinterpret_cast<uint4 *>(pout + q * 32 + j) = make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                    } else {
                        uint32_t w[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float y0 = l == 0.f ? 0.f : __uint_as_float(o[2 * j]) * f;
                            const float y1 = l == 0.f ? 0.f : __uint_as_float(o[2 * j + 1]) * f;
                            w[j] = pack2<kHalf>(y0, y1);
                        }
#pragma unroll
                        for (int j = 0; j < 16; j += 4)
                            *reinterpret_cast<uint4 *>(out + q * 32 + j * 2) = make_uint4(w[j], w[j + 1], w[j + 2], w[j + 3]);
                    }
                }
            }
        }
        if (tiles > 0) {
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&ctl->o_free);
        }
    }
}

template <int D, bool kHalf>
__global__ void __launch_bounds__(kThreads, 1) attention_kernel(const __grid_constant__ AttentionLaunch L) {
    using Sh = Shape<D>;
    extern __shared__ uint8_t raw[];
    uint8_t *base = raw + ((1024u - (tc::smem_u32(raw) & 1023u)) & 1023u);
    uint8_t *ring = base + Sh::kQ;
    Control<D> *ctl = reinterpret_cast<Control<D> *>(ring + Sh::kStages * Sh::kStage);
    static_assert(sizeof(Control<D>) <= 1536, "control block");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        for (int i = 0; i < Sh::kStages; ++i) {
            tc::mbar_init(ctl->kv_full + i, 1);
            tc::mbar_init(ctl->kv_empty + i, 1);
        }
        tc::mbar_init(&ctl->q_full, 1);
        tc::mbar_init(&ctl->q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(ctl->s_full + i, 1);
            tc::mbar_init(ctl->p_full + i, 4);
        }
        tc::mbar_init(&ctl->o_done, 1);
        tc::mbar_init(&ctl->o_free, 4);
        for (int i = 0; i < kItems; ++i) {
            tc::mbar_init(ctl->item_full + i, 1);
            tc::mbar_init(ctl->item_empty + i, 6);  // load, mma, four softmax warps
        }
        tc::mbar_init(&ctl->drain, 1);
        ctl->fail = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 3) tc::tmem_alloc(&ctl->tmem, kTmemCols);
    tc::fence_proxy_async_smem();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = ctl->tmem;
    const Waiter wait = {&ctl->fail, L.a.dev_status};
    if (warp == 0) {
        load_tiles<D>(L, ctl, tc::smem_u32(base), tc::smem_u32(ring), wait);
    } else if (warp == 1) {
        if (lane == 0) issue_products<D, kHalf>(ctl, tc::smem_u32(base), tc::smem_u32(ring), tmem, wait);
    } else if (warp == 2) {
        schedule<D>(L, ctl, wait);
    } else if (warp == 3) {
        // Tokens of no request: zeros.
        const PagedAttentionArgs &a = L.a;
        const int32_t end = a.num_reqs > 0 ? a.cu_seqlens[a.num_reqs] : 0;
        const int64_t chunk = static_cast<int64_t>(a.h_q) * D / 8;
        for (int64_t i = (end > 0 ? end : 0) * chunk + blockIdx.x * 32 + lane; i < a.num_tokens * chunk; i += gridDim.x * 32)
            reinterpret_cast<uint4 *>(a.o)[i] = make_uint4(0, 0, 0, 0);
    } else {
        softmax_rows<D, kHalf>(L, ctl, ring, tmem, wait);
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 3) {
        tc::tmem_relinquish();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

// ---- joining the splits -----------------------------------------------------------------------

constexpr int kJoinWarps = 4;

// Last r in [0, n) with cu[r] <= t, by the warp: 32 probes a step.
__device__ __forceinline__ int32_t find_request(const int32_t *cu, int32_t n, int32_t t, int lane) {
    int32_t lo = 0, hi = n;  // cu[lo] <= t, and cu[hi] > t or hi == n
    while (hi - lo > 1) {
        const int32_t step = ceil_div(hi - lo, 32);
        const int64_t at = lo + static_cast<int64_t>(step) * lane;
        const bool le = at < hi && cu[at] <= t;
        const int last = 31 - __clz(__ballot_sync(0xffffffffu, le) | 1u);
        const int64_t top = lo + static_cast<int64_t>(step) * (last + 1);
        lo += step * last;
        if (top < hi) hi = static_cast<int32_t>(top);
    }
    return lo;
}

// o = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s over a row's splits, in
// split order: one warp per (token, query head), lane i holding every 32nd
// group of four columns.
template <int D, bool kHalf>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ AttentionLaunch L) {
    const PagedAttentionArgs &a = L.a;
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kJoinWarps + (threadIdx.x >> 5);
    const bool any = row < a.num_tokens * a.h_q;
    const int32_t t = any ? static_cast<int32_t>(row / a.h_q) : 0;
    const int32_t r = find_request(a.cu_seqlens, a.num_reqs, t, lane);
    const Request q = load_request(a, r, false);
    const Plan p = plan_request(q.kv, q.m, L.group, a.cache.h_kv, a.window);
    const int32_t u = t - q.first, u0 = u / p.tile_tokens * p.tile_tokens;
    const int32_t n = q.m - u0 < p.tile_tokens ? q.m - u0 : p.tile_tokens;
    int32_t lo, hi;
    key_tiles(q.kv, q.m, u0, n, a.window, &lo, &hi);
    const int32_t s0 = lo / p.split_tiles, s1 = hi > lo ? (hi - 1) / p.split_tiles + 1 : s0;
    // Every block waits for the attention kernel's end, also one with nothing to join: what follows this kernel in
    // the stream relies on both.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // One split wrote the row itself.
    if (!any || t < q.first || t >= q.first + q.m || s1 - s0 < 2) return;
    const int64_t base = L.ws.base[r];
    if (base < 0 || base + p.partials > L.partials) return;  // not written: the call timed out or its ranges overlap
    const int64_t first = (base + static_cast<int64_t>(u) * p.splits + (s0 - p.split0)) * a.h_q + row % a.h_q;
    float top = -INFINITY;
    for (int32_t s = lane; s < s1 - s0; s += 32) top = fmaxf(top, L.ws.ml[first + static_cast<int64_t>(s) * a.h_q].x);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    if (top == -INFINITY) top = 0.f;
    constexpr int kVec = D / 64;  // pairs of columns of a lane
    float acc[kVec][2] = {}, l = 0.f;
#pragma unroll 4
    for (int32_t s = 0; s < s1 - s0; ++s) {
        const int64_t at = first + static_cast<int64_t>(s) * a.h_q;
        const float2 ml = L.ws.ml[at];
        const float w = ex2(ml.x - top);
        l = fmaf(w, ml.y, l);
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
            const float2 o = *reinterpret_cast<const float2 *>(L.ws.o + at * D + v * 64 + lane * 2);
            acc[v][0] = fmaf(w, o.x, acc[v][0]);
            acc[v][1] = fmaf(w, o.y, acc[v][1]);
        }
    }
    const float f = 1.f / l;
#pragma unroll
    for (int v = 0; v < kVec; ++v)
        *reinterpret_cast<uint32_t *>(a.o + row * D + v * 64 + lane * 2) =
            pack2<kHalf>(l == 0.f ? 0.f : acc[v][0] * f, l == 0.f ? 0.f : acc[v][1] * f);
}

template <int D, bool kHalf>
cudaError_t launch_d(const AttentionLaunch &L, int64_t items, cudaStream_t stream) {
    static int set[kMaxDevices] = {};
    int dev = 0, sms = 0;
    if (!current_device(&dev, &sms)) return cudaErrorInvalidDevice;
    cudaError_t e;
    if (dev < 0 || dev >= kMaxDevices || !__atomic_load_n(&set[dev], __ATOMIC_ACQUIRE)) {
        e = cudaFuncSetAttribute(attention_kernel<D, kHalf>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(Shape<D>::kSmem));
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < kMaxDevices) __atomic_store_n(&set[dev], 1, __ATOMIC_RELEASE);
    }
    const unsigned blocks = static_cast<unsigned>(items < sms ? (items > 0 ? items : 1) : sms);
    attention_kernel<D, kHalf><<<blocks, kThreads, Shape<D>::kSmem, stream>>>(L);
    e = cudaGetLastError();
    if (e != cudaSuccess || !L.ws.o) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((L.a.num_tokens * L.a.h_q + kJoinWarps - 1) / kJoinWarps));
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = stream;
    // Its blocks may come up while the last items run; they wait for them before reading a partial.
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_kernel<D, kHalf>, L);
}

}  // namespace

size_t paged_attention_workspace(int32_t h_q, int32_t h_kv, int32_t d, int32_t num_reqs, int64_t num_tokens,
                                 int64_t max_kv_len) {
    const int64_t partials = partials_bound(h_q / h_kv, h_kv, num_reqs, num_tokens, max_kv_len);
    return partials > 0 ? workspace_at(nullptr, num_reqs, partials, h_q, d).bytes : 0;
}

cudaError_t launch_paged_attention(const PagedAttentionArgs &a, cudaStream_t stream) {
    const gdn_paged_cache_t &c = a.cache;
    AttentionLaunch L = {};
    L.a = a;
    L.group = a.h_q / c.h_kv;
    L.box_rows = kKeys;
    while (c.page_size % L.box_rows != 0) L.box_rows /= 2;
    // A scale of zero weighs all keys alike; the least one keeps masked scores at minus infinity (0 x inf is NaN).
    L.c = fmaxf(a.scale * 1.4426950408889634f, 1e-30f);
    const int64_t partials = L.partials = partials_bound(L.group, c.h_kv, a.num_reqs, a.num_tokens, a.max_kv_len);
    if (partials > 0) L.ws = workspace_at(a.workspace, a.num_reqs, partials, a.h_q, c.d);
    const cuuint64_t d = static_cast<cuuint64_t>(c.d);
    const cuuint64_t q_dims[3] = {d, static_cast<cuuint64_t>(a.h_q), static_cast<cuuint64_t>(a.num_tokens)};
    const cuuint64_t q_strides[2] = {d * 2, static_cast<cuuint64_t>(a.q_token_stride) * 2};
    const cuuint32_t tile_tokens = static_cast<cuuint32_t>(kRows / L.group);
    const cuuint32_t q_box[3] = {64, static_cast<uint32_t>(L.group), tile_tokens}, q_one[3] = {64, q_box[1], 1};
    const cuuint64_t dims[4] = {d, static_cast<cuuint64_t>(c.page_size), static_cast<cuuint64_t>(c.h_kv),
                              static_cast<cuuint64_t>(c.num_pages)};
    auto bytes = [](int64_t s) { return static_cast<cuuint64_t>(s) * 2; };
    const cuuint64_t k_strides[3] = {bytes(c.k_slot_stride), bytes(c.k_head_stride), bytes(c.k_page_stride)};
    const cuuint64_t v_strides[3] = {bytes(c.v_slot_stride), bytes(c.v_head_stride), bytes(c.v_page_stride)};
    const cuuint32_t box[4] = {64, static_cast<uint32_t>(L.box_rows), 1, 1};
    if (!encode_tiles(&L.tm_q, a.q, c.dtype, 3, q_dims, q_strides, q_box) ||
        !encode_tiles(&L.tm_q_one, a.q, c.dtype, 3, q_dims, q_strides, q_one) ||
        !encode_tiles(&L.tm_k, c.k, c.dtype, 4, dims, k_strides, box) ||
        !encode_tiles(&L.tm_v, c.v, c.dtype, 4, dims, v_strides, box))
        return cudaErrorNotSupported;
    // Bound of the item count: row tiles times heads times splits.
    const int64_t tiles = a.num_tokens / tile_tokens + a.num_reqs;
    const int64_t items = (tiles < a.num_tokens ? tiles : a.num_tokens) * c.h_kv * (partials > 0 ? kMaxSplits + 1 : 1);
    const bool half = c.dtype == GDN_FP16;
    switch (c.d) {
        case 64: return half ? launch_d<64, true>(L, items, stream) : launch_d<64, false>(L, items, stream);
        case 128: return half ? launch_d<128, true>(L, items, stream) : launch_d<128, false>(L, items, stream);
        default: return half ? launch_d<256, true>(L, items, stream) : launch_d<256, false>(L, items, stream);
    }
}

}  // namespace gdn
