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
// persistent grid (one block per SM) takes the items from a counter, the
// requests from the last to the first and each one's longest row items first;
// lengths are read on the device, so a captured call replays for others.
//
// One block, twelve warps:
//   load (2)   TMA boxes of K and V (one per page piece) into a ring of stages
//              128 keys x up to 128 columns, running ahead over item borders
//   mma        S = Q K^T into one of two TMEM buffers, O += P V with P from
//              TMEM; the scores of one unit are computed while the weights of
//              the one before are (struct Ring)
//   sched      walks the requests, cutting them into items
//              (d = 64: one load warp, and one MMA warp for each of the products)
//   softmax (2 x 4)  one row per thread: S from TMEM, masks, maximum, exp2, P
//              back to TMEM over S; at the end O from TMEM to memory.  With
//              d <= 128 each warpgroup has its own O; with d = 256 there is
//              one, and the second warpgroup writes it while the first is on
//              with the next item.
//
// The running maximum only moves when a score passes it by more than 8 (in
// powers of two): weights are then at most 2^8 (2^15 in fp16, which holds them
// times 2^7), and O is rarely touched.  The rule is per row, so a row's bits do
// not depend on its neighbours.
//
// What bounds it: HBM for single tokens over long contexts (8 rows of 100 to
// 131 thousand keys, 32/8 heads of 128: 3.68 GB in 545 us, 0.99 of the copy
// peak; 256 rows of up to 4095 keys, 16/2 of 256: 6.3 TB/s); the tensor pipe
// for long chunks (2048 tokens twice at 32 thousand keys, 16/2 of 256: 1450 to
// 1560 us, 1.44 to 1.55 PF/s; a prompt of 8192 tokens, 32/8 of 128: 385 to 423
// us, 1.30 to 1.43 PF/s); the softmax warps with d = 64; the fill and drain of
// the pipe per item for short prompts (8 of 116 to 2000 tokens: 95 us, the
// tensor pipe 49 % busy); a chain of ~10 us (lengths, page ids, first tile,
// softmax, result, part of it instruction fetch) for a few short rows.  (Ranges:
// calls apart and back to back, and between GPUs, by the clock they keep.)
//
// Every wait is bounded (one for a whole item's end by the time that no tile
// is asked for in): one that runs out sets GDN_DEV_TIMEOUT and a flag that
// ends all the others; before the block leaves, its MMAs and copies in
// flight are waited for and TMEM is freed.
//
// Trees (kTree; tree_attention.cu).  A request's new tokens are the nodes of a
// tree in an order that puts parents first, so what a node sees is what a token
// in its place would see, less the nodes before it that are not above it: one
// 64-bit word per token, looked at only in the last one or two key tiles, by the
// softmax threads whose row it is; scheduling, splits and the join are the same.
// 8 trees of 25 to 32 nodes over 60 to 100 thousand keys, 32/8 heads of 128: 2.87
// GB in 442 to 454 us, 0.93 to 0.95 of the copy peak; 128 of up to 12 over 2000 to 8000,
// 16/16 of 64: 2.55 GB in 418 to 423, 0.90; 64 of 16 to 64 over 500 to 8000, 16/2
// of 256: 195 GF in 218 to 230 us, as gdn_paged_attention of the same lengths
// (215): row tiles of 16 tokens a seventh empty, parts that a request alone would
// need and the join of their 97 MB (the kernel itself 188 us, the tensor pipe 63 %
// busy); 64 equal ones of 64 nodes over 8000 keys 1.19 PF/s.  One tree of 7 over
// 1058 keys: 20 us, the chain above.  A tree's part of LeftOut is a structure of
// its own: in the causal kernels' it cost a prompt of 8192 tokens 1.3 %.
#pragma once

#include "paged.cuh"
#include "tc_ptx.cuh"

#include <cuda.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>
#include <limits.h>
#include <stddef.h>
#include <type_traits>

#ifndef GDN_WAIT_CYCLES
#define GDN_WAIT_CYCLES 2000000000LL  // about a second; under 2^32
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

constexpr int kRows = 128;     // query rows of a tile (TMEM lanes)
constexpr int kKeys = 128;     // keys of a tile
constexpr int kPanel = 16384;  // 128 rows of 64 16-bit elements
constexpr int kItems = 4;      // items between the scheduler and the other warps
// Items are taken ahead of their turn while those that have not begun hold no more keys and values than this: what a
// block holds no other can take at the end.  (512 KB: mixed step with a window 60 -> 64 us, eight prompts 96 -> 101;
// 64 KB: 58 and 97.)
constexpr int kAheadBytes = 256 * 1024;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 256;  // O after the two S buffers

// Splits.  A request alone should fill kSplitUnits SMs where its row tiles are
// full, half of them where they are not: then memory is the bound, and 76 SMs
// draw all of it.  The constant stands in for the SM count so that results do
// not depend on the device.
constexpr int kSplitUnits = 152;
constexpr int kMaxSplits = 64;
constexpr int kMinSplitTiles = 2;
constexpr int kMaxSplitTiles = 16;  // of few rows, while kMaxSplits allow: long items balance badly over the SMs
// The least key tiles of a split of `tiles` by an item of `rows` query rows.  A
// part's cost beside its keys is its partial result, in proportion to its rows:
// a full tile's is that of two key tiles.  And each part costs the joining
// kernel as the others do, so their number grows with the root of the keys.
__host__ __device__ __forceinline__ int32_t least_split_tiles(int32_t tiles, int32_t rows) {
    int32_t n = rows / 8 > kMinSplitTiles ? rows / 8 : kMinSplitTiles;
#pragma unroll 1
    while (n * n * 2 < tiles) ++n;
    return n;
}

// Row tiles that a block works on at once: two where two accumulators fit TMEM.
__host__ __device__ constexpr int streams_of(int d) { return d <= 128 ? 2 : 1; }

struct Plan {
    int32_t row_items;    // pieces of the new tokens
    int32_t item_tokens;  // tokens of one
    int32_t first_tile;   // that any of its tokens sees: where its splits start
    int32_t split_tiles;  // key tiles of a split
    int32_t splits;
    int64_t items;
    int64_t partials;  // (token, split) pairs that may leave partial results
};

__host__ __device__ __forceinline__ int32_t ceil_div(int32_t a, int32_t b) { return (a + b - 1) / b; }

// ceil(a / b) for 0 <= a < 2^23, b > 0: a reciprocal and a correction, half the time of an integer division.
__device__ __forceinline__ int32_t ceil_quotient(int32_t a, int32_t b) {
    int32_t q = __float2int_rz(__fdividef(static_cast<float>(a), static_cast<float>(b)));  // off by one at most
    if (q * b < a) ++q;
    if (q * b < a) ++q;
    if ((q - 1) * b >= a) --q;
    return q;
}

// Key tiles [lo, hi) that tokens [u, u + n) of a request see together.
__device__ __forceinline__ void key_tiles(int32_t kv, int32_t m, int32_t u, int32_t n, int32_t window, int32_t *lo,
                                          int32_t *hi) {
    const int32_t first = kv - m + u, last = first + n;  // positions [first, last)
    *hi = last > 0 ? ceil_div(last, kKeys) : 0;
    *lo = window > 0 && first >= window ? (first - window + 1) / kKeys : 0;
    if (*lo > *hi) *lo = *hi;
}

// Splits that let a request of few rows fill half of kSplitUnits.
int32_t few_splits_of(int32_t h_kv) { return h_kv < kSplitUnits / 2 ? kSplitUnits / 2 / h_kv : 1; }

// How a request of m new tokens and kv keys is cut; depends on nothing else of the batch.
__device__ __forceinline__ Plan plan_request(int32_t kv, int32_t m, int32_t group, int32_t tile_tokens, int32_t few_splits,
                                             int32_t d, int32_t h_kv, int32_t window) {
    Plan p;
    p.item_tokens = tile_tokens * streams_of(d);
    p.row_items = m <= p.item_tokens ? (m > 0 ? 1 : 0) : ceil_div(m, p.item_tokens);  // (divisions are most of the time here)
    int32_t lo, hi;
    key_tiles(kv, m, 0, m, window, &lo, &hi);
    p.first_tile = lo;
    p.split_tiles = INT_MAX;
    p.splits = 1;
    const int64_t units = static_cast<int64_t>(p.row_items) * h_kv;
    const int32_t rows = (m < p.item_tokens ? m : p.item_tokens) * group;
    const bool few = rows < kRows / 2;
    if (m > 0 && (few || units * 2 <= kSplitUnits)) {
        int32_t want = few ? few_splits : kSplitUnits / static_cast<int32_t>(units);
        if (want > kMaxSplits) want = kMaxSplits;
        const int32_t even = ceil_quotient(hi - lo, want), least = least_split_tiles(hi - lo, rows);
        p.split_tiles = even > least ? even : least;
        if (few) {
            const int32_t most = ceil_div(hi - lo, kMaxSplits) > kMaxSplitTiles ? ceil_div(hi - lo, kMaxSplits) : kMaxSplitTiles;
            if (p.split_tiles > most) p.split_tiles = most;
        }
        p.splits = hi > lo ? ceil_quotient(hi - lo, p.split_tiles) : 1;
    }
    p.items = units * p.splits;
    p.partials = p.splits > 1 ? static_cast<int64_t>(m) * p.splits : 0;
    return p;
}

// Bound of a request's splits: no more than kMaxSplits or than the longest
// context's.  least_split_tiles(s) >= sqrt(s / 2), so s tiles make at most
// sqrt(2 s) splits, or as many as the cap makes of them.
int64_t splits_bound(int64_t max_kv_len) {
    const int64_t tiles = (max_kv_len + kKeys - 1) / kKeys;
    if (tiles <= kMinSplitTiles) return 1;
    int64_t splits = (tiles + kMaxSplitTiles - 1) / kMaxSplitTiles;
    if (splits > kMaxSplits) return kMaxSplits;
    while (splits * splits < 2 * tiles && splits < kMaxSplits) ++splits;
    return splits;
}

// Bound of `partials` over the requests of a call.
int64_t partials_bound(int32_t group, int32_t d, int32_t h_kv, int32_t num_reqs, int64_t num_tokens, int64_t max_kv_len) {
    const int64_t splits = splits_bound(max_kv_len);
    if (splits == 1 || num_tokens == 0 || num_reqs == 0) return 0;
    // With full tiles m tokens make at least m / item_tokens row items and at most kSplitUnits / (h_kv * row items)
    // splits; fewer tokens than half a tile's make at most kMaxSplits.
    const int64_t full = static_cast<int64_t>(kRows / group * streams_of(d)) * ceil_div(kSplitUnits, h_kv);
    const int64_t few = static_cast<int64_t>(kRows / 2 / group + 1) * kMaxSplits;
    const int64_t by_request = num_reqs * (full > few ? full : few), by_token = num_tokens * splits;
    return by_token < by_request ? by_token : by_request;
}

// Bound of the items of a call.
int64_t items_bound(int32_t group, int32_t d, int32_t h_kv, int32_t num_reqs, int64_t num_tokens, int64_t max_kv_len) {
    const int64_t rows = num_tokens / (kRows / group * streams_of(d)) + num_reqs;
    return (rows < num_tokens ? rows : num_tokens) * h_kv * splits_bound(max_kv_len);
}

// What the joining kernel needs of a row (token and query head) of a request
// that was split: its place in o, its first partial and how many there are (0:
// the row is in o already).
struct JoinRow {
    int32_t out, parts;
    int64_t first;
};

// Workspace: the item counter (zeroed by each call), the number of rows of
// split requests and those rows, then (m, l) and O of the partials.
struct Workspace {
    unsigned long long *counter;  // null: items are dealt round robin
    int64_t *num_rows;
    JoinRow *rows;
    float2 *ml;
    float *o;  // null: no request of this call can be split
    int64_t partials, max_rows;
    size_t bytes;
};
Workspace workspace_at(void *ws, int32_t h_q, int32_t h_kv, int32_t d, int32_t num_reqs, int64_t num_tokens,
                       int64_t max_kv_len) {
    auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
    const int32_t group = h_q / h_kv;
    Workspace w = {};
    char *p = static_cast<char *>(ws);
    w.partials = partials_bound(group, d, h_kv, num_reqs, num_tokens, max_kv_len);
    // With few items per block there is little to balance, less than the counter's reset costs.
    if (items_bound(group, d, h_kv, num_reqs, num_tokens, max_kv_len) > 3 * kSplitUnits) {
        w.counter = reinterpret_cast<unsigned long long *>(p);
        w.bytes = 256;
    }
    if (w.partials > 0) {
        const size_t rows = static_cast<size_t>(w.partials) * h_q;
        w.num_rows = reinterpret_cast<int64_t *>(p + w.bytes);
        w.rows = reinterpret_cast<JoinRow *>(p + w.bytes + 256);
        w.max_rows = num_tokens * h_q;
        w.bytes += up(256 + static_cast<size_t>(w.max_rows) * sizeof(JoinRow));
        w.ml = reinterpret_cast<float2 *>(p + w.bytes);
        w.bytes += up(rows * sizeof(float2));
        w.o = reinterpret_cast<float *>(p + w.bytes);
        w.bytes += rows * d * sizeof(float);
    }
    return w;
}

struct AttentionLaunch {
    CUtensorMap tm_q;      // [T][h_q][d]: boxes of a full tile's tokens x group x 64
    CUtensorMap tm_q_one;  // the same, one token
    CUtensorMap tm_k, tm_v;  // [page][head][row][d]: boxes of box_rows x 64
    PagedAttentionArgs a;
    Workspace ws;
    int32_t group, tile_tokens, few_splits, box_rows;
    bool o_32;  // o starts at a 32-byte boundary, and so do its rows
    float c;    // scale * log2(e)
};

struct Item {
    int32_t stop;
    int32_t req, head;  // request, K/V head
    int32_t tok, n;     // first token (row of q) and tokens
    int32_t pos;        // position of the first token
    int32_t lo, hi;     // key tiles
    // Of a request that is split (rows >= 0): its row items' places among the rows to join (first token, head 0); the
    // first token's first partial, partials from one token to the next, parts of the row item, which one this is.
    int64_t rows, partial;
    int32_t splits, parts, part;
    int32_t ctx;  // with kTree: keys before the request's new tokens (negative: as many of those have none)
};

template <int D>
struct Shape {
    static constexpr int kStreams = streams_of(D);
    // A tile's maximum is sought beside its exponentials (softmax_rows) where a stream's softmax and products follow one
    // another: with d = 128 chunks of 1000 and 2000 tokens on 32 thousand keys take 822 -> 798 and 832 -> 807 us, a
    // prompt of 8192 396 -> 385, sixteen prompts of 100 to 900 80 -> 81.  With d = 64 and 256 it costs 5 and 2 %.
    static constexpr bool kBeside = D == 128;
    static constexpr bool kEarly = D == 64;  // scores run ahead of the weights (struct Ring)
    static constexpr int kThreads = 384;
    static constexpr int kCols = D < 128 ? D : 128;  // columns of a stage
    static constexpr int kHalves = D / kCols;        // stages of a K or V tile
    static constexpr int kPanels = kCols / 64;
    static constexpr uint32_t kStage = kPanels * kPanel;
    static constexpr uint32_t kQTile = D / 64 * kPanel;
    static constexpr uint32_t kQ = kStreams * kQTile;
    // Q of an item while the next one's loads: with two streams each single tile has its own half, else few rows
    // (kSmallRows) lie at row 0 or 64 of the tile (a product reads the 128 rows from there; the rest is not used).
    static constexpr int kSmallRows = 64;
    static constexpr uint32_t kQSlot = kStreams == 2 ? kQTile : kSmallRows * 128;
    // As many stages as 227 KB hold beside Q and the control block.
    static constexpr int kControl = 2048;
    static constexpr int kStages = (227 * 1024 - 1024 - kControl - static_cast<int>(kQ)) / static_cast<int>(kStage);
    static constexpr uint32_t kSide = kStages / 2;  // of K, and of V, where they have a ring each
    // P of unit g in TMEM: over its S, or behind O.
    static __device__ __forceinline__ uint32_t p_at(uint32_t g) {
        return kEarly ? kTmemO + kStreams * D + (g & 1) * (kKeys / 2) : (g & 1) * kKeys;
    }
    static constexpr uint32_t kSmem = 1024 + kQ + kStages * kStage + kControl;
};

template <int D>
struct Control {
    uint64_t kv_full[Shape<D>::kStages], kv_empty[Shape<D>::kStages];
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2], s_free[2], p_full[2];
    uint64_t o_done[2], o_free[2], ml_full[2], ml_empty, item_done;
    uint64_t item_full[kItems], item_empty[kItems];
    uint64_t drain[2];
    Item items[kItems];
    uint32_t bad[kItems];  // per item slot: number of the last item (from 1) with values left out of its products
    uint32_t tmem;
    int fail;
    int32_t tile;  // the last that the load warp has begun, of its item
    // (m, l) of one warpgroup for the other; row r is only touched by the two threads of row r, in turn.
    float2 ml[kRows];
};

// Units.  The work of an item is a sequence of units, each one S = Q K^T and
// one O += P V over a tile of keys; units of all items are numbered on, and
// unit g uses S/P buffer g % 2.  With one stream (d = 256) unit j of an item
// is key tile j and there is one O.  With two streams buffer, O and softmax
// warpgroup go together (w = g % 2): an item of two row tiles ("dual") takes
// each key tile twice, once per row tile; an item of one row tile gives its
// even key tiles to one warpgroup and its odd ones to the other, each with its
// own m, l and O, joined at the end.  The tensor core gets
// QK(g), PV(g - 1), QK(g + 1), ..., so the scores of one unit are computed
// while the weights of the one before are.
//
// The ring holds K and V tiles in the order of their first use.  V of the last
// tile of an item of one row tile is used after the next item's first K and
// lies behind it.  `first` is the item's first stage, `late` whether such a V
// of the item before lies behind its first K.
//
// With d = 64 (kEarly) TMEM has room for P beside S, and scores run ahead of
// the weights: S of unit g + 2 is written as soon as that of g is in registers,
// so a warpgroup that is done with a unit finds the next one's scores there
// instead of waiting for two products in turn.  K and V then have their own
// rings, and `first` counts tiles.  (Five chunks of 700 tokens on 16 thousand
// keys, 16/4 of 64: 382 -> 331 us; 8192 tokens, 16/16: 216 -> 190.)
template <int D>
struct Ring {
    using Sh = Shape<D>;
    struct Place {
        uint32_t stage, parity;
    };
    uint32_t first = 0, late = 0;
    // Half h of the K or V of the item's key tile t.
    __device__ __forceinline__ Place at(bool is_k, uint32_t t, bool dual, uint32_t h) const {
        if (Sh::kEarly) {
            const uint32_t n = first + t;
            return {n % Sh::kSide + (is_k ? 0 : Sh::kSide), n / Sh::kSide & 1};
        }
        const uint32_t past = late + 2 * t;
        const uint32_t tile = !is_k ? past + (dual ? 1 : 2) : t == 0 ? 0 : past - (dual ? 0 : 1);
        const uint32_t n = first + Sh::kHalves * tile + h;
        return {n % Sh::kStages, n / Sh::kStages & 1};
    }
    __device__ __forceinline__ void next(uint32_t tiles, bool dual) {
        if (Sh::kEarly) {
            first += tiles;
            return;
        }
        first += Sh::kHalves * (late + 2 * tiles - (dual ? 0 : 1));
        late = dual ? 0 : 1;
    }
};

constexpr uint32_t kWaitCycles = GDN_WAIT_CYCLES;
constexpr long long kDrainCycles = 2000000000LL;

// Bounded wait of a whole warp for the phase of `bar` with the given parity:
// true for all lanes or for none.  Gives up as soon as any thread has flagged a
// failure, and flags one when it runs out (the block reports it at its end).
struct Waiter {
    volatile int *fail;
    volatile const int32_t *tile;  // moves on while the block works on an item of many tiles
    // (try_wait suspends the thread for some microseconds by itself: a shorter limit asks without that)
    static __device__ __forceinline__ bool poll(uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu,
                          kWaitCycles < 10000 ? tc::mbar_test_wait(bar, parity) : tc::mbar_try_wait(bar, parity));
    }
    __device__ __forceinline__ bool all(uint32_t bar, uint32_t parity) const {  // bar: shared-memory address
        if (poll(bar, parity)) return true;
        const uint32_t start = static_cast<uint32_t>(clock());
#pragma unroll 1
        do {
            if (__any_sync(0xffffffffu, *fail || static_cast<uint32_t>(clock()) - start > kWaitCycles)) {
                *fail = 1;
                return false;
            }
        } while (!poll(bar, parity));
        return true;
    }
    __device__ __forceinline__ bool all(uint64_t *bar, uint32_t parity) const { return all(tc::smem_u32(bar), parity); }
    // For a whole item's end, which may be any time away: the limit begins anew while tiles go by.
    __device__ __forceinline__ bool item(uint64_t *bar, uint32_t parity) const {
        const uint32_t at = tc::smem_u32(bar);
        if (poll(at, parity)) return true;
        uint32_t start = static_cast<uint32_t>(clock());
        int32_t seen = *tile;
#pragma unroll 1
        do {
            const uint32_t now = static_cast<uint32_t>(clock());
            const int32_t last = *tile;
            if (last != seen) start = now;
            seen = last;
            if (__any_sync(0xffffffffu, *fail || now - start > kWaitCycles)) {
                *fail = 1;
                return false;
            }
        } while (!poll(at, parity));
        return true;
    }
};
__device__ __forceinline__ void drain_bar(uint64_t *bar, uint32_t parity) {
    const long long start = clock64();
#pragma unroll 1
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
// Lengths of request r; m = 0 (nothing to do) where its token range is bad, kv = 0 (no keys) where its length is, or its
// tree has more nodes than a word has bits.
template <bool kTree>
__device__ __forceinline__ Request load_request(const PagedAttentionArgs &a, int64_t r, bool tell) {
    Request q = {0, 0, 0};
    if (r >= 0 && r < a.num_reqs) {
        const int32_t b = a.cu_seqlens[r], e = a.cu_seqlens[r + 1], kv = a.kv_lens[r];
        const bool range = b >= 0 && b <= e && e <= a.num_tokens, len = kv >= 0 && kv <= a.max_kv_len && (!kTree || e - b <= kTreeNodes);
        if (range) q = {b, e - b, len ? kv : 0};
        if (tell && (!range || !len)) report(a.dev_status, GDN_DEV_BAD_LENGTH);
    }
    return q;
}

// Tokens that see no key: zeros, by the scheduler itself.
template <int D>
__device__ __forceinline__ void zero_rows(const AttentionLaunch &L, const Item &it, int lane) {
    const PagedAttentionArgs &a = L.a;
    const int32_t pieces = L.group * (D / 8);
#pragma unroll 1
    for (int32_t i = lane; i < it.n * pieces; i += 32) {
        const int32_t u = i / pieces, k = i - u * pieces;
        uint16_t *out = a.o + ((static_cast<int64_t>(it.tok) + u) * a.h_q + it.head * L.group) * D;
        reinterpret_cast<uint4 *>(out)[k] = make_uint4(0, 0, 0, 0);
        if (it.rows >= 0 && k < L.group)
            L.ws.rows[it.rows + static_cast<int64_t>(u) * a.h_q + it.head * L.group + k] = {0, 0, 0};
    }
}

template <int D, bool kTree>
__device__ void schedule(const AttentionLaunch &L, Control<D> *ctl, const Waiter &wait, const Request &first_read) {
    const PagedAttentionArgs &a = L.a;
    const int lane = threadIdx.x & 31;
    uint32_t n = 0;
    constexpr int32_t kAheadTiles = kAheadBytes / (kKeys * D * 4);
    uint32_t begun = 0;  // items known to have begun
    int32_t ahead = 0;   // key tiles of those that are not
    int64_t next = -1;
    bool counted = false;
    // The next item's number, taken when there is room for the item.
    auto advance = [&]() {
        if (!wait.item(ctl->item_empty + n % kItems, (n / kItems & 1) ^ 1)) return false;
        auto pass = [&]() {  // the oldest item taken has begun
            ahead -= __reduce_max_sync(0xffffffffu, lane == 0 ? ctl->items[begun % kItems].hi - ctl->items[begun % kItems].lo : 0);
            ++begun;
        };
        if (n >= kItems && begun == n - kItems) pass();
#pragma unroll 1
        while (ahead > kAheadTiles) {
            if (!wait.item(ctl->item_empty + begun % kItems, begun / kItems & 1)) return false;
            pass();
        }
        if (next < 0) {
            next = blockIdx.x;
        } else if (!L.ws.counter) {
            next += gridDim.x;
        } else {
            if (!counted) asm volatile("griddepcontrol.wait;" ::: "memory");  // the counter's reset
            counted = true;
            unsigned long long x = 0;
            if (lane == 0) x = atomicAdd(L.ws.counter, 1ull);
            next = gridDim.x + static_cast<int64_t>(__shfl_sync(0xffffffffu, x, 0));
        }
        return true;
    };
    auto publish = [&](const Item &it) {
        const uint32_t s = n % kItems;
        if (lane == 0) {
            ctl->items[s] = it;
            tc::mbar_arrive(ctl->item_full + s);
        }
        ++n;
        ahead += it.hi - it.lo;
        __syncwarp();
    };
    if (!advance()) return;
    int64_t items0 = 0, partials0 = 0, rows0 = 0;
    // From the last request to the first: long prompts stand behind the decode rows and should start first.
#pragma unroll 1
    for (int64_t base = 0; base < a.num_reqs; base += 32) {
        const int64_t r = a.num_reqs - 1 - base - lane;
        const Request q = base == 0 ? first_read : load_request<kTree>(a, r, blockIdx.x == 0);
        const Plan p = plan_request(q.kv, q.m, L.group, L.tile_tokens, L.few_splits, D, a.cache.h_kv, a.window);
        const int64_t split_rows = p.splits > 1 ? static_cast<int64_t>(q.m) * a.h_q : 0;
        int64_t items = p.items, partials = p.partials, rows = split_rows;
        if (__all_sync(0xffffffffu, (items | partials | rows) < (1 << 26))) {  // their sums fit 32 bits
            int32_t i32 = static_cast<int32_t>(items), p32 = static_cast<int32_t>(partials), r32 = static_cast<int32_t>(rows);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t x = __shfl_up_sync(0xffffffffu, i32, o), y = __shfl_up_sync(0xffffffffu, p32, o);
                const int32_t z = __shfl_up_sync(0xffffffffu, r32, o);
                if (lane >= o) {
                    i32 += x;
                    p32 += y;
                    r32 += z;
                }
            }
            items = i32;
            partials = p32;
            rows = r32;
        } else
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, items, o), y = __shfl_up_sync(0xffffffffu, partials, o);
            const int64_t z = __shfl_up_sync(0xffffffffu, rows, o);
            if (lane >= o) {
                items += x;
                partials += y;
                rows += z;
            }
        }
        if (blockIdx.x == 0 && L.ws.o && r == 0) *L.ws.num_rows = rows0 + rows;
        const int64_t group_items = __shfl_sync(0xffffffffu, items, 31);
#pragma unroll 1
        while (next < items0 + group_items) {
            const int src = __ffs(__ballot_sync(0xffffffffu, items0 + items > next)) - 1;
            // Items of a request: the last row item first (it sees the most keys), all its splits and heads.
            // (at most h_kv times the row items, or few splits of few: 32 bits)
            const uint32_t local = static_cast<uint32_t>(next - items0 - __shfl_sync(0xffffffffu, items - p.items, src));
            const int32_t m = __shfl_sync(0xffffffffu, q.m, src), kv = __shfl_sync(0xffffffffu, q.kv, src);
            const int32_t row_items = __shfl_sync(0xffffffffu, p.row_items, src);
            const int32_t split_tiles = __shfl_sync(0xffffffffu, p.split_tiles, src);
            const int32_t first_tile = __shfl_sync(0xffffffffu, p.first_tile, src);
            const int32_t splits = __shfl_sync(0xffffffffu, p.splits, src);
            const int32_t first = __shfl_sync(0xffffffffu, q.first, src);
            const int64_t pbase = partials0 + __shfl_sync(0xffffffffu, partials - p.partials, src);
            const uint32_t heads = static_cast<uint32_t>(a.cache.h_kv), per_piece = heads * static_cast<uint32_t>(splits);
            const uint32_t nth = row_items == 1 ? 0 : local / per_piece, rest = local - nth * per_piece;
            const int32_t piece = row_items - 1 - static_cast<int32_t>(nth);
            const int32_t split = static_cast<int32_t>(splits == 1 ? 0 : rest / heads);
            const int64_t rbase = rows0 + __shfl_sync(0xffffffffu, rows - split_rows, src);
            Item it;
            it.stop = 0;
            it.req = static_cast<int32_t>(a.num_reqs - 1 - base) - src;
            it.head = static_cast<int32_t>(rest - static_cast<uint32_t>(split) * heads);
            const int32_t u = piece * p.item_tokens;
            it.n = m - u < p.item_tokens ? m - u : p.item_tokens;
            it.tok = first + u;
            it.pos = kv - m + u;
            if (kTree) it.ctx = kv - m;
            int32_t lo, hi;
            key_tiles(kv, m, u, it.n, a.window, &lo, &hi);
            int32_t split_lo = 0, split_hi = splits - 1;
            if (row_items > 1) {
                split_lo = splits == 1 ? 0 : (lo - first_tile) / split_tiles;
                split_hi = splits == 1 || hi == lo ? split_lo : (hi - 1 - first_tile) / split_tiles;
            }
            const int64_t s_lo = first_tile + static_cast<int64_t>(split) * split_tiles, s_hi = s_lo + split_tiles;
            it.lo = s_lo > lo ? static_cast<int32_t>(s_lo) : lo;
            it.hi = s_hi < hi ? static_cast<int32_t>(s_hi) : hi;
            it.parts = split_hi - split_lo + 1;
            it.part = split - split_lo;
            it.splits = splits;
            it.partial = pbase + static_cast<int64_t>(u) * splits + split_lo;
            it.rows = splits > 1 ? rbase + static_cast<int64_t>(u) * a.h_q : -1;
            // A split past what the tokens see has nothing to do; tokens that see nothing are written by the first.
            bool run = it.lo < it.hi || (lo == hi && split == 0);
            // Token ranges that overlap can ask for more partials and rows than there are tokens for.
            if (run && splits > 1 &&
                (pbase + static_cast<int64_t>(m) * splits > L.ws.partials || rbase + static_cast<int64_t>(m) * a.h_q > L.ws.max_rows)) {
                if (lane == 0) report(a.dev_status, GDN_DEV_BAD_LENGTH);
                run = false;
            }
            if (run && it.lo < it.hi)
                publish(it);
            else if (run)
                zero_rows<D>(L, it, lane);
            if (!advance()) return;
        }
        items0 += group_items;
        partials0 += __shfl_sync(0xffffffffu, partials, 31);
        rows0 += __shfl_sync(0xffffffffu, rows, 31);
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

// ---- the load warps -----------------------------------------------------------------

// Page and row of this lane's box of a key tile, tile after tile (a step
// without divisions).  A box that no token sees, or whose page id is bad, is
// loaded from past the last page: TMA fills zeros.
struct Boxes {
    const PagedAttentionArgs &a;
    int32_t box_rows, box;        // this lane's box of a tile
    int32_t step_idx, step_row;   // of kKeys keys: whole pages, rows beyond
    int32_t key, idx, row;        // of the box whose id is fetched next: first key, place in the table, row in the page
    int32_t row_lo, row_hi, end;  // keys that some token sees, end of the item's
    const int32_t *table;
    int32_t next_id, next_row;
    bool next_seen;
    __device__ __forceinline__ void start(const Item &it) {
        visible_rows(it, a.window, &row_lo, &row_hi);
        end = it.hi * kKeys;
        if (row_hi < end) end = row_hi;
        table = a.block_table + it.req * a.table_stride;
        key = it.lo * kKeys + box * box_rows;
        idx = key / a.cache.page_size;
        row = key - idx * a.cache.page_size;
        fetch();
    }
    // The table's entry, asked for one tile ahead of its use.
    __device__ __forceinline__ void fetch() {
        next_seen = key < end && key + box_rows > row_lo;
        next_id = next_seen ? table[idx] : 0;
        next_row = row;
        key += kKeys;
        idx += step_idx;
        row += step_row;
        if (row >= a.cache.page_size) {
            row -= a.cache.page_size;
            ++idx;
        }
    }
    __device__ __forceinline__ void place(int32_t *page, int32_t *at) {
        *page = static_cast<int32_t>(a.cache.num_pages);
        *at = 0;
        if (next_seen) {
            if (next_id >= 0 && next_id < *page) {
                *page = next_id;
                *at = next_row;
            } else {
                report(a.dev_status, GDN_DEV_BAD_SLOT);
            }
        }
        fetch();
    }
};

// Warp 0 loads Q and the K tiles, warp 3 the V tiles: a box takes a warp 65 to
// 100 cycles to issue, one lane's after another's, which pages of 16 rows (16
// boxes per 32 KB) would make the bound of a single load warp.  (One body for
// both: the block's code is large enough for instruction fetch to matter.)
// With d = 64 there are only 16 KB a tile, and warp 0 loads K and V, a box of
// each from the same coordinates; warp 3 issues products.
template <int D>
__device__ void load_tiles(const AttentionLaunch &L, Control<D> *ctl, uint32_t q_smem, uint32_t ring, const Waiter &wait,
                           bool is_k) {
    using Sh = Shape<D>;
    const PagedAttentionArgs &a = L.a;
    const int lane = threadIdx.x & 31;
    const int boxes = kKeys / L.box_rows;
    const CUtensorMap *map = is_k ? &L.tm_k : &L.tm_v;
    Boxes where = {a, L.box_rows, lane % boxes, kKeys / a.cache.page_size, kKeys % a.cache.page_size};
    Ring<D> pos;
    uint32_t n_items = 0;
    bool ok = true, wide_before = false;
    int32_t filled = -1;  // of stage `lane`: this warp's last fill
    for (uint32_t n = 0; ok; ++n) {
        const uint32_t s = n % kItems;
        ok = wait.all(ctl->item_full + s, n / kItems & 1);
        if (!ok) break;
        const Item it = ctl->items[s];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(ctl->item_empty + s);
        if (it.stop) break;
        const int32_t tiles = it.hi - it.lo;
        where.start(it);
        const int32_t tile_tokens = L.tile_tokens;
        const bool dual = Sh::kStreams == 2 && it.n > tile_tokens;
        if (is_k) {
            // Few tokens: a box per token and panel, one per lane, instead of the full tile's.
            constexpr int kQPanels = D / 64;
            const bool few = it.n < tile_tokens && it.n * kQPanels <= 32;
            const bool wide = Sh::kStreams == 2 ? dual : !(few && it.n * L.group <= Sh::kSmallRows);
            const uint32_t slot = n_items & 1;
            ok = wait.all(ctl->q_empty + slot, (n_items >> 1 & 1) ^ 1);
            if (ok && (wide || wide_before) && n_items > 0)
                ok = wait.all(ctl->q_empty + (slot ^ 1), (n_items - 1) >> 1 & 1);
            if (!ok) break;
            wide_before = wide;
            const uint32_t token_bytes = L.group * 128u;
            const uint32_t q_at = q_smem + (wide ? 0 : slot * Sh::kQSlot);
            if (lane == 0)
                tc::mbar_expect_tx(ctl->q_full + slot,
                                   kQPanels * token_bytes * static_cast<uint32_t>(few ? it.n : (dual ? 2 : 1) * tile_tokens));
            __syncwarp();
            if (few) {
                if (lane < it.n * kQPanels)
                    tc::tma_load_3d(q_at + lane % kQPanels * kPanel + lane / kQPanels * token_bytes, &L.tm_q_one,
                                    lane % kQPanels * 64, it.head * L.group, it.tok + lane / kQPanels, ctl->q_full + slot);
            } else if (lane < kQPanels * (dual ? 2 : 1)) {
                tc::tma_load_3d(q_at + lane * kPanel, &L.tm_q, lane % kQPanels * 64, it.head * L.group,
                                it.tok + lane / kQPanels * tile_tokens, ctl->q_full + slot);
            }
        }
        ++n_items;
#pragma unroll 1
        for (int32_t t = 0; ok && t < tiles; ++t) {
            int32_t page, row;
            where.place(&page, &row);
            if (is_k && lane == 0) *static_cast<volatile int32_t *>(&ctl->tile) = t;
            if constexpr (Sh::kEarly) {
                const auto [sk, parity] = pos.at(true, t, dual, 0);
                const uint32_t sv = sk + Sh::kSide;
                ok = wait.all(ctl->kv_empty + sk, parity ^ 1) && wait.all(ctl->kv_empty + sv, parity ^ 1);
                if (!ok) break;
                if (lane == 0) {
                    tc::mbar_expect_tx(ctl->kv_full + sk, Sh::kStage);
                    tc::mbar_expect_tx(ctl->kv_full + sv, Sh::kStage);
                }
                __syncwarp();
                if (lane < boxes) {
                    const uint32_t to = ring + sk * Sh::kStage + lane * L.box_rows * 128;
                    tc::tma_load_4d(to, &L.tm_k, 0, row, it.head, page, ctl->kv_full + sk);
                    tc::tma_load_4d(to + Sh::kSide * Sh::kStage, &L.tm_v, 0, row, it.head, page, ctl->kv_full + sv);
                }
                if (lane == static_cast<int>(sk) || lane == static_cast<int>(sv)) filled = static_cast<int32_t>(parity);
            } else
#pragma unroll 1
            for (int h = 0; h < Sh::kHalves; ++h) {
                const auto [st, parity] = pos.at(is_k, t, dual, h);
                ok = wait.all(ctl->kv_empty + st, parity ^ 1);
                if (!ok) break;
                if (lane == 0) tc::mbar_expect_tx(ctl->kv_full + st, Sh::kStage);
                __syncwarp();
                if (lane < boxes)
#pragma unroll
                    for (int p = 0; p < Sh::kPanels; ++p)
                        tc::tma_load_4d(ring + st * Sh::kStage + p * kPanel + lane * L.box_rows * 128, map,
                                        h * Sh::kCols + p * 64, row, it.head, page, ctl->kv_full + st);
                if (lane == static_cast<int>(st)) filled = static_cast<int32_t>(parity);
            }
        }
        pos.next(tiles, dual);
    }
    // After a failure: copies in flight land before the block may leave (else every copy has been consumed).
    if (!ok) {
        if (lane < Sh::kStages && filled >= 0) drain_bar(ctl->kv_full + lane, filled);
        if (is_k && lane < 2 && n_items > static_cast<uint32_t>(lane)) {
            const uint32_t i = n_items - 1 - lane;
            drain_bar(ctl->q_full + (i & 1), i >> 1 & 1);
        }
    }
    __syncwarp();
}

// ---- the MMA warp ------------------------------------------------------------------------
//
// The whole warp runs the code and one elected lane issues: operands then stay
// in uniform registers.  The tensor pipe holds about three products (64 cycles
// each) beyond the one it runs, and a wait costs 50 cycles and more even where
// nothing is left to wait for, so what the next batch needs is looked at
// between a batch's products, while the pipe has work; after a batch's last
// product only its commits and the wait for the weights stand before the next
// one.  Stages are used in ring order: the place only steps.

// Instruction descriptors of the two products.
template <int D, bool kHalf>
struct Products {
    static constexpr uint32_t kType = kHalf ? 0u : tc::kIdescBf16;
    static constexpr uint32_t kIdescS = tc::idesc_f16_f32acc(kRows, kKeys) | kType;
    static constexpr uint32_t kIdescO = tc::idesc_f16_f32acc(kRows, Shape<D>::kCols) | kType | tc::kIdescBmn;
};

template <int D, bool kHalf>
struct Issuer {
    using Sh = Shape<D>;
    static constexpr uint32_t kIdescS = Products<D, kHalf>::kIdescS, kIdescO = Products<D, kHalf>::kIdescO;
    static constexpr int kScoreSteps = Sh::kCols / 16, kWeightSteps = kKeys / 16;  // products of a stage
    // A place in the ring: stage and the parity of its filling.
    struct Place {
        uint32_t stage, phase;
        __device__ __forceinline__ void step(uint32_t n) {
            stage += n;
            if (stage >= Sh::kStages) {
                stage -= Sh::kStages;
                phase ^= 1;
            }
        }
    };
    const Waiter &wait;
    uint32_t bars;  // address of the control block
    uint32_t ring, tmem;
    Place next;     // of the next first use
    uint32_t used;  // per O: parity of the items that used it
    // The unit whose product with P is still to be issued: its number, whether it starts O, whether its V is the next
    // in the ring (else it is at `v`, loaded), whether it is its item's last.
    uint32_t left;
    bool any, fresh, take, final;
    Place v;
    bool early;    // the V behind the next K has been used already
    bool k_ready;  // the next K has been seen to be there
    bool v_ready;  // so has the V of the unit left over

#define GDN_BAR(name, i) (bars + static_cast<uint32_t>(offsetof(Control<D>, name)) + (i) * 8u)

    __device__ __forceinline__ bool seen(uint32_t bar, uint32_t parity) const {
        return __all_sync(0xffffffffu, tc::mbar_test_wait(bar, parity));
    }
    // S of unit g from Q at q (low descriptor word) and the K tile at `k`; `between` runs after most products are issued.
    template <bool kFree, typename Between>
    __device__ __forceinline__ bool scores(uint32_t g, uint32_t q, Place k, bool q_free, uint32_t q_bar, Between between) {
#pragma unroll
        for (int h = 0; h < Sh::kHalves; ++h) {
            if (h > 0 && !wait.all(GDN_BAR(kv_full, k.stage), k.phase)) return false;
            tc::fence_after_sync();
            const uint32_t kd = tc::desc_lo(ring + k.stage * Sh::kStage, 16);
            const uint32_t qd = q + h * Sh::kPanels * (kPanel >> 4), d = tmem + (g & 1) * kKeys;
            constexpr int kFirst = kScoreSteps - kScoreSteps / 3;
            const bool last = h + 1 == Sh::kHalves;
            if (tc::elect_lane()) {
#pragma unroll
                for (int i = 0; i < kFirst; ++i)
                    tc::mma_f16_lo(d, qd + i / 4 * (kPanel >> 4) + (i % 4) * 2, kd + i / 4 * (kPanel >> 4) + (i % 4) * 2, kIdescS,
                                   h > 0 || i > 0);
            }
            __syncwarp();
            if (last) between();
            if (tc::elect_lane()) {
#pragma unroll
                for (int i = kFirst; i < kScoreSteps; ++i)
                    tc::mma_f16_lo(d, qd + i / 4 * (kPanel >> 4) + (i % 4) * 2, kd + i / 4 * (kPanel >> 4) + (i % 4) * 2, kIdescS, 1);
                if (last) tc::mma_commit(GDN_BAR(s_full, g & 1));
                if (kFree) tc::mma_commit(GDN_BAR(kv_empty, k.stage));
                if (last && q_free) tc::mma_commit(q_bar);
            }
            __syncwarp();
            k.step(1);
        }
        return true;
    }
    // O (+)= P V of the unit left over, V at `at`.
    template <bool kFree, typename Between>
    __device__ __forceinline__ bool weights(Place at, Between between) {
        const uint32_t b = left & 1, w = Sh::kStreams == 2 ? b : 0;
        any = false;
        if (!v_ready && !wait.all(GDN_BAR(kv_full, at.stage), at.phase)) return false;
        if (fresh) {
            if (!wait.all(GDN_BAR(o_free, w), (used >> w & 1) ^ 1)) return false;
            used ^= 1u << w;
        }
        if (!wait.all(GDN_BAR(p_full, b), left >> 1 & 1)) return false;
#pragma unroll
        for (int h = 0; h < Sh::kHalves; ++h) {
            if (h > 0 && !wait.all(GDN_BAR(kv_full, at.stage), at.phase)) return false;
            tc::fence_after_sync();
            const uint32_t vd = tc::desc_lo(ring + at.stage * Sh::kStage, kPanel);
            const uint32_t d = tmem + kTmemO + w * D + h * Sh::kCols, p = tmem + b * kKeys;
            constexpr int kFirst = kWeightSteps - 3;
            const bool last = h + 1 == Sh::kHalves;
            if (tc::elect_lane()) {
#pragma unroll
                for (int i = 0; i < kFirst; ++i)
                    tc::mma_f16_ta_lo(d, p + i * 8, vd + i * (2048 >> 4), kIdescO, !fresh || i > 0);
            }
            __syncwarp();
            if (last) between();
            if (tc::elect_lane()) {
#pragma unroll
                for (int i = kFirst; i < kWeightSteps; ++i) tc::mma_f16_ta_lo(d, p + i * 8, vd + i * (2048 >> 4), kIdescO, 1);
                if (kFree) tc::mma_commit(GDN_BAR(kv_empty, at.stage));
                if (last) tc::mma_commit(GDN_BAR(o_done, w));
                if (Sh::kStreams == 1 && last && final) tc::mma_commit(GDN_BAR(item_done, 0));
            }
            __syncwarp();
            at.step(1);
        }
        return true;
    }
    // Looked at between other products: the next K, and the V of the unit left over (behind `skip` tiles of the ring).
    __device__ __forceinline__ void look_k() { k_ready = seen(GDN_BAR(kv_full, next.stage), next.phase); }
    __device__ __forceinline__ void look_v() {
        if (any && take) v_ready = seen(GDN_BAR(kv_full, next.stage), next.phase);
    }
    // K of the next tile, which is then passed in the ring (and the V behind it, where that has been used).
    __device__ __forceinline__ bool take_k(Place *k) {
        if (!k_ready && !wait.all(GDN_BAR(kv_full, next.stage), next.phase)) return false;
        k_ready = false;
        *k = next;
        next.step(Sh::kHalves);
        if (early) next.step(Sh::kHalves);
        early = false;
        return true;
    }
    // The product held back, V from the ring where it is not at hand.
    template <typename Between>
    __device__ __forceinline__ bool use_left(Between between) {
        if (take) {
            v = next;
            next.step(Sh::kHalves);
        }
        return weights<true>(v, between);
    }
    __device__ __forceinline__ void leave(uint32_t unit, bool starts, bool from_ring, bool ends) {
        any = true;
        final = ends;
        left = unit;
        fresh = starts;
        take = from_ring;
        v_ready = !from_ring;
    }
    // An item of one row tile: unit g + t is key tile t.
    __device__ __forceinline__ bool single(uint32_t g, int32_t tiles, uint32_t q, uint32_t q_bar) {
#pragma unroll 1
        for (int32_t t = 0; t < tiles; ++t, ++g) {
            const bool more = t + 1 < tiles;
            Place k;
            if (!take_k(&k) || !scores<true>(g, q, k, !more, q_bar, [&] { look_v(); })) return false;
            if (any && !use_left([&] {
                    if (more) look_k();
                }))
                return false;
            leave(g, t < Sh::kStreams, true, !more);
        }
        return true;
    }
    // An item of two row tiles: units g + 2t and g + 2t + 1 are key tile t.
    __device__ __forceinline__ bool dual(uint32_t g, int32_t tiles, uint32_t q, uint32_t q_bar) {
#pragma unroll 1
        for (int32_t t = 0; t < tiles; ++t, g += 2) {
            const bool more = t + 1 < tiles;
            Place k;
            if (!take_k(&k) || !scores<false>(g, q, k, false, q_bar, [&] { look_v(); })) return false;
            if (any && !use_left([] {})) return false;
            leave(g, t == 0, true, false);
            if (!scores<true>(g + 1, q + (Sh::kQTile >> 4), k, !more, q_bar, [&] { look_v(); })) return false;
            v = next;
            next.step(Sh::kHalves);
            if (!weights<false>(v, [&] {
                    if (more) look_k();
                }))
                return false;
            leave(g + 1, t == 0, false, !more);
        }
        return true;
    }
    __device__ __forceinline__ void run(Control<D> *ctl, const AttentionLaunch &L, uint32_t q_smem) {
        const int32_t tile_tokens = L.tile_tokens;
        uint32_t unit = 0, n_items = 0;
        for (uint32_t n = 0;; ++n) {
            const uint32_t s = n % kItems, slot = n_items & 1;
            // The product held back does not wait for what is late: the next item, its Q or its first K.  Its V lies
            // behind the place of that K.
            if (any) {
                k_ready = seen(GDN_BAR(kv_full, next.stage), next.phase);
                if (!k_ready || !seen(GDN_BAR(item_full, s), n / kItems & 1) || !seen(GDN_BAR(q_full, slot), n_items >> 1 & 1)) {
                    Place at = v;
                    early = take;
                    if (take) {
                        at = next;
                        at.step(Sh::kHalves);
                    }
                    if (!weights<true>(at, [] {})) break;
                }
            }
            if (!wait.all(GDN_BAR(item_full, s), n / kItems & 1)) break;
            // (through a warp reduction: what the compiler knows to be uniform it keeps in uniform registers)
            const int32_t stop = __reduce_max_sync(0xffffffffu, ctl->items[s].stop);
            const int32_t tokens = __reduce_max_sync(0xffffffffu, ctl->items[s].n);
            const int32_t tiles = __reduce_max_sync(0xffffffffu, ctl->items[s].hi - ctl->items[s].lo);
            if (tc::elect_lane()) tc::mbar_arrive(ctl->item_empty + s);
            __syncwarp();
            if (stop) break;
            const bool two = Sh::kStreams == 2 && tokens > tile_tokens;
            const bool few = tokens < tile_tokens && tokens * (D / 64) <= 32;
            const bool wide = Sh::kStreams == 2 ? two : !(few && tokens * L.group <= Sh::kSmallRows);
            if (!wait.all(GDN_BAR(q_full, slot), n_items >> 1 & 1)) break;
            const uint32_t q = tc::desc_lo(q_smem + (wide ? 0 : slot * Sh::kQSlot), 16);
            const uint32_t q_bar = GDN_BAR(q_empty, slot);
            if (!(Sh::kStreams == 2 && two ? dual(unit, tiles, q, q_bar) : single(unit, tiles, q, q_bar))) break;
            unit += two ? 2 * tiles : tiles;
            ++n_items;
        }
        if (tc::elect_lane()) tc::mma_commit(GDN_BAR(drain, 0));
        __syncwarp();
        drain_bar(ctl->drain, 0);
    }
};

// With scores ahead of the weights (d = 64) nothing orders the two but the
// barriers, and a warp for each issues them: one for both takes 1500 cycles a
// unit with everything there, of which the products are 640.
template <int D, bool kHalf>
struct EarlyIssuer {
    using Sh = Shape<D>;
    static constexpr uint32_t kIdescS = Products<D, kHalf>::kIdescS, kIdescO = Products<D, kHalf>::kIdescO;
    // A place in the ring of K or of V.
    struct Place {
        uint32_t stage, phase;
        __device__ __forceinline__ void step() {
            if (++stage == Sh::kSide) {
                stage = 0;
                phase ^= 1;
            }
        }
    };
    const Waiter &wait;
    uint32_t bars;  // address of the control block
    uint32_t ring, tmem;
    Place at;       // of the next K or V
    uint32_t unit;

    // Tokens and key tiles of the n-th item; false at the end.
    __device__ __forceinline__ bool take(Control<D> *ctl, uint32_t n, int32_t *tokens, int32_t *tiles) const {
        const uint32_t s = n % kItems;
        if (!wait.all(GDN_BAR(item_full, s), n / kItems & 1)) return false;
        // (through a warp reduction: what the compiler knows to be uniform it keeps in uniform registers)
        const int32_t stop = __reduce_max_sync(0xffffffffu, ctl->items[s].stop);
        *tokens = __reduce_max_sync(0xffffffffu, ctl->items[s].n);
        *tiles = __reduce_max_sync(0xffffffffu, ctl->items[s].hi - ctl->items[s].lo);
        if (tc::elect_lane()) tc::mbar_arrive(ctl->item_empty + s);
        __syncwarp();
        return !stop;
    }
    // S of the next unit from Q at q and the next K (`passes`: its last use).
    __device__ __forceinline__ bool scores(uint32_t q, bool passes, bool q_free, uint32_t q_bar) {
        const uint32_t b = unit & 1;
        if (!wait.all(GDN_BAR(kv_full, at.stage), at.phase)) return false;
        if (!wait.all(GDN_BAR(s_free, b), (unit >> 1 & 1) ^ 1)) return false;
        tc::fence_after_sync();
        const uint32_t kd = tc::desc_lo(ring + at.stage * Sh::kStage, 16), d = tmem + b * kKeys;
        if (tc::elect_lane()) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i) tc::mma_f16_lo(d, q + i * 2, kd + i * 2, kIdescS, i > 0);
            tc::mma_commit(GDN_BAR(s_full, b));
            if (passes) tc::mma_commit(GDN_BAR(kv_empty, at.stage));
            if (q_free) tc::mma_commit(q_bar);
        }
        __syncwarp();
        if (passes) at.step();
        ++unit;
        return true;
    }
    // O (+)= P V of the next unit.
    __device__ __forceinline__ bool weights(bool passes, bool starts, uint32_t &used) {
        const uint32_t b = unit & 1, stage = Sh::kSide + at.stage;
        if (starts) {
            if (!wait.all(GDN_BAR(o_free, b), (used >> b & 1) ^ 1)) return false;
            used ^= 1u << b;
        }
        if (!wait.all(GDN_BAR(kv_full, stage), at.phase)) return false;
        if (!wait.all(GDN_BAR(p_full, b), unit >> 1 & 1)) return false;
        tc::fence_after_sync();
        const uint32_t vd = tc::desc_lo(ring + stage * Sh::kStage, kPanel);
        const uint32_t d = tmem + kTmemO + b * D, p = tmem + Sh::p_at(unit);
        if (tc::elect_lane()) {
#pragma unroll
            for (int i = 0; i < kKeys / 16; ++i) tc::mma_f16_ta_lo(d, p + i * 8, vd + i * (2048 >> 4), kIdescO, !starts || i > 0);
            tc::mma_commit(GDN_BAR(o_done, b));
            if (passes) tc::mma_commit(GDN_BAR(kv_empty, stage));
        }
        __syncwarp();
        if (passes) at.step();
        ++unit;
        return true;
    }
    __device__ __forceinline__ void run_scores(Control<D> *ctl, const AttentionLaunch &L, uint32_t q_smem) {
        int32_t tokens, tiles;
        bool ok = true;
#pragma unroll 1
        for (uint32_t n = 0; ok && take(ctl, n, &tokens, &tiles); ++n) {
            const uint32_t slot = n & 1;
            const bool two = tokens > L.tile_tokens;
            if (!wait.all(GDN_BAR(q_full, slot), n >> 1 & 1)) break;
            const uint32_t q = tc::desc_lo(q_smem + (two ? 0 : slot * Sh::kQSlot), 16), q_bar = GDN_BAR(q_empty, slot);
            const int32_t units = two ? 2 * tiles : tiles;
#pragma unroll 1
            for (int32_t j = 0; ok && j < units; ++j) {
                const bool second = two && (j & 1);
                ok = scores(second ? q + (Sh::kQTile >> 4) : q, second || !two, j + 1 == units, q_bar);
            }
        }
        drain(ctl, 0);
    }
    __device__ __forceinline__ void run_weights(Control<D> *ctl, const AttentionLaunch &L) {
        int32_t tokens, tiles;
        uint32_t used = 0;  // per O: parity of the items that used it
        bool ok = true;
#pragma unroll 1
        for (uint32_t n = 0; ok && take(ctl, n, &tokens, &tiles); ++n) {
            const bool two = tokens > L.tile_tokens;
            const int32_t units = two ? 2 * tiles : tiles;
#pragma unroll 1
            for (int32_t j = 0; ok && j < units; ++j) ok = weights(!two || (j & 1), j < Sh::kStreams, used);
        }
        drain(ctl, 1);
    }
    __device__ __forceinline__ void drain(Control<D> *ctl, int i) const {
        if (tc::elect_lane()) tc::mma_commit(GDN_BAR(drain, i));
        __syncwarp();
        drain_bar(ctl->drain + i, 0);
    }
#undef GDN_BAR
};

// ---- the softmax warps ----------------------------------------------------------------------

// Instruction fetch bounds this code before arithmetic does: a pass over 128
// scores unrolled with compares, selects and scalar arithmetic is ~1200
// instructions, and ncu showed the softmax warps stalled on `no_instruction`
// most of the time (issue slots 19 % used, tensor pipe 44 %).  So masks are
// applied in a rolled pass of their own through TMEM, only on tiles that need
// one, and the rest uses three-input maxima and packed pairs.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ void unpair(uint64_t d, float *lo, float *hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(*lo), "=f"(*hi) : "l"(d));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Scores outside columns [lo, hi) of this thread's row become minus infinity.
__device__ __forceinline__ void mask_scores(uint32_t t_s, int32_t lo, int32_t hi) {
#pragma unroll 1
    for (int q = 0; q < kKeys; q += 32) {  // (columns that all the warp's rows see stay)
        if (!__any_sync(0xffffffffu, lo > q || hi < q + 32)) continue;
        uint32_t x[32];
        tc::tmem_ld32(t_s + q, x);
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (q + i < lo || q + i >= hi) x[i] = 0xff800000u;
        tc::tmem_st32(t_s + q, x);
    }
}

// Of 32 keys from node `off` of a tree on (before node 0: keys of the context), those that a node with this word sees.
__device__ __forceinline__ uint32_t tree_bits(uint64_t word, int32_t off) {
    if (off >= 0) return off < 64 ? static_cast<uint32_t>(word >> off) : 0u;
    return off <= -32 ? 0xffffffffu : static_cast<uint32_t>(word << -off) | ((1u << -off) - 1);
}
// Scores of keys that this thread's node does not see become minus infinity; node 0's key stands in column `first`.
__device__ __forceinline__ void mask_tree(uint32_t t_s, uint64_t word, int32_t first) {
#pragma unroll 1
    for (int q = 0; q < kKeys; q += 32) {
        const uint32_t bits = tree_bits(word, q - first);
        if (!__any_sync(0xffffffffu, bits != 0xffffffffu)) continue;
        uint32_t x[32];
        tc::tmem_ld32(t_s + q, x);
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (!(bits >> i & 1)) x[i] = 0xff800000u;
        tc::tmem_st32(t_s + q, x);
    }
}

// Moves the running maximum m where the scores x make it; the factor for l and
// O (1 where it stayed) comes back in *f.  True if any row of the warp moved.
__device__ __forceinline__ bool move_max(const uint32_t (&x)[kKeys], bool valid, float c, float &m, float *f) {
    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int j = 0; j < kKeys; j += 2)
        top[j / 2 & 3] = max3(top[j / 2 & 3], __uint_as_float(x[j]), __uint_as_float(x[j + 1]));
    float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    mx = valid ? fmaxf(m, mx) : -INFINITY;
    const bool move = (m == -INFINITY && mx > -INFINITY) || (mx - m) * c > 8.f;
    *f = move ? ex2((m - mx) * c) : 1.f;  // 0 from the empty maximum
    if (move) m = mx;
    return __any_sync(0xffffffffu, move);
}

// Weights are held as 2^7 times exp2(c (S - m)) in fp16: with the maximum that lags by up to 2^8 they reach 2^15, under its
// largest value, and of a long context's small weights those down to 2^-32 of the largest stay (with the 2^-25 that a
// largest weight of 1 would leave, 131 thousand keys could lose 0.4 % of the sum).  The factor is the same for the sums and
// all parts of a row, and is gone in O / l.
template <bool kHalf>
constexpr float kWeightShift = kHalf ? 7.f : 0.f;

// P = exp2(c S - mc) over S in TMEM; the sum of the row's weights, and with kTop the largest score.
template <bool kHalf, bool kTop>
__device__ __forceinline__ float store_weights(uint32_t t_s, const uint32_t (&x)[kKeys], float c, float mc, float *top) {
    float most[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    const uint64_t c2 = pair(c, c), mc2 = pair(-mc, -mc);
    uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        uint32_t pw[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const int j = q * 64 + 2 * i;
            float p0, p1;
            if (kTop) most[i & 3] = max3(most[i & 3], __uint_as_float(x[j]), __uint_as_float(x[j + 1]));
            unpair(fma2(pair(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), c2, mc2), &p0, &p1);
            p0 = ex2(p0);
            p1 = ex2(p1);
            sum[i & 3] = add2(sum[i & 3], pair(p0, p1));
            pw[i] = pack2<kHalf>(p0, p1);
        }
        tc::tmem_st32(t_s + q * 32, pw);
    }
    if (kTop) *top = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
    float lo, hi;
    unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), &lo, &hi);
    return lo + hi;
}

// O of `cols` columns times f, in TMEM.
template <int kCount>
__device__ __forceinline__ void scale_o(uint32_t t_o, float f) {
#pragma unroll 1
    for (int q = 0; q < kCount / 16; ++q) {
        uint32_t o[16];
        tc::tmem_ld16(t_o + q * 16, o);
#pragma unroll
        for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
        tc::tmem_st16(t_o + q * 16, o);
    }
}

// 32 bytes at once, at a multiple of 32: whole sectors from threads that each write their own row.
__device__ __forceinline__ void store32(void *p, const uint32_t *x) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]), "r"(x[1]), "r"(x[2]),
                 "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
}

// Packed magnitudes: the larger of each half, NaN above all.
template <bool kHalf>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t d;
    if (kHalf)
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b & 0x7fff7fffu));
    else
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b & 0x7fff7fffu));
    return d;
}
template <bool kHalf>
__device__ __forceinline__ uint32_t max_magnitude(uint32_t top, uint4 x) {
    return max2<kHalf>(max2<kHalf>(max2<kHalf>(max2<kHalf>(top, x.x), x.y), x.z), x.w);
}
template <bool kHalf>
__device__ __forceinline__ bool not_finite(uint32_t top) {
    constexpr uint32_t kExp = kHalf ? 0x7c00u : 0x7f80u;
    return (top & kExp) == kExp || (top >> 16 & kExp) == kExp;
}

template <bool kHalf>
__device__ __forceinline__ float2 unpack2(uint32_t x) {
    if (kHalf) return __half22float2(*reinterpret_cast<__half2 *>(&x));
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}

// Packed pairs with zeros for NaN and infinities.
template <bool kHalf>
__device__ __forceinline__ uint32_t finite_part(uint32_t x) {
    constexpr uint32_t kExp = kHalf ? 0x7c00u : 0x7f80u;
    if ((x & kExp) == kExp) x &= 0xffff0000u;
    if ((x >> 16 & kExp) == kExp) x &= 0x0000ffffu;
    return x;
}

// s + the products of a pair.
template <bool kHalf>
__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float s) {
    const float2 x = unpack2<kHalf>(a), y = unpack2<kHalf>(b);
    return fmaf(x.y, y.y, fmaf(x.x, y.x, s));
}

// Adds to this thread's row of O, in TMEM, what the products left out: p V of the values that are NaN or infinite, over the
// keys that the row sees of [past.x, past.y) and [next.x, next.y), which not all of the item's tokens see.  p is made anew
// from the row's maximum.  At most the item's tokens and a window's edge of keys are looked at, whatever the context.  Out of
// line, as leave_out is: in line they cost a prompt of 8192 tokens, which calls neither, 2 % (instruction fetch).
struct LeftOut {
    int2 past, next;
    int32_t key_lo, key_hi;  // what the row sees
    int64_t req, head;       // request, K/V head
    const uint16_t *q;       // of the row
    float mc;                // its maximum times c
    uint32_t t_o, t_other;   // its accumulators: the sum of both with these factors is left in the first
    bool two;
    float f0, f1;
};
struct TreeLeftOut : LeftOut {
    int32_t ctx;    // the first new token's key,
    uint64_t word;  // and which of theirs the row sees
};
template <int D, bool kHalf, bool kTree>
__device__ __noinline__ void add_left_out(const AttentionLaunch &L, const std::conditional_t<kTree, TreeLeftOut, LeftOut> r) {
    const gdn_paged_cache_t &c = L.a.cache;
    const int lane = threadIdx.x & 31;
    // Element 0 of key j's K or V; null: a bad page, whose keys are zeros.
    auto key = [&](int32_t j, const void *base, int64_t page_stride, int64_t slot_stride, int64_t head_stride) {
        const int32_t idx = j / c.page_size, page = L.a.block_table[r.req * L.a.table_stride + idx];
        const bool good = page >= 0 && page < c.num_pages;
        return good ? static_cast<const uint16_t *>(base) + page * page_stride + (j - idx * c.page_size) * slot_stride +
                          r.head * head_stride
                    : nullptr;
    };
    if (r.two) {
#pragma unroll 1
        for (int col = 0; col < D; col += 16) {
            uint32_t o[16], o1[16];
            tc::tmem_ld16(r.t_o + col, o);
            tc::tmem_ld16(r.t_other + col, o1);
#pragma unroll
            for (int j = 0; j < 16; ++j)
                o[j] = __float_as_uint(fmaf(__uint_as_float(o1[j]), r.f1, __uint_as_float(o[j]) * r.f0));
            tc::tmem_st16(r.t_o + col, o);
        }
    }
    const int32_t n_past = max(r.past.y - r.past.x, 0), n = n_past + max(r.next.y - r.next.x, 0);
#pragma unroll 1
    for (int32_t base = 0; base < n; base += 32) {
        // A key per lane: those with such values.
        const int32_t i = base + lane, mine = i < n_past ? r.past.x + i : r.next.x + i - n_past;
        const uint16_t *at = i < n ? key(mine, c.v, c.v_page_stride, c.v_slot_stride, c.v_head_stride) : nullptr;
        uint32_t top = 0;
#pragma unroll 4
        for (int x = 0; x < D / 8; ++x)
            if (at) top = max_magnitude<kHalf>(top, reinterpret_cast<const uint4 *>(at)[x]);
#pragma unroll 1
        for (uint32_t found = __ballot_sync(0xffffffffu, not_finite<kHalf>(top)); found; found &= found - 1) {
            const int32_t j = __shfl_sync(0xffffffffu, mine, __ffs(found) - 1);
            bool sees = j >= r.key_lo && j < r.key_hi;
            if constexpr (kTree) sees = sees && (j < r.ctx || (r.word >> (j - r.ctx) & 1));
            const uint4 *k = reinterpret_cast<const uint4 *>(key(j, c.k, c.k_page_stride, c.k_slot_stride, c.k_head_stride));
            const uint4 *v = reinterpret_cast<const uint4 *>(key(j, c.v, c.v_page_stride, c.v_slot_stride, c.v_head_stride));
            float s = 0.f;
#pragma unroll 2
            for (int x = 0; x < D / 8; ++x) {
                if (!sees) continue;
                const uint4 a = reinterpret_cast<const uint4 *>(r.q)[x], b = k[x];
                s = dot2<kHalf>(a.w, b.w, dot2<kHalf>(a.z, b.z, dot2<kHalf>(a.y, b.y, dot2<kHalf>(a.x, b.x, s))));
            }
            const float p = ex2(fmaf(s, L.c, -r.mc));
            __syncwarp();
#pragma unroll 1
            for (int col = 0; col < D; col += 16) {
                const uint4 lo = v[col / 8], hi = v[col / 8 + 1];
                if (!not_finite<kHalf>(max_magnitude<kHalf>(max_magnitude<kHalf>(0, lo), hi))) continue;  // (as for all lanes)
                const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                uint32_t o[16];
                tc::tmem_ld16(r.t_o + col, o);
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const uint32_t left = sees ? w[x] ^ finite_part<kHalf>(w[x]) : 0;  // (a zero where the product has it)
                    const float2 y = unpack2<kHalf>(left);
                    if (left & 0xffffu) o[2 * x] = __float_as_uint(fmaf(p, y.x, __uint_as_float(o[2 * x])));
                    if (left >> 16) o[2 * x + 1] = __float_as_uint(fmaf(p, y.y, __uint_as_float(o[2 * x + 1])));
                }
                __syncwarp();
                tc::tmem_st16(r.t_o + col, o);
            }
        }
    }
}

// f(byte offset) for each 16-byte piece of rows [r0, r1) of a V stage, dealt over the warpgroup's threads.
template <int D, typename F>
__device__ __forceinline__ void value_rows(int32_t r0, int32_t r1, int32_t thread, F f) {
    constexpr int kPieces = Shape<D>::kPanels * 8;
    if (r0 < 0) r0 = 0;
    if (r1 > kKeys) r1 = kKeys;
#pragma unroll 1
    for (int32_t i = r0 * kPieces + thread; i < r1 * kPieces; i += 128)
        f((i % kPieces / 8) * kPanel + i / kPieces * 128 + i % 8 * 16);
}

// Zeros for the values that are NaN or infinite in rows [next, next_end) and [first, past) of a V stage, and the item's
// number `nth` in *mark.
template <int D, bool kHalf>
__device__ __noinline__ void leave_out(uint8_t *tile, uint32_t *mark, uint32_t nth, int32_t next, int32_t next_end, int32_t first,
                                       int32_t past, int32_t thread) {
    // (The mark first: of two row tiles' warpgroups, which look through the same values, one may find them left out by the
    // other.)
    *static_cast<volatile uint32_t *>(mark) = nth;
    __threadfence_block();
#pragma unroll 1
    for (int i = 0; i < 2; ++i)
        value_rows<D>(i ? first : next, i ? past : next_end, thread, [&](uint32_t x) {
            uint4 *p = reinterpret_cast<uint4 *>(tile + x);
            *p = make_uint4(finite_part<kHalf>(p->x), finite_part<kHalf>(p->y), finite_part<kHalf>(p->z), finite_part<kHalf>(p->w));
        });
}

template <int D, bool kHalf, bool kTree>
__device__ void softmax_rows(const AttentionLaunch &L, Control<D> *ctl, uint8_t *ring, uint32_t tmem, const Waiter &wait) {
    using Sh = Shape<D>;
    const PagedAttentionArgs &a = L.a;
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3;
    const uint32_t group = (threadIdx.x >> 7) - 1;
    const uint32_t w = Sh::kStreams == 2 ? group : 0;  // warpgroup = buffer = O, with two streams
    const int row = warp * 32 + lane;
    const int32_t u_tile = row / L.group, g = row - u_tile * L.group;
    const int32_t tile_tokens = L.tile_tokens;
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;  // this warp's TMEM lanes
    const uint32_t t_o = tmem + kTmemO + lanes;
    const float c = L.c;
    Ring<D> pos;
    uint32_t unit0 = 0;              // first unit of the item
    uint32_t n_items = 0, ml_got = 0;
    for (uint32_t n = 0;; ++n) {
        const uint32_t sl = n % kItems;
        if (!wait.all(ctl->item_full + sl, n / kItems & 1)) return;
        const Item it = ctl->items[sl];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(ctl->item_empty + sl);
        if (it.stop) return;
        const int32_t tiles = it.hi - it.lo;
        const bool dual = Sh::kStreams == 2 && it.n > tile_tokens;
        // Which part of the item is this warpgroup's: row tile of a dual one, even or odd key tiles of another.
        const int32_t part = Sh::kStreams == 2 ? static_cast<int32_t>((w ^ unit0) & 1) : 0;
        const int32_t u = u_tile + (dual ? part * tile_tokens : 0);
        const int32_t rows = (dual ? (part ? it.n - tile_tokens : tile_tokens) : it.n) * L.group;
        const bool valid = row < rows && u_tile < tile_tokens;
        const bool any_row = warp * 32 < rows;
        const int32_t key_hi = it.pos + u + 1;
        const int32_t key_lo = a.window > 0 && key_hi > a.window ? key_hi - a.window : 0;
        int32_t row_lo, row_hi;
        visible_rows(it, a.window, &row_lo, &row_hi);
        const int32_t units = dual ? 2 * tiles : tiles;
        // The nodes that this row's sees: itself and those before it that its word names.  (Rows of no token: all keys.)
        uint64_t word = 0;
        if (kTree && valid) word = a.masks[static_cast<int64_t>(it.tok) + u] & ((2ull << (it.pos + u - it.ctx)) - 1);
        float m = -INFINITY, l = 0.f;
        // (with one stream the second warpgroup writes an item's O while the first one is on with the next)
        for (int32_t j = part; j < units && (Sh::kStreams == 2 || group == 0); j += Sh::kStreams) {
            const uint32_t unit = unit0 + j, b = unit & 1;
            const int32_t t = dual ? j >> 1 : j;
            const int32_t k0 = (it.lo + t) * kKeys;
            if (!wait.all(ctl->s_full + b, unit >> 1 & 1)) return;
            tc::fence_after_sync();
            // With scores ahead of the weights S may be written again once it is in registers.
            auto taken = [&] {
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(ctl->s_free + b);
            };
            // And the weights before these have to be used (the last of the item before were waited for with its O).
            auto used = [&] {
                if (j >= Sh::kStreams && !wait.all(ctl->o_done + w, (unit - 2) >> 1 & 1)) return false;
                tc::fence_after_sync();
                return true;
            };
            if (Sh::kEarly && !any_row) {
                taken();
                if (!used()) return;
            }
            if (any_row) {
                const uint32_t t_s = tmem + b * kKeys + lanes;
                if (kTree) {
                    if (k0 + kKeys > it.ctx) mask_tree(t_s, word, valid ? it.ctx - k0 : kKeys);
                } else if (__any_sync(0xffffffffu, valid && (k0 + kKeys > key_hi || k0 < key_lo)))
                    mask_scores(t_s, valid ? key_lo - k0 : 0, valid ? key_hi - k0 : kKeys);
                uint32_t x[kKeys];
                tc::tmem_ld128(t_s, x);
                if (Sh::kEarly) taken();
                // With kBeside the weights are made by the maximum so far and the tile's is found beside them; only if
                // that passes it by too much for some row are they made again.  (Rows without one get theirs first.)
                float f = 1.f, sum, top;
                bool moved = (!Sh::kBeside || __any_sync(0xffffffffu, valid && m == -INFINITY)) && move_max(x, valid, c, m, &f);
                if (Sh::kEarly && !used()) return;
#pragma unroll 1
                while (true) {
                    if (moved) {
                        l *= f;
                        if (j >= Sh::kStreams) {
                            // With two streams O is done: S of this unit came after it, or see above.
                            if (Sh::kStreams == 1) {
                                if (!wait.all(ctl->o_done, (unit - 1) & 1)) return;
                                tc::fence_after_sync();
                            }
                            scale_o<D>(t_o + w * D, f);
                        }
                    }
                    sum = store_weights<kHalf, Sh::kBeside>(tmem + Sh::p_at(unit) + lanes, x, c,
                                                            (m == -INFINITY ? 0.f : m * c) - kWeightShift<kHalf>, &top);
                    if (!Sh::kBeside) break;
                    const bool up = valid && (top - m) * c > 8.f;
                    moved = __any_sync(0xffffffffu, up);
                    if (!moved) break;
                    f = up ? ex2((m - top) * c) : 1.f;
                    if (up) m = top;
                }
                l += sum;
            }
            // A weight of zero does not keep a NaN or infinity out of the product.  Value rows that no token of the item
            // sees are zeroed before it; where tokens see different keys of the tile, the rest is looked through, and what
            // is not finite there is left out (zeroed) and added to the rows that see it when O is written.
            const bool some = k0 + kKeys > row_hi || k0 < row_lo;
            const bool differ = kTree ? k0 + kKeys > it.ctx
                                      : it.n > 1 && (k0 + kKeys > it.pos + 1 || (a.window > 0 && it.pos + it.n - k0 > a.window));
            if (some || differ) {
#pragma unroll 1
                for (uint32_t h = 0; h < Sh::kHalves; ++h) {
                    // Two waits: a parity tells this fill from the one before only once that one has been consumed.
                    const auto [st, parity] = pos.at(false, t, dual, h);
                    if (!wait.all(ctl->kv_empty + st, parity ^ 1) || !wait.all(ctl->kv_full + st, parity)) return;
                    uint8_t *tile = ring + st * Sh::kStage;
                    if (some) {
                        value_rows<D>(row_hi - k0, kKeys, row, [&](uint32_t x) { *reinterpret_cast<uint4 *>(tile + x) = make_uint4(0, 0, 0, 0); });
                        value_rows<D>(0, row_lo - k0, row, [&](uint32_t x) { *reinterpret_cast<uint4 *>(tile + x) = make_uint4(0, 0, 0, 0); });
                    }
                    if (differ) {  // past the first token, and behind the last one's window
                        const int32_t next = (kTree ? it.ctx : it.pos + 1) - k0, past = a.window > 0 ? it.pos + it.n - a.window - k0 : 0;
                        uint32_t top = 0;  // largest magnitudes seen
#pragma unroll 1
                        for (int i = 0; i < 2; ++i)
                            value_rows<D>(i ? row_lo - k0 : next, i ? past : row_hi - k0, row,
                                          [&](uint32_t x) { top = max_magnitude<kHalf>(top, *reinterpret_cast<uint4 *>(tile + x)); });
                        if (not_finite<kHalf>(top))
                            leave_out<D, kHalf>(tile, ctl->bad + sl, n + 1, next, row_hi - k0, row_lo - k0, past, row);
                    }
                }
                tc::fence_proxy_async_smem();
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(ctl->p_full + b);
        }
        // O to memory: the result, or this split's part of it.
        const bool pair = Sh::kStreams == 2 && !dual && tiles > 1;  // two warpgroups hold one row tile's parts
        if (Sh::kStreams == 1 && group == 0) {
            if (!wait.all(&ctl->ml_empty, (n_items & 1) ^ 1)) return;
            ctl->ml[row] = make_float2(m, l);
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(ctl->ml_full);
        } else if (Sh::kStreams == 1) {
            if (!wait.item(ctl->ml_full, n_items & 1)) return;
            m = ctl->ml[row].x;
            l = ctl->ml[row].y;
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&ctl->ml_empty);
            if (!wait.all(&ctl->item_done, n_items & 1)) return;
            tc::fence_after_sync();
        } else if (dual || part < tiles) {
            const uint32_t last = unit0 + units - 1 - ((units - 1 - part) & 1);
            if (!wait.all(ctl->o_done + w, last >> 1 & 1)) return;
            tc::fence_after_sync();
        }
        ++n_items;
        float f0 = 1.f, f1 = 0.f;  // factors of this warpgroup's O and the other's
        const bool writer = Sh::kStreams == 2 ? dual || part == 0 : group == 1;
        if (pair && part == 1) {
            ctl->ml[row] = make_float2(m, l);
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(ctl->ml_full + w);
        } else if (pair) {
            if (!wait.all(ctl->ml_full + (w ^ 1), ml_got++ & 1)) return;
            tc::fence_after_sync();
            const float2 other = ctl->ml[row];
            // (Both empty: factors of one.  Either half's sum may still be NaN, from scores that are.)
            const float top = fmaxf(m, other.x);
            f1 = 1.f;
            if (top > -INFINITY) {
                f0 = ex2((m - top) * c);
                f1 = ex2((other.x - top) * c);
                m = top;
            }
            l = l * f0 + other.y * f1;
        }
        if (writer && any_row) {
            const int64_t head = static_cast<int64_t>(it.head) * L.group + g;
            const bool split = it.parts > 1;
            const int64_t first = (it.partial + static_cast<int64_t>(u) * it.splits) * a.h_q + head;
            const int64_t prow = first + static_cast<int64_t>(it.part) * a.h_q;
            if (valid && it.rows >= 0 && it.part == 0)
                L.ws.rows[it.rows + static_cast<int64_t>(u) * a.h_q + head] = {
                    static_cast<int32_t>((it.tok + u) * a.h_q + head), split ? it.parts : 0, first};
            const bool none = l == 0.f;  // no key seen, or all weights zero
            if (!split) {
                const float inv = none ? 0.f : 1.f / l;
                f0 *= inv;
                f1 *= inv;
            } else if (valid) {
                L.ws.ml[prow] = make_float2(m * c, l);
            }
            uint16_t *out = a.o + ((static_cast<int64_t>(it.tok) + u) * a.h_q + head) * D;
            float *pout = L.ws.o + prow * D;
            if (__any_sync(0xffffffffu, none)) {  // a row that saw no key
#pragma unroll 1
                for (int j = 0; valid && none && j < D; j += 8) {
                    if (split) {
                        *reinterpret_cast<uint4 *>(pout + j) = make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4 *>(pout + j + 4) = make_uint4(0, 0, 0, 0);
                    } else {
                        *reinterpret_cast<uint4 *>(out + j) = make_uint4(0, 0, 0, 0);
                    }
                }
            }
            const bool writes = valid && !none;
            bool two = pair;  // the row's O is in both accumulators
            if (__any_sync(0xffffffffu, *static_cast<volatile uint32_t *>(ctl->bad + sl) == n + 1)) {
                // Keys of the item's tiles that its tokens see differently, as they were looked through above: behind the
                // last token's window, past the first token.
                std::conditional_t<kTree, TreeLeftOut, LeftOut> left;
                const int32_t end = it.hi * kKeys < row_hi ? it.hi * kKeys : row_hi;
                left.past = make_int2(0, 0);
                if (a.window > 0) left.past = make_int2(max(row_lo, it.lo * kKeys), min(it.pos + it.n - a.window, end));
                left.next = make_int2(max(max(kTree ? it.ctx : it.pos + 1, it.lo * kKeys), left.past.y), end);
                if constexpr (kTree) {
                    left.ctx = it.ctx;
                    left.word = word;
                }
                left.key_lo = writes ? key_lo : INT_MAX;
                left.key_hi = key_hi;
                left.req = it.req;
                left.head = it.head;
                left.q = a.q + (static_cast<int64_t>(it.tok) + u) * a.q_token_stride + head * D;
                left.mc = m == -INFINITY ? 0.f : m * c;
                left.t_o = t_o + w * D;
                left.t_other = t_o + (w ^ 1) * D;
                left.two = pair;
                left.f0 = f0;
                left.f1 = f1;
                add_left_out<D, kHalf, kTree>(L, left);
                if (pair) f0 = 1.f;
                two = false;
            }
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
                uint32_t o[32];
                tc::tmem_ld32(t_o + w * D + q * 32, o);
                if (two) {
                    uint32_t o1[32];
                    tc::tmem_ld32(t_o + (w ^ 1) * D + q * 32, o1);
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        o[j] = __float_as_uint(fmaf(__uint_as_float(o1[j]), f1, __uint_as_float(o[j]) * f0));
                }
                if (split) {  // (f0 is 1 without a pair)
                    if (writes)
#pragma unroll
                        for (int j = 0; j < 32; j += 8) store32(pout + q * 32 + j, o + j);
                } else if (writes) {
                    const float f = two ? 1.f : f0;
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        o[j] = pack2<kHalf>(__uint_as_float(o[2 * j]) * f, __uint_as_float(o[2 * j + 1]) * f);
#pragma unroll
                    for (int j = 0; j < 16; j += 8) {
                        if (L.o_32) {
                            store32(out + q * 32 + j * 2, o + j);
                        } else {  // the caller's o lies at a multiple of 16
                            *reinterpret_cast<uint4 *>(out + q * 32 + j * 2) = make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                            *reinterpret_cast<uint4 *>(out + q * 32 + j * 2 + 8) = make_uint4(o[j + 4], o[j + 5], o[j + 6], o[j + 7]);
                        }
                    }
                }
            }
        }
        if (writer) {
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                tc::mbar_arrive(ctl->o_free + w);
                if (pair) tc::mbar_arrive(ctl->o_free + (w ^ 1));
            }
        }
        pos.next(tiles, dual);
        unit0 += units;
    }
}

template <int D, bool kHalf, bool kTree>
__global__ void __launch_bounds__(Shape<D>::kThreads, 1) attention_kernel(const __grid_constant__ AttentionLaunch L) {
    using Sh = Shape<D>;
    extern __shared__ uint8_t raw[];
    uint8_t *base = raw + ((1024u - (tc::smem_u32(raw) & 1023u)) & 1023u);
    uint8_t *ring = base + Sh::kQ;
    Control<D> *ctl = reinterpret_cast<Control<D> *>(ring + Sh::kStages * Sh::kStage);
    static_assert(sizeof(Control<D>) <= Sh::kControl && Sh::kSmem <= 227 * 1024, "shared memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        for (int i = 0; i < Sh::kStages; ++i) {
            tc::mbar_init(ctl->kv_full + i, 1);
            tc::mbar_init(ctl->kv_empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(ctl->q_full + i, 1);
            tc::mbar_init(ctl->q_empty + i, 1);
            tc::mbar_init(ctl->drain + i, 1);
            tc::mbar_init(ctl->s_full + i, 1);
            tc::mbar_init(ctl->s_free + i, 4);
            tc::mbar_init(ctl->p_full + i, 4);
            tc::mbar_init(ctl->o_done + i, 1);
            tc::mbar_init(ctl->o_free + i, 4);
            tc::mbar_init(ctl->ml_full + i, 4);
        }
        for (int i = 0; i < kItems; ++i) {
            tc::mbar_init(ctl->item_full + i, 1);
            tc::mbar_init(ctl->item_empty + i, 3 + 8);  // load and MMA warps, softmax warps
            ctl->bad[i] = 0;
        }
        tc::mbar_init(&ctl->ml_empty, 4);
        tc::mbar_init(&ctl->item_done, 1);
        ctl->fail = 0;
        ctl->tile = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    Request first_read = {0, 0, 0};  // the scheduler's first lengths, on their way while the block sets up
    if (warp == 2) first_read = load_request<kTree>(L.a, static_cast<int64_t>(L.a.num_reqs) - 1 - lane, blockIdx.x == 0);
    if (warp == 3) {
        if (lane == 0) {
            tc::prefetch_tensor_map(&L.tm_k);
            tc::prefetch_tensor_map(&L.tm_v);
            tc::prefetch_tensor_map(&L.tm_q);
            tc::prefetch_tensor_map(&L.tm_q_one);
        }
        __syncwarp();
        tc::tmem_alloc(&ctl->tmem, kTmemCols);
    }
    tc::fence_proxy_async_smem();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = ctl->tmem;
    const Waiter wait = {&ctl->fail, &ctl->tile};
    // 384 threads are launched with 168 registers each: 128 x 72 + 256 x 216 is the same sum.
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 0 || (warp == 3 && !Sh::kEarly)) {
            load_tiles<D>(L, ctl, tc::smem_u32(base), tc::smem_u32(ring), wait, warp == 0);
        } else if (warp != 2) {
            const uint32_t t = __reduce_max_sync(0xffffffffu, tmem);
            if constexpr (Sh::kEarly) {
                EarlyIssuer<D, kHalf> issuer = {wait, tc::smem_u32(ctl), tc::smem_u32(ring), t};
                if (warp == 1)
                    issuer.run_scores(ctl, L, tc::smem_u32(base));
                else
                    issuer.run_weights(ctl, L);
            } else {
                Issuer<D, kHalf> issuer = {wait, tc::smem_u32(ctl), tc::smem_u32(ring), t};
                issuer.run(ctl, L, tc::smem_u32(base));
            }
        } else {
            schedule<D, kTree>(L, ctl, wait, first_read);
            // What follows this kernel in the stream relies on the counter's reset being over, and a block that took one
            // item or none has not waited for it.
            asm volatile("griddepcontrol.wait;" ::: "memory");
            // Tokens of no request: zeros.  (The last range may run backwards, into the tokens of a request before it.)
            const PagedAttentionArgs &a = L.a;
            int32_t end = a.num_reqs > 0 ? a.cu_seqlens[a.num_reqs] : 0;
            if (end < a.num_tokens) {
                int32_t served = 0;
#pragma unroll 8
                for (int64_t r = lane; r < a.num_reqs; r += 32) {
                    const int32_t b = a.cu_seqlens[r], e = a.cu_seqlens[r + 1];
                    if (b >= 0 && b <= e && e <= a.num_tokens) served = max(served, e);
                }
                end = max(end, __reduce_max_sync(0xffffffffu, served));
            }
            const int64_t chunk = static_cast<int64_t>(a.h_q) * D / 8;
#pragma unroll 1
            for (int64_t i = end * chunk + blockIdx.x * 32 + lane; i < a.num_tokens * chunk; i += gridDim.x * 32)
                reinterpret_cast<uint4 *>(a.o)[i] = make_uint4(0, 0, 0, 0);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        softmax_rows<D, kHalf, kTree>(L, ctl, ring, tmem, wait);
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (threadIdx.x == 0 && ctl->fail) report(L.a.dev_status, GDN_DEV_TIMEOUT);
    if (warp == 3) {
        tc::tmem_relinquish();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

// ---- joining the splits -----------------------------------------------------------------------

constexpr int kJoinWarps = 4;
constexpr int kJoinBlocksPerSm = 8;

// Parts s0 + j * step (j < 4) of a row; lane i holds columns 2 i + 64 v.
template <int D>
__device__ __forceinline__ void read_parts(const float *o, int64_t stride, int32_t s0, int32_t step, int32_t parts,
                                           float2 (&x)[4][D / 64], int lane) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (s0 + j * step < parts)
#pragma unroll
            for (int v = 0; v < D / 64; ++v)
                x[j][v] = *reinterpret_cast<const float2 *>(o + (s0 + j * step) * stride + v * 64 + lane * 2);
}
// Adds them to sums[j * kMore]; a part's weight is in ml[s / 32].x of lane s % 32.
template <int D, int kWords, int kMore>
__device__ __forceinline__ void add_parts(const float2 (&x)[4][D / 64], int32_t s0, int32_t step, int32_t parts,
                                          const float2 (&ml)[kWords], float2 (&sums)[3 * kMore + 1][D / 64]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int32_t s = s0 + j * step;
        float w = 0.f;
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
            const float y = __shfl_sync(0xffffffffu, ml[k].x, s & 31);
            if (s >> 5 == k) w = y;
        }
        if (s < parts)
#pragma unroll
            for (int v = 0; v < D / 64; ++v) {
                sums[j * kMore][v].x = fmaf(w, x[j][v].x, sums[j * kMore][v].x);
                sums[j * kMore][v].y = fmaf(w, x[j][v].y, sums[j * kMore][v].y);
            }
    }
}

// o = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s over a row's parts.  Four
// sums, of parts k, k + 4, ..., are added up in order: where rows are few, by
// the four warps of a block, one block a row; else by one warp, four rows a
// block - in the same order, so a row's bits do not depend on how many there
// are.  Requests that were not split have no rows here.  Bound by the latency
// of dependent reads (the row, then its partials) where there are few rows, by
// L2 or, behind long contexts, by memory where there are many.
template <int D, bool kHalf>
__global__ void __launch_bounds__(kJoinWarps * 32, 5) join_kernel(const __grid_constant__ AttentionLaunch L) {
    constexpr int kVec = D / 64;
    constexpr int kWords = (kMaxSplits + 31) / 32;
    __shared__ float2 sum[kJoinWarps - 1][D / 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t h_q = L.a.h_q;
    // Every thread waits for the attention kernel's end, also one with nothing to join: what follows this kernel in
    // the stream relies on both.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // A descriptor is asked for with the number of rows: of the row that is this team's where there are as many teams.
    const int64_t nth = blockIdx.x * static_cast<int64_t>(kJoinWarps) + warp;
    JoinRow of_block = {0, 0, 0}, of_warp = {0, 0, 0};
    if (lane == 0 && blockIdx.x < L.ws.max_rows) of_block = L.ws.rows[blockIdx.x];
    if (lane == 0 && nth < L.ws.max_rows) of_warp = L.ws.rows[nth];
    const int64_t rows = *L.ws.num_rows < L.ws.max_rows ? *L.ws.num_rows : L.ws.max_rows;
    const bool alone = rows <= gridDim.x;  // a block a row
    // The rows of a block or warp, up to 32 at a time, one descriptor per lane: those that are in o already cost no
    // round of their own.
    const int64_t teams = alone ? gridDim.x : gridDim.x * kJoinWarps, team = alone ? blockIdx.x : nth;
    const int64_t per = (rows + teams - 1) / teams, begin = team * per, end = begin + per < rows ? begin + per : rows;
    for (int64_t i0 = begin; i0 < end; i0 += 32) {
        JoinRow mine = {0, 0, 0};
        if (per == 1) {
            if (lane == 0) mine = alone ? of_block : of_warp;
        } else if (i0 + lane < end) {
            mine = L.ws.rows[i0 + lane];
        }
        // (a call that timed out or was given overlapping token ranges leaves rows unwritten)
        uint32_t todo = __ballot_sync(0xffffffffu, mine.parts >= 2 && mine.parts <= kMaxSplits && mine.first >= 0 &&
                                                       mine.first + (mine.parts - 1) * h_q < L.ws.partials * h_q &&
                                                       mine.out >= 0 && mine.out < L.ws.max_rows);
        for (; todo; todo &= todo - 1) {
            const int src = __ffs(todo) - 1;
            const int32_t row_out = __shfl_sync(0xffffffffu, mine.out, src), parts = __shfl_sync(0xffffffffu, mine.parts, src);
            const int64_t first = __shfl_sync(0xffffffffu, mine.first, src);
            const float *o = L.ws.o + first * D;
            const int32_t s0 = alone ? warp : 0, step = alone ? kJoinWarps : 1;
            float2 x[4][kVec];
            read_parts<D>(o, h_q * D, s0, step, parts, x, lane);
            float2 ml[kWords];
            float top = -INFINITY;
#pragma unroll
            for (int k = 0; k < kWords; ++k) {
                ml[k] = make_float2(-INFINITY, 0.f);
                if (lane + 32 * k < parts) ml[k] = L.ws.ml[first + (lane + 32 * k) * h_q];
                top = fmaxf(top, ml[k].x);
            }
#pragma unroll
            for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
            if (top == -INFINITY) top = 0.f;
            float l = 0.f;
#pragma unroll
            for (int k = 0; k < kWords; ++k) {
                ml[k].x = ex2(ml[k].x - top);  // the part's weight
                l = fmaf(ml[k].x, ml[k].y, l);
            }
#pragma unroll
            for (int k = 16; k > 0; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
            float2 acc[kVec];
            if (alone) {
                float2 mine4[1][kVec] = {};
#pragma unroll 1
                for (int32_t s = warp; s < parts; s += 4 * kJoinWarps) {
                    if (s > warp) read_parts<D>(o, h_q * D, s, step, parts, x, lane);
                    add_parts<D, kWords, 0>(x, s, kJoinWarps, parts, ml, mine4);
                }
                if (warp > 0)
#pragma unroll
                    for (int v = 0; v < kVec; ++v) sum[warp - 1][v * 32 + lane] = mine4[0][v];
                __syncthreads();
#pragma unroll
                for (int v = 0; v < kVec; ++v) {
                    acc[v] = mine4[0][v];
#pragma unroll
                    for (int k = 0; k < kJoinWarps - 1; ++k) {
                        acc[v].x += sum[k][v * 32 + lane].x;
                        acc[v].y += sum[k][v * 32 + lane].y;
                    }
                }
                __syncthreads();
            } else {
                float2 four[4][kVec] = {};
#pragma unroll 1
                for (int32_t s = 0; s < parts; s += 4) {
                    if (s > 0) read_parts<D>(o, h_q * D, s, step, parts, x, lane);
                    add_parts<D, kWords, 1>(x, s, 1, parts, ml, four);
                }
#pragma unroll
                for (int v = 0; v < kVec; ++v) {
                    acc[v] = four[0][v];
#pragma unroll
                    for (int k = 1; k < 4; ++k) {
                        acc[v].x += four[k][v].x;
                        acc[v].y += four[k][v].y;
                    }
                }
            }
            if (!alone || warp == 0) {
                const bool none = l == 0.f;
                const float f = none ? 0.f : 1.f / l;
                uint16_t *out = L.a.o + static_cast<int64_t>(row_out) * D + lane * 2;
#pragma unroll
                for (int v = 0; v < kVec; ++v)
                    *reinterpret_cast<uint32_t *>(out + v * 64) = none ? 0u : pack2<kHalf>(acc[v].x * f, acc[v].y * f);
            }
        }
    }
}

// Zeroes the item counter.  The attention kernel starts beside it and waits for
// it before its blocks take a second item; a memory-set node in its place costs
// 4 us more.
__global__ void reset_kernel(unsigned long long *counter) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    *counter = 0;
}

template <int D, bool kHalf, bool kTree>
cudaError_t launch_d(const AttentionLaunch &L, int64_t items, cudaStream_t stream) {
    static int set[kMaxDevices] = {};
    int dev = 0, sms = 0;
    if (!current_device(&dev, &sms)) return cudaErrorInvalidDevice;
    cudaError_t e;
    if (dev < 0 || dev >= kMaxDevices || !__atomic_load_n(&set[dev], __ATOMIC_ACQUIRE)) {
        e = cudaFuncSetAttribute(attention_kernel<D, kHalf, kTree>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(Shape<D>::kSmem));
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < kMaxDevices) __atomic_store_n(&set[dev], 1, __ATOMIC_RELEASE);
    }
    // A kernel whose launch may overlap the end of the one before; each waits for that where it has to.
    cudaLaunchAttribute overlap[1];
    overlap[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    overlap[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = overlap;
    cfg.gridDim = dim3(static_cast<unsigned>(items < sms ? (items > 0 ? items : 1) : sms));
    cfg.blockDim = dim3(Shape<D>::kThreads);
    cfg.dynamicSmemBytes = Shape<D>::kSmem;
    if (L.ws.counter) {
        reset_kernel<<<1, 1, 0, stream>>>(L.ws.counter);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        cfg.numAttrs = 1;
    }
    e = cudaLaunchKernelEx(&cfg, attention_kernel<D, kHalf, kTree>, L);
    if (e != cudaSuccess || !L.ws.o) return e;
    const int64_t joins = L.a.num_tokens * L.a.h_q, most = int64_t{sms} * kJoinBlocksPerSm;
    cfg.gridDim = dim3(static_cast<unsigned>(joins < most ? joins : most));
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_kernel<D, kHalf>, L);
}

template <bool kTree>
cudaError_t launch_attention(const PagedAttentionArgs &a, cudaStream_t stream) {
    const gdn_paged_cache_t &c = a.cache;
    AttentionLaunch L = {};
    L.a = a;
    L.group = a.h_q / c.h_kv;
    L.tile_tokens = kRows / L.group;
    L.few_splits = few_splits_of(c.h_kv);
    L.box_rows = kKeys;
    while (c.page_size % L.box_rows != 0) L.box_rows /= 2;
    L.o_32 = (reinterpret_cast<uintptr_t>(a.o) & 31u) == 0;
    // A scale of zero weighs all keys alike; the least one keeps masked scores at minus infinity (0 x inf is NaN).
    L.c = fmaxf(a.scale * 1.4426950408889634f, 1e-30f);
    L.ws = workspace_at(a.workspace, a.h_q, c.h_kv, c.d, a.num_reqs, a.num_tokens, a.max_kv_len);
    const cuuint64_t d = static_cast<cuuint64_t>(c.d);
    const cuuint64_t q_dims[3] = {d, static_cast<cuuint64_t>(a.h_q), static_cast<cuuint64_t>(a.num_tokens)};
    const cuuint64_t q_strides[2] = {d * 2, static_cast<cuuint64_t>(a.q_token_stride) * 2};
    const cuuint32_t tile_tokens = static_cast<cuuint32_t>(L.tile_tokens);
    const cuuint32_t q_box[3] = {64, static_cast<uint32_t>(L.group), tile_tokens}, q_one[3] = {64, q_box[1], 1};
    const cuuint64_t dims[4] = {d, static_cast<cuuint64_t>(c.page_size), static_cast<cuuint64_t>(c.h_kv),
                              static_cast<cuuint64_t>(c.num_pages)};
    auto bytes = [](int64_t s) { return static_cast<cuuint64_t>(s) * 2; };
    const cuuint64_t k_strides[3] = {bytes(c.k_slot_stride), bytes(c.k_head_stride), bytes(c.k_page_stride)};
    const cuuint64_t v_strides[3] = {bytes(c.v_slot_stride), bytes(c.v_head_stride), bytes(c.v_page_stride)};
    const cuuint32_t box[4] = {64, static_cast<uint32_t>(L.box_rows), 1, 1};
    // (with so few tokens no item takes the full tile's box)
    const bool no_full = a.num_tokens < L.tile_tokens && a.num_tokens * (c.d / 64) <= 32;
    if (!encode_tiles(&L.tm_q_one, a.q, c.dtype, 3, q_dims, q_strides, q_one) ||
        (!no_full && !encode_tiles(&L.tm_q, a.q, c.dtype, 3, q_dims, q_strides, q_box)) ||
        !encode_tiles(&L.tm_k, c.k, c.dtype, 4, dims, k_strides, box) ||
        !encode_tiles(&L.tm_v, c.v, c.dtype, 4, dims, v_strides, box))
        return cudaErrorNotSupported;
    if (no_full) L.tm_q = L.tm_q_one;
    const int64_t items = items_bound(L.group, c.d, c.h_kv, a.num_reqs, a.num_tokens, a.max_kv_len);
    const bool half = c.dtype == GDN_FP16;
    switch (c.d) {
        case 64: return half ? launch_d<64, true, kTree>(L, items, stream) : launch_d<64, false, kTree>(L, items, stream);
        case 128: return half ? launch_d<128, true, kTree>(L, items, stream) : launch_d<128, false, kTree>(L, items, stream);
        default: return half ? launch_d<256, true, kTree>(L, items, stream) : launch_d<256, false, kTree>(L, items, stream);
    }
}

}  // namespace
}  // namespace gdn
