// The gated delta rule along a tree of drafted tokens.
//
// Node u of a request continues the state of its parent (the root nodes that
// of the request's slot, S):
//     S_u = a_u (I - b_u k_u k_u^T) S_parent + b_u k_u v_u^T,   o_u = scale S_u^T q_u
// with a = exp(g), b = beta.  The states of the nodes are never formed: walked
// from u to the root, with p = q_u at first,
//     p^T S_w = c v_w + p'^T S_parent(w),   c = b_w (p.k_w),   p' = a_w (p - c k_w)
// so with G_u the product of the decays on u's path and C[u][w] the c of step w
//     o_u = scale (G_u S^T q_u + sum_w C[u][w] (v_w - G_w S^T k_w)).
// Of the state only S^T [K; Q] is needed, one product of all nodes with it.
// The p.k_w come from the products of keys and queries among each other:
// g_x = p.k_x is q_u.k_x at first, and each node w on the way makes it a_w (g_x - c k_w.k_x).
//
// One block per (request, value head), a warp per 32 rows of S^T (values), 16
// at a time.
//   1. k, q (and v of up to 32 nodes) to shared memory; each warp asks for its
//      first rows of the state.
//   2. K K^T and Q K^T on the tensor cores (mma.sync, bf16: exact products),
//      what lies on or below the diagonal.
//   3. The walks, in registers: C and G.  Short paths place by place, a thread
//      a node; longer ones node by node, several lanes a node.
//   4. S^T [K; Q] with the state's rows as the A operand, each value as the sum
//      of two bf16 (2^-16 of it is left at most), straight from registers: the
//      state is read once and never staged.
//   5. R = v - G S^T k in the accumulator's layout, which is the A layout of
//      the last product: O^T += R^T C^T, both as sums of two bf16, rounded so
//      that 2^-15 of a product is left at most.
//
// What bounds it.  Up to 16 nodes: the state's 64 KB per head.  256 requests of
// 4 to 12 nodes, 16 heads: 303 MB in 53.5 us, 5.7 TB/s, 0.83 of the copy peak,
// the tensor pipe 30 % busy; what is missing are the loads that a block does not
// have in flight while it walks.  With 33 to 64 nodes (64 requests, 32 heads:
// 76 us) a block's phases: 9000 cycles until k and q are there, 4000 for their
// products, 3000 for the walks, 10000 for each slab's product with the state and
// 2500 for the rest of it, four blocks of an SM in turn: the tensor pipe is 46 %
// busy (712 products a warp, 2 cycles each of the SM, are 36 us), the shared
// memory's pipe 55 %, and neither is the bound alone.  One tree: 5.2 us, the
// chain of these phases.  Heads of 64 (out of L2): 256 of 4 to 12 nodes 11 us with
// 8/8 heads, 14 with 4/12; 64 of 33 to 64 nodes 14 and 17.
//
// Why mma.sync and not tcgen05.  Up to 16 nodes the products hide behind the
// state.  A tcgen05 product takes the state as two bf16 operands out of shared
// memory (64 KB a block) or TMEM: two blocks per SM instead of four to seven, and
// one more trip of 64 KB, for a pipe that is not the bound (counted, not measured);
// and with one arithmetic for every size a request's bits do not depend on max_nodes.
//
// Tried and worse (256 small trees / 64 large ones, us, at 61 / 91): blocks that
// take several (request, head) in turn 65 / 98, the state of the next block to
// L2 65 / 91, the block's own state to L2 for up to 16 nodes 63, k and q by 8-byte
// pieces 61 / 97.
//
// A node's bits depend on its word, the nodes on its path and the state alone (on the
// word, since the last product sums over node numbers, 16 at a time).  A value that is
// not finite stays with the nodes whose path it is on: it is left out of the
// last product and added to those alone.
#include "gdn_internal.cuh"

namespace gdn {
namespace {

// D += A B, 16 x 8 x 16, bf16 with fp32 accumulators.
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// x and y as sums of two bf16: the upper halves cut off, and the rest, under 2^-7 of it, rounded: within 2^-16.
__device__ __forceinline__ void split2(float x, float y, uint32_t *hi, uint32_t *lo) {
    const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
    *hi = __byte_perm(a, b, 0x7632);
    *lo = pack_bf16(x - __uint_as_float(a & 0xffff0000u), y - __uint_as_float(b & 0xffff0000u));
}
// The same with the upper halves rounded to the nearest (never up to infinity), so that the rests are at most 2^-8 of the
// number: of a product of two such sums, without that of the rests, 2^-15 is missing at most (cut off 2^-14 and more).
__device__ __forceinline__ void split2_near(float x, float y, uint32_t *hi, uint32_t *lo) {
    asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(*hi) : "f"(y), "f"(x));
    *lo = pack_bf16(x - __uint_as_float(*hi << 16), y - __uint_as_float(*hi & 0xffff0000u));
}

// 16 bytes from global to shared memory, or zeros.
__device__ __forceinline__ void copy16(uint32_t to, const void *from, bool some) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(some ? 16 : 0) : "memory");
}

// 8 values, read once: whole sectors (in 16-byte pieces: 64 large trees 84 us, so 76).
struct Eight {
    float x[8];
};
__device__ __forceinline__ Eight load_state(const float *p) {
    Eight v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v.x[0]), "=f"(v.x[1]), "=f"(v.x[2]), "=f"(v.x[3]), "=f"(v.x[4]), "=f"(v.x[5]), "=f"(v.x[6]), "=f"(v.x[7])
                 : "l"(p));
    return v;
}

__device__ __forceinline__ bool finite(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }

// The transpose of an 8 x 8 matrix of 16-bit elements, row lane / 4, columns 2 (lane % 4) and the next.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// First float of node u's row of k.k, with nodes 0 to u: 16-byte pieces, rows of 4, 4, 4, 4, 8, 8, ... floats.
__host__ __device__ constexpr int key_row(int u) { return 4 * (u / 4 + 1) * (u - 2 * (u / 4)); }

// Sizes for up to NT * 8 nodes.
template <int D, int NT>
struct TreeShape {
    static constexpr int kThreads = D;                         // a warp per 32 values
    // Blocks of an SM (D = 128), and groups of the state that a lane holds in registers, by what these allow without spilling
    // to matter.  Up to 8 nodes six and two (256 trees / one 49.0 / 4.8 us, seven and two 48.6 / 4.9, six and one - / 5.1); up
    // to 16 seven and one (256 trees of 12 to 16 / one of 16: 54.7 / 5.5; six and two 57.3 / 5.6, eight and one 58.0 / 6.1); up
    // to 32 five and one (256 trees of 17 to 20 / one of 24: 75.5 / 6.9; four and two 83 / 6.9, five and two 80 / 8.0, six and
    // one 81 / 8.2); 64 four and one.
    static constexpr int kBlocks = (NT == 1 ? 768 : NT == 2 ? 896 : NT == 4 ? 640 : 512) / D, kAhead = NT == 1 ? 2 : 1;
    static constexpr int kNodes = 8 * NT;
    static constexpr int kCols = kNodes < 16 ? 16 : kNodes;  // whole steps of 16
    // Nodes whose paths a warp walks: at least 8 where they may be long, so that four lanes at most have one.
    static constexpr int kPer = NT > 1 && kNodes / (D / 32) < 8 ? 8 : kNodes / (D / 32);
    static constexpr int kGroups = D / 32;                   // of 32 state columns
    static constexpr int kRowK = 2 * D;                      // bytes of a row of k or q
    // Of k.k and q.k only what lies on or below the diagonal: k.k as a triangle (key_row), q.k by tiles of 16 (struct Row).
    static constexpr int kQ = kCols * kRowK, kFQ = 2 * kQ, kFK = kFQ + (128 * (kCols / 16) * (kCols / 16 + 1) + 64 * (kCols / 16)) * 4,
                         kWord = kFK + key_row(kCols) * 4, kGate = kWord + 8 * kNodes;
    // v; of 64 nodes it is read where it is used, so that four blocks have room.
    static constexpr bool kStageV = NT <= 4;
    static constexpr int kRowV = 2 * D + 16, kV = (kGate + 3 * kNodes * 4 + 15) / 16 * 16;
    static constexpr int kSmem = kV + (kStageV ? kNodes * kRowV : 0);
};

// Offset of a 16-byte piece of a row of k or q: odd rows have the halves of each 128 bytes changed over, so that eight
// lanes that read four pieces of two neighbouring rows meet no bank twice.
template <int D>
__device__ __forceinline__ int piece_at(int row, int piece) {
    return row * (2 * D) + ((piece ^ ((row & 1) << 2)) << 4);
}

// Node u's row of q.k: as many floats as there are nodes up to the end of its tile of 16, and 4 more (4-byte reads of 8 rows
// x 4 lanes meet no bank twice).  Its row of C takes that place: the upper halves, then the rests.
struct Row {
    int at, cols;  // first float; nodes
    __device__ __forceinline__ explicit Row(int u) : at(128 * (u / 16) * (u / 16 + 1) + 64 * (u / 16) + u % 16 * (16 * (u / 16) + 20)), cols(16 * (u / 16) + 16) {}
    __device__ __forceinline__ int lo() const { return 2 * cols; }  // bytes from the upper halves to the rests
};

// k.k and q.k of nodes [16 rt, + 16) with nodes [16 ct, + 16), exact products of bf16.  With few nodes a warp takes one of
// them for 8 nodes (part: q.k, second 8), so that four share what there is to do.
template <int D, int NT, int kParts>
__device__ __forceinline__ void products(const uint8_t *sk, const uint8_t *sq, int rt, int ct, int part, float *fk, float *fq, int lane) {
    using Sh = TreeShape<D, NT>;
    constexpr int kTiles = NT == 1 || kParts > 1 ? 1 : 2, kSides = kParts > 1 ? 1 : 2;
    const int r = lane >> 2, c = lane & 3, side0 = kParts > 1 ? part & 1 : 0, tile0 = kParts > 1 ? part >> 1 : 0;
    float acc[kSides][kTiles][4] = {};
#pragma unroll
    for (int g = 0; g < Sh::kGroups; ++g) {
        uint4 b[kTiles];
        uint32_t f[kSides][2][4];
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
            b[t] = *reinterpret_cast<const uint4 *>(sk + piece_at<D>(ct * 16 + (tile0 + t) * 8 + r, g * 4 + c));
#pragma unroll
        for (int x = 0; x < kSides; ++x) {
            const uint8_t *rows = side0 + x ? sq : sk;
            const uint4 a0 = *reinterpret_cast<const uint4 *>(rows + piece_at<D>(rt * 16 + r, g * 4 + c));
            const uint4 a1 = *reinterpret_cast<const uint4 *>(rows + piece_at<D>(rt * 16 + r + 8, g * 4 + c));
            f[x][0][0] = a0.x, f[x][0][1] = a1.x, f[x][0][2] = a0.y, f[x][0][3] = a1.y;
            f[x][1][0] = a0.z, f[x][1][1] = a1.z, f[x][1][2] = a0.w, f[x][1][3] = a1.w;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int x = 0; x < kSides; ++x)
#pragma unroll
                for (int t = 0; t < kTiles; ++t) mma(acc[x][t], f[x][h], h ? b[t].z : b[t].x, h ? b[t].w : b[t].y);
    }
#pragma unroll
    for (int x = 0; x < kSides; ++x)
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            const int u = rt * 16 + r, w = ct * 16 + (tile0 + t) * 8 + 2 * c;
            if (side0 + x) {
                *reinterpret_cast<float2 *>(fq + Row(u).at + w) = make_float2(acc[x][t][0], acc[x][t][1]);
                *reinterpret_cast<float2 *>(fq + Row(u + 8).at + w) = make_float2(acc[x][t][2], acc[x][t][3]);
            } else {
                if (w <= u) fk[key_row(u) + w] = acc[x][t][0];
                if (w + 1 <= u) fk[key_row(u) + w + 1] = acc[x][t][1];
                if (w <= u + 8) fk[key_row(u + 8) + w] = acc[x][t][2];
                if (w + 1 <= u + 8) fk[key_row(u + 8) + w + 1] = acc[x][t][3];
            }
        }
}

// Node u's walk up its path.  g_x is p.k_x of the nodes x that are still above, first q_u.k_x (in `row`); node w's c is
// b_w g_w, and p' = a_w (p - c k_w) changes the others by k_w.k_x.  C[u] takes the row's place, as sums of two bf16, zeros
// off the path.  Gives the product of the decays.
//
// Of up to kShortPath nodes the walk is held in registers, place by place, a thread a node.  (41 requests of 15 to 26 nodes
// in a chain, 32 heads: with up to 16 nodes so 39 us, 10 32.8, 8 and 6 31.9; trees 29.7, and 32 with none so.  256 chains of 12
// to 16: with 16 66.8, 8 58.4.)
constexpr int kShortPath = 8;

template <int D, int NT>
__device__ __forceinline__ float walk_short(uint64_t path, int most, float *row, int cols, const float *fk, const float2 *gates) {
    using Sh = TreeShape<D, NT>;
    constexpr int kMost = kShortPath;
    const int steps = __popcll(path);
    int x[kMost];
    float g[kMost];
#pragma unroll
    for (int i = 0; i < kMost; ++i) {  // (behind the last one: it again)
        if (i >= most) break;  // (the warp's longest)
        const int w = NT <= 4 ? 31 - __clz(static_cast<uint32_t>(path)) : 63 - __clzll(static_cast<long long>(path));
        x[i] = path ? w : i > 0 ? x[i > 0 ? i - 1 : 0] : 0;
        path &= ~(1ull << x[i]);
        g[i] = row[x[i]];
    }
    asm volatile("" ::: "memory");  // (the row is read as floats, then written as other types)
#pragma unroll
    for (int i = 0; i < Sh::kCols / 4; ++i)
        if (4 * i < cols) reinterpret_cast<uint4 *>(row)[i] = make_uint4(0, 0, 0, 0);
    asm volatile("" ::: "memory");
    uint16_t *const hi = reinterpret_cast<uint16_t *>(row), *const lo = hi + cols;
    float decay = 1.f;
    float2 ab = most > 0 ? gates[x[0]] : make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
        if (i >= most) break;
        const float a = ab.x, c = ab.y * g[i], ac = -a * c;
        const float *const kk = fk + key_row(x[i]);  // (places behind the last: any number)
        if (i + 1 < kMost && i + 1 < most) ab = gates[x[i + 1 < kMost ? i + 1 : i]];
#pragma unroll
        for (int j = i + 1; j < kMost; ++j) {
            if (j >= most) break;
            g[j] = fmaf(ac, kk[x[j]], a * g[j]);
        }
        if (i < steps) {
            uint32_t h, l;
            split2_near(c, 0.f, &h, &l);
            hi[x[i]] = static_cast<uint16_t>(h);
            lo[x[i]] = static_cast<uint16_t>(l);
            decay *= a;
        }
    }
    return decay;
}

// Paths of any length, of a pass of 16 nodes or the warp's, each with 32 / pass lanes: node by node from the last to the
// first, so that k.k is read by whole lines for all nodes whose path the node is on.  A node's lanes hold its g_x in turns
// of four neighbouring nodes x, those behind the current ones shifted down.  The same operations, and so the same bits.
// (A quad a node, each with its own place and its numbers in shared memory: a chain of 64 nodes 71 us, 64 of them with 32
// heads 248; so 19 and 100.)
constexpr int pass_of(int per) { return per < 16 ? per : 16; }

template <int D, int NT>
__device__ __forceinline__ void walk_long(int first, int m, const uint64_t *word, float *fq, const float *fk, const float2 *gates,
                                          float *gamma, int lane) {
    using Sh = TreeShape<D, NT>;
    constexpr int kSplit = 32 / pass_of(Sh::kPer), kSteps = 4 * kSplit, kTurns = Sh::kNodes / kSteps;
    const int u = first + lane / kSplit, sub = lane % kSplit;
    const Row at(u);
    float *const row = fq + at.at;
    const uint64_t path = u < m ? word[u] : 0;
    const uint64_t all = static_cast<uint64_t>(__reduce_or_sync(0xffffffffu, static_cast<uint32_t>(path >> 32))) << 32 |
                         __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(path));
    int b = all ? (63 - __clzll(static_cast<long long>(all))) / kSteps : -1;
    float g[kTurns][4];  // of nodes kSteps (b - i) + 4 sub and the next three
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        const int x = (b - i) * kSteps + 4 * sub;
        const float4 v = i <= b && x < at.cols ? *reinterpret_cast<const float4 *>(row + x) : make_float4(0.f, 0.f, 0.f, 0.f);
        g[i][0] = v.x, g[i][1] = v.y, g[i][2] = v.z, g[i][3] = v.w;
    }
    asm volatile("" ::: "memory");  // (the row is read as floats, then written as other types)
    __syncwarp();
#pragma unroll
    for (int i = 0; i < Sh::kCols / 4; i += kSplit)
        if (4 * (i + sub) < at.cols) reinterpret_cast<uint4 *>(row)[i + sub] = make_uint4(0, 0, 0, 0);
    __syncwarp();
    asm volatile("" ::: "memory");
    float decay = 1.f;
#pragma unroll 1
    for (; b >= 0; --b) {
        float mine[4] = {0.f, 0.f, 0.f, 0.f};  // c of the lane's own four nodes
#pragma unroll
        for (int j = kSteps - 1; j >= 0; --j) {
            const int w = b * kSteps + j;
            if (!(all >> w & 1)) continue;
            const float2 ab = gates[w];
            const float *const kk = fk + key_row(w) + b * kSteps + 4 * sub;  // (of nodes from w on: any number)
            constexpr int kFirst = kTurns < 4 ? kTurns : 4;  // lines asked for before c is there
            float4 z[kFirst];
#pragma unroll
            for (int i = 0; i < kFirst; ++i) z[i] = *reinterpret_cast<const float4 *>(kk - (i <= b ? i : 0) * kSteps);
            const float a = ab.x, c = ab.y * __shfl_sync(0xffffffffu, g[0][j % 4], (lane & -kSplit) | j / 4), ac = -a * c;
            if (!(path >> w & 1)) continue;
            if (sub == j / 4) mine[j % 4] = c;
            decay *= a;
#pragma unroll
            for (int i = 0; i < kTurns; ++i) {
                if (i >= kFirst && i % 2 == 0 && i > b) break;
                const float4 y = i < kFirst ? z[i < kFirst ? i : 0] : *reinterpret_cast<const float4 *>(kk - (i <= b ? i : 0) * kSteps);
                g[i][0] = fmaf(ac, y.x, a * g[i][0]);
                g[i][1] = fmaf(ac, y.y, a * g[i][1]);
                g[i][2] = fmaf(ac, y.z, a * g[i][2]);
                g[i][3] = fmaf(ac, y.w, a * g[i][3]);
            }
        }
        const int x = b * kSteps + 4 * sub;
        if (x < at.cols) {
            uint2 h, l;
            split2_near(mine[0], mine[1], &h.x, &l.x);
            split2_near(mine[2], mine[3], &h.y, &l.y);
            *reinterpret_cast<uint2 *>(row + x / 2) = h;
            *reinterpret_cast<uint2 *>(row + x / 2 + at.cols / 2) = l;
        }
#pragma unroll
        for (int i = 0; i + 1 < kTurns; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) g[i][j] = g[i + 1][j];
    }
    if (sub == 0) gamma[u] = decay;
}

template <int D, int NT>
__global__ void __launch_bounds__(TreeShape<D, NT>::kThreads, TreeShape<D, NT>::kBlocks) tree_decode_kernel(const __grid_constant__ TreeDecodeArgs a) {
    using Sh = TreeShape<D, NT>;
    extern __shared__ __align__(16) uint8_t smem[];
    uint8_t *const sk = smem, *const sq = smem + Sh::kQ;
    float *const fk = reinterpret_cast<float *>(smem + Sh::kFK), *const fq = reinterpret_cast<float *>(smem + Sh::kFQ);
    const uint8_t *const rows = smem + Sh::kFQ;  // of C
    uint64_t *const word = reinterpret_cast<uint64_t *>(smem + Sh::kWord);
    float2 *const gates = reinterpret_cast<float2 *>(smem + Sh::kGate);  // decay and beta
    float *const gamma = reinterpret_cast<float *>(gates + Sh::kNodes);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, c = lane & 3;
    const int32_t req = blockIdx.x / a.h_v, head = blockIdx.x - req * a.h_v, head_k = head / (a.h_v / a.h_k);
    const int32_t b = a.cu_seqlens[req], e = a.cu_seqlens[req + 1], slot = a.src_slot[req];
    int32_t end = a.cu_seqlens[a.num_rows];
    if (end < 0 || end > a.num_tokens) end = static_cast<int32_t>(a.num_tokens);
    // Tokens behind the last request's: zeros, dealt out over the blocks.
    if (end < a.num_tokens) {
        const int64_t pieces = static_cast<int64_t>(a.h_v) * (D / 8);
        for (int64_t i = end * pieces + static_cast<int64_t>(blockIdx.x) * Sh::kThreads + tid; i < a.num_tokens * pieces;
             i += static_cast<int64_t>(gridDim.x) * Sh::kThreads)
            reinterpret_cast<uint4 *>(a.o)[i] = make_uint4(0, 0, 0, 0);
    }
    if (b < 0 || b > e || e > end) {
        if (tid == 0 && head == 0) report(a.dev_status, GDN_DEV_BAD_LENGTH);
        return;
    }
    const int32_t m = e - b;
    if (m == 0) return;
    if (slot < 0 || slot >= a.num_slots || m > a.max_nodes) {  // a padded row, or one that cannot be served
        if (tid == 0 && head == 0 && slot >= a.num_slots) report(a.dev_status, GDN_DEV_BAD_SLOT);
        if (tid == 0 && head == 0 && m > a.max_nodes) report(a.dev_status, GDN_DEV_BAD_LENGTH);
        for (int64_t i = tid; i < static_cast<int64_t>(m) * (D / 8); i += Sh::kThreads)
            reinterpret_cast<uint4 *>(a.o + ((b + i / (D / 8)) * a.h_v + head) * D)[i % (D / 8)] = make_uint4(0, 0, 0, 0);
        return;
    }

    // 1. The state's rows, of 16 those that make row r of a product's tile and row r + 8, in groups of 32 columns: 8
    // neighbouring columns a lane.  Rows 2c, 2c + 1, 2c + 8 and 2c + 9 of a tile are values 4c to 4c + 3, so that a lane has
    // four neighbouring values of v and o.
    const float *const s_row =
        a.state + ((static_cast<int64_t>(slot) * a.h_v + head) * D + warp * 32 + (r >> 1) * 4 + (r & 1)) * D + c * 8;
    Eight s[Sh::kAhead][2];
    auto ask = [&](int g) {  // group g, counted over both 16 rows
        const float *p = s_row + (g / Sh::kGroups) * (16 * D) + (g % Sh::kGroups) * 32;
        s[g % Sh::kAhead][0] = load_state(p);
        s[g % Sh::kAhead][1] = load_state(p + 2 * D);
    };
    // (k and q first, which the block waits for; the state's rows are there when it comes to them.)
    uint64_t path = 0;  // of node tid, as long as there is one (itself and nodes before it)
    float my_g = 0.f, my_beta = 0.f;
    if (tid < m) {
        const int64_t at = static_cast<int64_t>(b) + tid;
        path = a.masks[at] & ((2ull << tid) - 1);
        my_g = a.g[at * a.h_v + head];
        my_beta = a.beta[at * a.h_v + head];
    }
    {
        // (each thread's rows are 8 apart, so their parity and the piece's place stay)
        const int row = tid / (D / 8), piece = tid % (D / 8);
        const int64_t first = ((static_cast<int64_t>(b) + row) * a.h_k + head_k) * D + piece * 8, step = static_cast<int64_t>(8) * a.h_k * D;
        uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(sk + piece_at<D>(row, piece)));
        const uint16_t *k = a.k + first, *q = a.q + first;
#pragma unroll 2
        for (int u = row; u < ((m + 15) & ~15); u += 8, k += step, q += step, to += 8 * Sh::kRowK) {
            copy16(to, u < m ? k : a.k, u < m);
            copy16(to + Sh::kQ, u < m ? q : a.q, u < m);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (Sh::kStageV) {
            const uint16_t *v = a.v + ((static_cast<int64_t>(b) + row) * a.h_v + head) * D + piece * 8;
            to = static_cast<uint32_t>(__cvta_generic_to_shared(smem + Sh::kV + row * Sh::kRowV + piece * 16));
#pragma unroll 2
            for (int u = row; u < m; u += 8, v += static_cast<int64_t>(8) * a.h_v * D, to += 8 * Sh::kRowV) copy16(to, v, true);
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    }
#pragma unroll
    for (int g = 0; g < Sh::kAhead; ++g) ask(g);
    if (NT > 4) {  // the walks are long: the rest of the state waits in L2 (64 large trees 91 -> 84 us; up to 32 nodes no change)
        const float *p = a.state + (static_cast<int64_t>(slot) * a.h_v + head) * (D * D) + tid * 64;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + i * (64 * Sh::kThreads)));
    }
    if (tid < Sh::kNodes) {
        word[tid] = path;
        gates[tid] = make_float2(expf(my_g), my_beta);
    }
    if (Sh::kStageV)
        asm volatile("cp.async.wait_group 1;" ::: "memory");
    else
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();

    // 2. k.k and q.k of nodes and those before them.
    if (NT <= 2) {
#pragma unroll 1
        for (int part = warp; part < 2 * NT; part += D / 32) products<D, NT, 4>(sk, sq, 0, 0, part, fk, fq, lane);
    } else {
        int task = warp;
#pragma unroll 1
        for (int rt = 0; rt * 16 < m; ++rt) {
#pragma unroll 1
            for (; task <= rt; task += D / 32) products<D, NT, 1>(sk, sq, rt, task, 0, fk, fq, lane);
            task -= rt + 1;
        }
    }
    if (Sh::kStageV) asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();

    // 3. C and G, the nodes dealt out over the warps.
    if (warp * Sh::kPer < Sh::kNodes) {
        const int first = warp * Sh::kPer, u = first + lane;
        const bool mine = lane < Sh::kPer && u < m;
        path = mine ? word[u] : 0;
        const int most = __reduce_max_sync(0xffffffffu, __popcll(path));
        if (NT == 1 || most <= kShortPath) {
            float g = 0.f;
            if (mine) g = walk_short<D, NT>(path, most, fq + Row(u).at, Row(u).cols, fk, gates);
            if (lane < Sh::kPer) gamma[u] = g;
        } else if constexpr (NT > 1) {
#pragma unroll 1
            for (int i = 0; i < Sh::kPer; i += pass_of(Sh::kPer)) walk_long<D, NT>(first + i, m, word, fq, fk, gates, gamma, lane);
        }
    }
    __syncthreads();

#pragma unroll 1
    for (int slab = 0; slab < 2; ++slab) {
        const int64_t value = (static_cast<int64_t>(b) * a.h_v + head) * D + warp * 32 + slab * 16;  // node 0's first of the slab
        // S^T [K; Q]: 16 values by the nodes.
        float y[NT][4], o[NT][4];
        uint2 v[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) y[t][i] = o[t][i] = 0.f;
#pragma unroll
        for (int g = 0; g < Sh::kGroups; ++g) {
            const Eight(&x)[2] = s[g % Sh::kAhead];
            if (g == Sh::kGroups - 1) {  // v of node 8 t + r, values 4c to 4c + 3
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    v[t] = make_uint2(0, 0);
                    if (t * 8 + r < m)
                        v[t] = Sh::kStageV ? *reinterpret_cast<const uint2 *>(smem + Sh::kV + (t * 8 + r) * Sh::kRowV + warp * 64 + slab * 32 + c * 8)
                                           : __ldg(reinterpret_cast<const uint2 *>(a.v + value + static_cast<int64_t>(t * 8 + r) * a.h_v * D + c * 4));
                }
            }
            uint32_t hi[2][4], lo[2][4];  // of columns 0 to 3 and 4 to 7; element 2 j + i: row r + 8 i, columns 2 j and 2 j + 1 of them
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) split2(x[i & 1].x[4 * h + (i & 2)], x[i & 1].x[4 * h + (i & 2) + 1], &hi[h][i], &lo[h][i]);
            // The group after those in registers.
            if (slab == 0)
                ask(g + Sh::kAhead);
            else if (g + Sh::kAhead < Sh::kGroups)
                ask(Sh::kGroups + g + Sh::kAhead);
            // Two tiles at a time: four sums that do not wait for one another.
            constexpr int kStep = NT == 1 ? 1 : 2;
#pragma unroll
            for (int t0 = 0; t0 < NT; t0 += kStep) {
                if (t0 * 8 >= m) break;
                uint4 kq[2][kStep];
#pragma unroll
                for (int t = 0; t < kStep; ++t) {
                    kq[0][t] = *reinterpret_cast<const uint4 *>(sk + piece_at<D>((t0 + t) * 8 + r, g * 4 + c));
                    kq[1][t] = *reinterpret_cast<const uint4 *>(sq + piece_at<D>((t0 + t) * 8 + r, g * 4 + c));
                }
#pragma unroll
                for (int h = 0; h < 4; ++h)
#pragma unroll
                    for (int t = 0; t < kStep; ++t) {
                        if (t > 0 && (t0 + t) * 8 >= m) continue;
                        const uint32_t(&f)[4] = h & 1 ? lo[h >> 1] : hi[h >> 1];
                        mma(y[t0 + t], f, h & 2 ? kq[0][t].z : kq[0][t].x, h & 2 ? kq[0][t].w : kq[0][t].y);
                        mma(o[t0 + t], f, h & 2 ? kq[1][t].z : kq[1][t].x, h & 2 ? kq[1][t].w : kq[1][t].y);
                    }
            }
        }
        // R in y (elements 0, 1: row r, nodes 2c and 2c + 1 of the tile; 2, 3: row r + 8), G o in o.
        // (Nodes past the last have k, v and G of zero, so R of zero, or NaN, which is left out.)
        float not_zero = 0.f;  // NaN if some R is not finite
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const float2 g = *reinterpret_cast<const float2 *>(gamma + t * 8 + 2 * c);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t vt = transpose8(i ? v[t].y : v[t].x);
                y[t][2 * i] = fmaf(-g.x, y[t][2 * i], __uint_as_float(vt << 16));
                y[t][2 * i + 1] = fmaf(-g.y, y[t][2 * i + 1], __uint_as_float(vt & 0xffff0000u));
                o[t][2 * i] *= g.x;
                o[t][2 * i + 1] *= g.y;
                not_zero = fmaf(y[t][2 * i], 0.f, fmaf(y[t][2 * i + 1], 0.f, not_zero));
            }
        }
        if (__any_sync(0xffffffffu, not_zero != 0.f)) {  // what is not finite, to the nodes whose path it is on
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll 1
                for (int j = 0; j < 8 && t * 8 + j < m; ++j) {
                    const int from = (lane & ~3) | j >> 1, w = t * 8 + j;
                    const float x0 = __shfl_sync(0xffffffffu, j & 1 ? y[t][1] : y[t][0], from);
                    const float x1 = __shfl_sync(0xffffffffu, j & 1 ? y[t][3] : y[t][2], from);
                    if (!__any_sync(0xffffffffu, !finite(x0) || !finite(x1))) continue;
#pragma unroll
                    for (int t2 = 0; t2 < NT; ++t2)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int u = t2 * 8 + 2 * c + (i & 1), at = Row(u).at * 4 + w * 2;
                            const float x = i & 2 ? x1 : x0;
                            if (!finite(x) && (word[u] >> w & 1))
                                o[t2][i] = fmaf(bf16_bits_to_float(*reinterpret_cast<const uint16_t *>(rows + at)) +
                                                    bf16_bits_to_float(*reinterpret_cast<const uint16_t *>(rows + at + Row(u).lo())),
                                                x, o[t2][i]);
                        }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (!finite(y[t][i])) y[t][i] = 0.f;
            }
        }
#pragma unroll
        for (int kt = 0; kt < (NT + 1) / 2; ++kt) {
            if (kt * 16 >= m) break;
            uint32_t hi[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (2 * kt + j < NT) {
                    const float(&x)[4] = y[2 * kt + j];
                    split2_near(x[0], x[1], &hi[2 * j], &lo[2 * j]);
                    split2_near(x[2], x[3], &hi[2 * j + 1], &lo[2 * j + 1]);
                }
            constexpr int kStep = NT < 4 ? NT : 4;
#pragma unroll
            for (int t0 = 2 * kt / kStep * kStep; t0 < NT; t0 += kStep) {
                if (t0 * 8 >= m) break;
                uint32_t h[kStep][2], l[kStep][2];
#pragma unroll
                for (int t = 0; t < kStep; ++t) {
                    if (t0 + t < 2 * kt) continue;
                    const Row row(8 * (t0 + t));
                    const uint8_t *const p = rows + row.at * 4 + r * (4 * row.cols + 16) + kt * 32 + c * 4;
                    h[t][0] = *reinterpret_cast<const uint32_t *>(p), h[t][1] = *reinterpret_cast<const uint32_t *>(p + 16);
                    l[t][0] = *reinterpret_cast<const uint32_t *>(p + row.lo()), l[t][1] = *reinterpret_cast<const uint32_t *>(p + row.lo() + 16);
                }
#pragma unroll
                for (int t = 0; t < kStep; ++t)
                    if (t0 + t >= 2 * kt) mma(o[t0 + t], hi, h[t][0], h[t][1]);
#pragma unroll
                for (int t = 0; t < kStep; ++t)
                    if (t0 + t >= 2 * kt) mma(o[t0 + t], hi, l[t][0], l[t][1]);
#pragma unroll
                for (int t = 0; t < kStep; ++t)
                    if (t0 + t >= 2 * kt) mma(o[t0 + t], lo, h[t][0], h[t][1]);
            }
        }
        uint32_t out[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) out[t][i] = transpose8(pack_bf16(o[t][2 * i] * a.scale, o[t][2 * i + 1] * a.scale));
        uint16_t *p = a.o + value + static_cast<int64_t>(r) * a.h_v * D + 4 * c;
        const int64_t step = static_cast<int64_t>(8) * a.h_v * D;
#pragma unroll
        for (int t = 0; t < NT; ++t, p += step)
            if (t * 8 + r < m) *reinterpret_cast<uint2 *>(p) = make_uint2(out[t][0], out[t][1]);
    }
}

template <int D, int NT>
cudaError_t launch(const TreeDecodeArgs &a, cudaStream_t stream) {
    using Sh = TreeShape<D, NT>;
    static int set[kMaxDevices] = {};
    int dev = 0, sms = 0;
    if (!current_device(&dev, &sms)) return cudaErrorInvalidDevice;
    if (Sh::kSmem > 48 * 1024 && (dev < 0 || dev >= kMaxDevices || !__atomic_load_n(&set[dev], __ATOMIC_ACQUIRE))) {
        const cudaError_t e =
            cudaFuncSetAttribute(tree_decode_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < kMaxDevices) __atomic_store_n(&set[dev], 1, __ATOMIC_RELEASE);
    }
    tree_decode_kernel<D, NT><<<static_cast<unsigned>(a.num_rows) * static_cast<unsigned>(a.h_v), Sh::kThreads, Sh::kSmem, stream>>>(a);
    return cudaGetLastError();
}

// By the bound, which is all that the host knows of the rows: small rows beside a large one pay for its form (248 rows of 1
// to 8 nodes, 16 heads: bound 8 48.9 us, 16 51.4, 32 58.3, 64 70.6; with 8 rows of 64 nodes among them 80.4, in two calls
// with bounds of their own 64.2).
template <int D>
cudaError_t launch_d(const TreeDecodeArgs &a, cudaStream_t stream) {
    if (a.max_nodes <= 8) return launch<D, 1>(a, stream);
    if (a.max_nodes <= 16) return launch<D, 2>(a, stream);
    if (a.max_nodes <= 32) return launch<D, 4>(a, stream);
    return launch<D, 8>(a, stream);
}

}  // namespace

cudaError_t launch_tree_decode(const TreeDecodeArgs &a, int d, cudaStream_t stream) {
    return d == 128 ? launch_d<128>(a, stream) : launch_d<64>(a, stream);
}

}  // namespace gdn
