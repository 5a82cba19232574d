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
//   1. Each warp asks for its rows of the state; q, k to shared memory.
//   2. K K^T and Q K^T on the tensor cores (mma.sync, bf16: exact products).
//   3. A thread per node walks its path, on numbers in shared memory: C and G.
//      (Paths of more than 16 nodes by four lanes each.)
//   4. S^T [K; Q] with the state's rows as the A operand, each value as the sum
//      of two bf16 (2^-15 of it is left at most), straight from registers: the state is
//      read once and never staged.
//   5. R = v - G S^T k in the accumulator's layout, which is the A layout of
//      the last product: O^T += R^T C^T, both as sums of two bf16.
// mma.sync and not tcgen05: with up to 32 nodes the products take less time
// than the state's 64 KB, and the state goes through no shared memory.
//
// A node's bits depend on its own path and the state alone.  A value that is
// not finite stays with the nodes whose path it is on: it is left out of the
// last product and added to those alone.
#include "gdn_internal.cuh"
#include "tc_ptx.cuh"

#ifndef GDN_WAIT_CYCLES
#define GDN_WAIT_CYCLES 2000000000LL  // about a second; under 2^32
#endif

namespace gdn {
namespace {

constexpr uint32_t kWaitCycles = GDN_WAIT_CYCLES;
constexpr long long kDrainCycles = 2000000000LL;

// D += A B, 16 x 8 x 16, bf16 with fp32 accumulators.
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// x and y as sums of two bf16: the upper halves cut off, and the rest rounded.
__device__ __forceinline__ void split2(float x, float y, uint32_t *hi, uint32_t *lo) {
    const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
    *hi = __byte_perm(a, b, 0x7632);
    *lo = pack_bf16(x - __uint_as_float(a & 0xffff0000u), y - __uint_as_float(b & 0xffff0000u));
}

// 16 bytes from global to shared memory, or zeros.
__device__ __forceinline__ void copy16(uint32_t to, const void *from, bool some) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(some ? 16 : 0) : "memory");
}

template <int kBytes>
__device__ __forceinline__ void copy_small(uint32_t to, const void *from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(kBytes) : "memory");
}

__device__ __forceinline__ bool finite(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }

// The transpose of an 8 x 8 matrix of 16-bit elements, row lane / 4, columns 2 (lane % 4) and the next.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Sizes for up to NT * 8 nodes.
template <int D, int NT>
struct TreeShape {
    static constexpr int kNodes = 8 * NT;
    static constexpr int kCols = kNodes < 16 ? 16 : kNodes;  // whole steps of 16
    static constexpr int kGroups = D / 32;                   // of 32 state columns
    static constexpr int kSlabs = D / 16;                    // of 16 values
    // Warps: state loader, input loader, kPrep for C, kMain for the products with the state.
    static constexpr int kWarps = 16, kMain = NT <= 4 ? 12 : 8, kPrep = kWarps - kMain - 2;
    static constexpr int kRowK = 2 * D;           // bytes of a row of k or q
    static constexpr int kRowF = kCols + 1;       // floats
    static constexpr int kRowC = 2 * kCols + 16;  // bytes
    static constexpr int kSlot = 16 * 4 * D;      // bytes of a slab, which lie together in the state as they do in the ring
    // A unit's inputs, and what is made of them.
    static constexpr int kQ = kCols * kRowK, kC = 2 * kQ, kCLo = kC + kNodes * kRowC, kWord = kCLo + kNodes * kRowC;
    static constexpr int kG = kWord + 8 * kNodes, kBeta = kG + 4 * kNodes, kGamma = kBeta + 4 * kNodes;
    static constexpr int kBuffer = kGamma + 4 * kNodes;
    static constexpr int kBuffers = NT <= 2 ? 4 : NT <= 4 ? 3 : 2;
    // k.k and q.k of the unit whose C is made, and its decays.
    static constexpr int kFK = kBuffers * kBuffer, kFQ = kFK + kCols * kRowF * 4, kAlpha = kFQ + kCols * kRowF * 4;
    static constexpr int kControl = (kAlpha + kNodes * 4 + 15) / 16 * 16, kControlBytes = 1024;
    // The ring of slabs lies before all that.
    static constexpr int kFit = (227 * 1024 - kControl - kControlBytes) / kSlot;
    static constexpr int kSlots = kFit < 20 ? kFit : 20;
    static constexpr int kSmem = kSlots * kSlot + kControl + kControlBytes;
};

// What a block works on: a request's value head.
struct Unit {
    int32_t b, m, head;  // first token, nodes (0: the end)
    int32_t slot;
};

template <int D, int NT>
struct TreeControl {
    uint64_t in_full[TreeShape<D, NT>::kBuffers], in_empty[TreeShape<D, NT>::kBuffers], c_full[TreeShape<D, NT>::kBuffers];
    uint64_t full[TreeShape<D, NT>::kSlots], empty[TreeShape<D, NT>::kSlots];
    Unit unit[TreeShape<D, NT>::kBuffers];
    int fail;
    int refused;  // some unit of this block has no outputs but zeros
};

// Bounded wait of a whole warp: true for all lanes or for none.  Gives up as soon as any thread has flagged a failure,
// and flags one when it runs out.
struct TreeWait {
    volatile int *fail;
    static __device__ __forceinline__ bool poll(uint64_t *bar, uint32_t parity) {
        return __all_sync(0xffffffffu, kWaitCycles < 10000 ? tc::mbar_test_wait(bar, parity) : tc::mbar_try_wait(bar, parity));
    }
    __device__ __forceinline__ bool operator()(uint64_t *bar, uint32_t parity) const {
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
};

// A block's units, every gridDim.x-th; the lengths and slot of the one behind the last taken are asked for in time.
struct Units {
    const TreeDecodeArgs &a;
    uint32_t next, count;
    int32_t end;  // of the tokens that requests may have
    int32_t b, e, slot;
    __device__ __forceinline__ void look() {
        if (next >= count) return;
        const uint32_t req = next / static_cast<uint32_t>(a.h_v);
        b = a.cu_seqlens[req];
        e = a.cu_seqlens[req + 1];
        slot = a.src_slot[req];
    }
    __device__ __forceinline__ explicit Units(const TreeDecodeArgs &args) : a(args), next(blockIdx.x), b(0), e(0), slot(0) {
        count = static_cast<uint32_t>(a.num_rows) * static_cast<uint32_t>(a.h_v);  // (under 2^31)
        end = a.cu_seqlens[a.num_rows];
        if (end < 0 || end > a.num_tokens) end = static_cast<int32_t>(a.num_tokens);
        look();
    }
    __device__ __forceinline__ bool sound() const { return b >= 0 && b <= e && e <= end; }
    // A padded row, or one that cannot be served.
    __device__ __forceinline__ bool refused() const { return slot < 0 || slot >= a.num_slots || e - b > a.max_nodes; }
    // The next one with something to compute; `skip` is called for those that have not.
    template <typename Skip>
    __device__ __forceinline__ Unit take(Skip skip) {
        Unit u = {0, 0, 0, 0};
#pragma unroll 1
        while (next < count && u.m == 0) {
            const int32_t head = static_cast<int32_t>(next % static_cast<uint32_t>(a.h_v));
            if (!sound() || (e > b && refused()))
                skip(head);
            else
                u = {b, e - b, head, slot};
            next += gridDim.x;
            look();
        }
        return u;
    }
};

// Offset of a 16-byte piece of a row of k or q: odd rows have the halves of each 128 bytes changed over, so that eight
// lanes that read four pieces of two neighbouring rows meet no bank twice.
template <int D>
__device__ __forceinline__ int piece_at(int row, int piece) {
    return row * (2 * D) + ((piece ^ ((row & 1) << 2)) << 4);
}

// k.k and q.k of nodes [16 rt, + 16) with nodes [16 ct, + 16), exact products of bf16.
template <int D, int NT>
__device__ __forceinline__ void products(const uint8_t *sk, const uint8_t *sq, int rt, int ct, float *fk, float *fq, int lane) {
    using Sh = TreeShape<D, NT>;
    constexpr int kTiles = NT == 1 ? 1 : 2;
    const int r = lane >> 2, c = lane & 3;
    float acc[2][kTiles][4] = {};
#pragma unroll
    for (int g = 0; g < Sh::kGroups; ++g) {
        uint4 b[kTiles];
#pragma unroll
        for (int t = 0; t < kTiles; ++t) b[t] = *reinterpret_cast<const uint4 *>(sk + piece_at<D>(ct * 16 + t * 8 + r, g * 4 + c));
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const uint8_t *rows = x ? sq : sk;
            const uint4 a0 = *reinterpret_cast<const uint4 *>(rows + piece_at<D>(rt * 16 + r, g * 4 + c));
            const uint4 a1 = *reinterpret_cast<const uint4 *>(rows + piece_at<D>(rt * 16 + r + 8, g * 4 + c));
            const uint32_t f0[4] = {a0.x, a1.x, a0.y, a1.y}, f1[4] = {a0.z, a1.z, a0.w, a1.w};
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                mma(acc[x][t], f0, b[t].x, b[t].y);
                mma(acc[x][t], f1, b[t].z, b[t].w);
            }
        }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            float *p = (x ? fq : fk) + (rt * 16 + r) * Sh::kRowF + ct * 16 + t * 8 + 2 * c;
            p[0] = acc[x][t][0];
            p[1] = acc[x][t][1];
            p[8 * Sh::kRowF] = acc[x][t][2];
            p[8 * Sh::kRowF + 1] = acc[x][t][3];
        }
}

// Node u's walk up its path: row[x] is p.k_x of the nodes x that are still above, first q_u.k_x; node w leaves its c there,
// and p' = a (p - c k_w) changes the others by k_w.k_x.  Gives the product of the decays.  With kLanes = 4 a quad
// takes the nodes above in turn; what one lane has written is another's c four nodes on.
constexpr int kShortPath = 16;
template <int NT, int kLanes>
__device__ __forceinline__ float walk(uint64_t path, float *row, const float *fk, int stride, const float *alpha,
                                      const float *beta, int sub) {
    constexpr uint64_t kMine = kLanes == 1 ? ~0ull : 0x1111111111111111ull;
    const uint32_t quad = kLanes == 1 ? 0 : 0xfu << (threadIdx.x & 28);
    float decay = 1.f;
#pragma unroll 1
    while (path) {
        const int w = NT <= 4 ? 31 - __clz(static_cast<uint32_t>(path)) : 63 - __clzll(static_cast<long long>(path));
        path ^= 1ull << w;
        const float a = alpha[w], c = beta[w] * row[w], ac = -a * c;
        if (kLanes > 1) __syncwarp(quad);
        if (sub == 0) row[w] = c;
        decay *= a;
        const float *const kk = fk + w * stride;
        uint64_t mine = path & (kMine << sub);
#pragma unroll 1
        while (mine) {
            int x[4];
            float y[4], z[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // (past the last one: it again)
                if (NT <= 4) {
                    const uint32_t b = static_cast<uint32_t>(mine);
                    x[i] = b ? __ffs(static_cast<int>(b)) - 1 : x[i > 0 ? i - 1 : 0];
                    mine = b & (b - 1);
                } else {
                    x[i] = mine ? __ffsll(static_cast<long long>(mine)) - 1 : x[i > 0 ? i - 1 : 0];
                    mine &= mine - 1;
                }
                y[i] = row[x[i]];
                z[i] = kk[x[i]];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) row[x[i]] = fmaf(ac, z[i], a * y[i]);
        }
        if (kLanes > 1) __syncwarp(quad);
    }
    return decay;
}

// ---- the loader of the state -----------------------------------------------------

template <int D, int NT>
__device__ void load_states(const TreeDecodeArgs &a, TreeControl<D, NT> *ctl, uint8_t *ring, const TreeWait &wait) {
    using Sh = TreeShape<D, NT>;
    const int lane = threadIdx.x & 31;
    Units units(a);
    uint32_t q = 0;  // slabs asked for
    bool ok = true;
    while (ok) {
        const Unit u = units.take([](int32_t) {});
        if (u.m == 0) break;
        const float *const from = a.state + (static_cast<int64_t>(u.slot) * a.h_v + u.head) * (D * D);
#pragma unroll 1
        for (int slab = 0; slab < Sh::kSlabs; ++slab, ++q) {
            const uint32_t at = q % Sh::kSlots;
            ok = wait(ctl->empty + at, (q / Sh::kSlots & 1) ^ 1);
            if (!ok) break;
            if (lane == 0) {
                tc::mbar_expect_tx(ctl->full + at, Sh::kSlot);
                tc::bulk_load(tc::smem_u32(ring + at * Sh::kSlot), from + slab * (16 * D), Sh::kSlot, ctl->full + at);
            }
            __syncwarp();
        }
    }
    if (static_cast<uint32_t>(lane) < Sh::kSlots && static_cast<uint32_t>(lane) < q) {  // copies in flight land before the block leaves
        const uint32_t last = q - 1 - (q - 1 - lane) % Sh::kSlots;  // into slot `lane`
        const long long start = clock64();
        while (!tc::mbar_try_wait(ctl->full + lane, last / Sh::kSlots & 1) && clock64() - start < kDrainCycles) {}
    }
    __syncwarp();
}

// ---- the loader of the inputs ------------------------------------------------------

template <int D, int NT>
__device__ void load_inputs(const TreeDecodeArgs &a, TreeControl<D, NT> *ctl, uint8_t *smem, const TreeWait &wait) {
    using Sh = TreeShape<D, NT>;
    const int lane = threadIdx.x & 31;
    const int32_t ratio = a.h_v / a.h_k;
    Units units(a);
    for (uint32_t n = 0;; ++n) {
        const Unit u = units.take([&](int32_t head) {
            if (lane > 0) return;
            if (!units.sound()) {
                if (head == 0) report(a.dev_status, GDN_DEV_BAD_LENGTH);
                return;
            }
            ctl->refused = 1;
            if (head == 0 && units.slot >= a.num_slots) report(a.dev_status, GDN_DEV_BAD_SLOT);
            if (head == 0 && units.e - units.b > a.max_nodes) report(a.dev_status, GDN_DEV_BAD_LENGTH);
        });
        const uint32_t x = n % Sh::kBuffers;
        if (!wait(ctl->in_empty + x, (n / Sh::kBuffers & 1) ^ 1)) break;
        uint8_t *const to = smem + x * Sh::kBuffer;
        if (lane == 0) {
            ctl->unit[x] = u;
            tc::mbar_arrive(ctl->in_full + x);
        }
        __syncwarp();
        if (u.m > 0) {
            constexpr int kPieces = D / 8;
            const int row = lane / kPieces, piece = lane % kPieces;
            const int64_t step = static_cast<int64_t>(a.h_k) * D;
            const uint16_t *k = a.k + ((static_cast<int64_t>(u.b) + row) * a.h_k + u.head / ratio) * D + piece * 8;
            const uint16_t *q = a.q + (k - a.k);
            const uint32_t at = tc::smem_u32(to);
#pragma unroll 4
            for (int i = row; i < ((u.m + 15) & ~15); i += 32 / kPieces, k += step * (32 / kPieces), q += step * (32 / kPieces)) {
                copy16(at + piece_at<D>(i, piece), i < u.m ? k : a.k, i < u.m);
                copy16(at + Sh::kQ + piece_at<D>(i, piece), i < u.m ? q : a.q, i < u.m);
            }
            for (int i = lane; i < u.m; i += 32) {
                const int64_t t = static_cast<int64_t>(u.b) + i;
                copy_small<8>(at + Sh::kWord + i * 8, a.masks + t);
                copy_small<4>(at + Sh::kG + i * 4, a.g + t * a.h_v + u.head);
                copy_small<4>(at + Sh::kBeta + i * 4, a.beta + t * a.h_v + u.head);
                tc::bulk_prefetch_l2(a.v + (t * a.h_v + u.head) * D, 2 * D);
            }
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::smem_u32(ctl->in_full + x)) : "memory");
        if (u.m == 0) break;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// ---- the warps that make C -------------------------------------------------------------

template <int D, int NT>
__device__ void make_c(TreeControl<D, NT> *ctl, uint8_t *smem, const TreeWait &wait, int warp) {
    using Sh = TreeShape<D, NT>;
    constexpr int kThreads = Sh::kPrep * 32;
    const int lane = threadIdx.x & 31, tid = warp * 32 + lane;
    float *const fk = reinterpret_cast<float *>(smem + Sh::kFK), *const fq = reinterpret_cast<float *>(smem + Sh::kFQ);
    float *const alpha = reinterpret_cast<float *>(smem + Sh::kAlpha);
    auto meet = [] { asm volatile("barrier.cta.sync 1, %0;" ::"n"(kThreads) : "memory"); };
    // The same, and whether any warp is on its way out: then all are.
    auto leave = [](bool out) {
        uint32_t any;
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
            : "=r"(any)
            : "r"(static_cast<uint32_t>(out)), "n"(kThreads)
            : "memory");
        return any != 0;
    };
    for (uint32_t n = 0;; ++n) {
        const uint32_t x = n % Sh::kBuffers;
        const int32_t m = wait(ctl->in_full + x, n / Sh::kBuffers & 1) ? ctl->unit[x].m : 0;
        if (m == 0) {
            leave(true);
            return;
        }
        uint8_t *const in = smem + x * Sh::kBuffer;
        uint64_t *const word = reinterpret_cast<uint64_t *>(in + Sh::kWord);
        float *const beta = reinterpret_cast<float *>(in + Sh::kBeta), *const gamma = reinterpret_cast<float *>(in + Sh::kGamma);
        for (int u = tid; u < Sh::kNodes; u += kThreads) {
            word[u] = u < m ? word[u] & ((2ull << u) - 1) : 0;  // (itself and nodes before it)
            alpha[u] = u < m ? expf(reinterpret_cast<const float *>(in + Sh::kG)[u]) : 0.f;
        }
        int task = warp;
#pragma unroll 1
        for (int rt = 0; rt * 16 < m; ++rt) {
#pragma unroll 1
            for (; task <= rt; task += Sh::kPrep) products<D, NT>(in, in + Sh::kQ, rt, task, fk, fq, lane);
            task -= rt + 1;
        }
        if (leave(false)) return;
        bool deep = false;
        for (int u = lane; u < Sh::kNodes; u += 32) deep |= __popcll(word[u]) > kShortPath;
        if (!__any_sync(0xffffffffu, deep)) {
            for (int u = tid; u < Sh::kNodes; u += kThreads)
                gamma[u] = u < m ? walk<NT, 1>(word[u], fq + u * Sh::kRowF, fk, Sh::kRowF, alpha, beta, 0) : 0.f;
        } else {
#pragma unroll 1
            for (int u = tid >> 2; u < Sh::kNodes; u += kThreads / 4) {  // (whole quads: one node's lanes stay together)
                const float g = u < m ? walk<NT, 4>(word[u], fq + u * Sh::kRowF, fk, Sh::kRowF, alpha, beta, lane & 3) : 0.f;
                if ((lane & 3) == 0) gamma[u] = g;
            }
        }
        meet();
        // As sums of two bf16; zeros off the path.
        constexpr int kPairs = Sh::kCols / 2;
#pragma unroll 1
        for (int i = tid; i < Sh::kNodes * kPairs; i += kThreads) {
            const int u = i / kPairs, w = i % kPairs * 2;
            const uint64_t on = word[u];
            uint32_t hi, lo;
            split2(on >> w & 1 ? fq[u * Sh::kRowF + w] : 0.f, on >> w & 2 ? fq[u * Sh::kRowF + w + 1] : 0.f, &hi, &lo);
            *reinterpret_cast<uint32_t *>(in + Sh::kC + u * Sh::kRowC + w * 2) = hi;
            *reinterpret_cast<uint32_t *>(in + Sh::kCLo + u * Sh::kRowC + w * 2) = lo;
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(ctl->c_full + x);
        meet();  // the products are not written again before all are done with them
    }
}

// ---- the warps of the products with the state ----------------------------------------------

template <int D, int NT>
__device__ void multiply(const TreeDecodeArgs &a, TreeControl<D, NT> *ctl, uint8_t *smem, uint8_t *ring, const TreeWait &wait, int warp) {
    using Sh = TreeShape<D, NT>;
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    uint32_t q = warp;  // this warp's next slab, of all the block's
    for (uint32_t n = 0;; ++n) {
        const uint32_t buffer = n % Sh::kBuffers;
        if (!wait(ctl->in_full + buffer, n / Sh::kBuffers & 1)) return;
        const Unit unit = ctl->unit[buffer];
        if (unit.m == 0) return;
        const int32_t m = unit.m;
        const uint8_t *const sk = smem + buffer * Sh::kBuffer, *const sq = sk + Sh::kQ;
        const uint64_t *const word = reinterpret_cast<const uint64_t *>(sk + Sh::kWord);
        const float *const gamma = reinterpret_cast<const float *>(sk + Sh::kGamma);
#pragma unroll 1
        for (; q < (n + 1) * Sh::kSlabs; q += Sh::kMain) {
            const uint32_t slab = q - n * Sh::kSlabs, slot = q % Sh::kSlots;
            const int64_t value = (static_cast<int64_t>(unit.b) * a.h_v + unit.head) * D + slab * 16;  // node 0's first of the slab
            // v of node 8 t + r, values 2c and 2c + 1, and 8 further on.
            uint32_t v[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                v[t][0] = v[t][1] = 0;
                if (t * 8 + r < m) {
                    const uint32_t *p = reinterpret_cast<const uint32_t *>(a.v + value + static_cast<int64_t>(t * 8 + r) * a.h_v * D) + c;
                    v[t][0] = __ldg(p);
                    v[t][1] = __ldg(p + 4);
                }
            }
            if (!wait(ctl->full + slot, q / Sh::kSlots & 1)) return;
            // S^T [K; Q]: 16 values by the nodes.
            const float *const rows = reinterpret_cast<const float *>(ring + slot * Sh::kSlot) + r * D + c * 8;
            float y[NT][4], o[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) y[t][i] = o[t][i] = 0.f;
#pragma unroll
            for (int g = 0; g < Sh::kGroups; ++g) {
                const float4 x0 = *reinterpret_cast<const float4 *>(rows + g * 32), x1 = *reinterpret_cast<const float4 *>(rows + g * 32 + 4);
                const float4 x2 = *reinterpret_cast<const float4 *>(rows + g * 32 + 8 * D), x3 = *reinterpret_cast<const float4 *>(rows + g * 32 + 8 * D + 4);
                uint32_t hi[2][4], lo[2][4];
                split2(x0.x, x0.y, &hi[0][0], &lo[0][0]);
                split2(x0.z, x0.w, &hi[0][2], &lo[0][2]);
                split2(x1.x, x1.y, &hi[1][0], &lo[1][0]);
                split2(x1.z, x1.w, &hi[1][2], &lo[1][2]);
                split2(x2.x, x2.y, &hi[0][1], &lo[0][1]);
                split2(x2.z, x2.w, &hi[0][3], &lo[0][3]);
                split2(x3.x, x3.y, &hi[1][1], &lo[1][1]);
                split2(x3.z, x3.w, &hi[1][3], &lo[1][3]);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    if (t * 8 >= m) break;
                    const uint4 k = *reinterpret_cast<const uint4 *>(sk + piece_at<D>(t * 8 + r, g * 4 + c));
                    const uint4 q = *reinterpret_cast<const uint4 *>(sq + piece_at<D>(t * 8 + r, g * 4 + c));
                    mma(y[t], hi[0], k.x, k.y);
                    mma(o[t], hi[0], q.x, q.y);
                    mma(y[t], lo[0], k.x, k.y);
                    mma(o[t], lo[0], q.x, q.y);
                    mma(y[t], hi[1], k.z, k.w);
                    mma(o[t], hi[1], q.z, q.w);
                    mma(y[t], lo[1], k.z, k.w);
                    mma(o[t], lo[1], q.z, q.w);
                }
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(ctl->empty + slot);
            // R in y (elements 0, 1: value r, nodes 2c and 2c + 1 of the tile; 2, 3: value r + 8), G o in o.
            // (Nodes past the last have k, v and G of zero, so R of zero, or NaN, which is left out.)
            if (!wait(ctl->c_full + buffer, n / Sh::kBuffers & 1)) return;
            float not_zero = 0.f;  // NaN if some R is not finite
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const float2 g = *reinterpret_cast<const float2 *>(gamma + t * 8 + 2 * c);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t vt = transpose8(v[t][i]);
                    y[t][2 * i] = fmaf(-g.x, y[t][2 * i], __uint_as_float(vt << 16));
                    y[t][2 * i + 1] = fmaf(-g.y, y[t][2 * i + 1], __uint_as_float(vt & 0xffff0000u));
                    o[t][2 * i] *= g.x;
                    o[t][2 * i + 1] *= g.y;
                    not_zero = fmaf(y[t][2 * i], 0.f, fmaf(y[t][2 * i + 1], 0.f, not_zero));
                }
            }
            const uint8_t *const chi = sk + Sh::kC, *const clo = sk + Sh::kCLo;
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
                                const int u = t2 * 8 + 2 * c + (i & 1), at = u * Sh::kRowC + w * 2;
                                const float x = i & 2 ? x1 : x0;
                                if (!finite(x) && (word[u] >> w & 1))
                                    o[t2][i] = fmaf(bf16_bits_to_float(*reinterpret_cast<const uint16_t *>(chi + at)) +
                                                        bf16_bits_to_float(*reinterpret_cast<const uint16_t *>(clo + at)),
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
                        split2(x[0], x[1], &hi[2 * j], &lo[2 * j]);
                        split2(x[2], x[3], &hi[2 * j + 1], &lo[2 * j + 1]);
                    }
#pragma unroll
                for (int t = 2 * kt; t < NT; ++t) {
                    if (t * 8 >= m) break;
                    const int at = (t * 8 + r) * Sh::kRowC + kt * 32 + c * 4;
                    const uint32_t h0 = *reinterpret_cast<const uint32_t *>(chi + at), h1 = *reinterpret_cast<const uint32_t *>(chi + at + 16);
                    const uint32_t l0 = *reinterpret_cast<const uint32_t *>(clo + at), l1 = *reinterpret_cast<const uint32_t *>(clo + at + 16);
                    mma(o[t], hi, h0, h1);
                    mma(o[t], hi, l0, l1);
                    mma(o[t], lo, h0, h1);
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (t * 8 >= m) break;
                uint32_t *p = reinterpret_cast<uint32_t *>(a.o + value + static_cast<int64_t>(t * 8 + r) * a.h_v * D) + c;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t x = transpose8(pack_bf16(o[t][2 * i] * a.scale, o[t][2 * i + 1] * a.scale));
                    if (t * 8 + r < m) p[4 * i] = x;
                }
            }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(ctl->in_empty + buffer);
    }
}

template <int D, int NT>
__global__ void __launch_bounds__(TreeShape<D, NT>::kWarps * 32, 1) tree_decode_kernel(const __grid_constant__ TreeDecodeArgs a) {
    using Sh = TreeShape<D, NT>;
    extern __shared__ __align__(128) uint8_t ring[];
    uint8_t *const smem = ring + Sh::kSlots * Sh::kSlot;
    TreeControl<D, NT> *const ctl = reinterpret_cast<TreeControl<D, NT> *>(smem + Sh::kControl);
    static_assert(sizeof(TreeControl<D, NT>) <= Sh::kControlBytes && Sh::kSmem <= 227 * 1024 && Sh::kSlots >= Sh::kMain, "shared memory");
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < Sh::kBuffers; ++i) {
            tc::mbar_init(ctl->in_full + i, 33);  // the loader's copies, and its word on the unit
            tc::mbar_init(ctl->in_empty + i, Sh::kMain);
            tc::mbar_init(ctl->c_full + i, Sh::kPrep);
        }
        for (int i = 0; i < Sh::kSlots; ++i) {
            tc::mbar_init(ctl->full + i, 1);
            tc::mbar_init(ctl->empty + i, 1);
        }
        ctl->fail = 0;
        ctl->refused = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tc::fence_proxy_async_smem();
    __syncthreads();
    const TreeWait wait = {&ctl->fail};
    if (warp >= Sh::kWarps - Sh::kMain) {
        multiply<D, NT>(a, ctl, smem, ring, wait, warp - (Sh::kWarps - Sh::kMain));
    } else {
        if (warp == 0)
            load_states<D, NT>(a, ctl, ring, wait);
        else if (warp == 1)
            load_inputs<D, NT>(a, ctl, smem, wait);
        else
            make_c<D, NT>(ctl, smem, wait, warp - 2);
    }
    __syncthreads();
    if (threadIdx.x == 0 && ctl->fail) report(a.dev_status, GDN_DEV_TIMEOUT);
    // Zeros: the tokens behind the last request's, dealt out over the blocks, and the rows that have no outputs else.
    int32_t end = a.cu_seqlens[a.num_rows];
    if (end < 0 || end > a.num_tokens) end = static_cast<int32_t>(a.num_tokens);
    const int64_t pieces = static_cast<int64_t>(a.h_v) * (D / 8);
    for (int64_t i = end * pieces + static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < a.num_tokens * pieces;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x)
        reinterpret_cast<uint4 *>(a.o)[i] = make_uint4(0, 0, 0, 0);
    if (ctl->refused) {
        Units units(a);
        for (; units.next < units.count; units.next += gridDim.x) {
            units.look();
            if (!units.sound() || !units.refused()) continue;
            const int32_t head = static_cast<int32_t>(units.next % static_cast<uint32_t>(a.h_v));
            for (int64_t i = threadIdx.x; i < static_cast<int64_t>(units.e - units.b) * (D / 8); i += blockDim.x)
                reinterpret_cast<uint4 *>(a.o + ((units.b + i / (D / 8)) * a.h_v + head) * D)[i % (D / 8)] = make_uint4(0, 0, 0, 0);
        }
    }
}

template <int D, int NT>
cudaError_t launch(const TreeDecodeArgs &a, cudaStream_t stream) {
    using Sh = TreeShape<D, NT>;
    static int set[kMaxDevices] = {};
    int dev = 0, sms = 0;
    if (!current_device(&dev, &sms)) return cudaErrorInvalidDevice;
    if (dev < 0 || dev >= kMaxDevices || !__atomic_load_n(&set[dev], __ATOMIC_ACQUIRE)) {
        const cudaError_t e =
            cudaFuncSetAttribute(tree_decode_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < kMaxDevices) __atomic_store_n(&set[dev], 1, __ATOMIC_RELEASE);
    }
    const int64_t units = static_cast<int64_t>(a.num_rows) * a.h_v;
    tree_decode_kernel<D, NT><<<static_cast<unsigned>(units < sms ? units : sms), Sh::kWarps * 32, Sh::kSmem, stream>>>(a);
    return cudaGetLastError();
}

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
