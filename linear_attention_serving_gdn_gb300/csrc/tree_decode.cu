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
//     C[u][w] = b_w (E(w,u) q_u.k_w - sum_{x between w and u} C[u][x] E(w,x) k_x.k_w)
// with E(w,x) the product of the decays from x up to before w.
//
// One block per (request, value head), a warp per 16 rows of S^T (values).
//   1. Each warp asks for its rows of the state; q, k, v to shared memory.
//   2. K K^T and Q K^T on the tensor cores (mma.sync, bf16: exact products).
//   3. Each node's quad walks its path: decays into those products, then C.
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

namespace gdn {
namespace {

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

__device__ __forceinline__ float4 load_state(const float *p) {
    float4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ bool finite(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }

// Sizes for up to NT * 8 nodes.
template <int D, int NT>
struct TreeShape {
    static constexpr int kThreads = 2 * D;  // a warp per 16 values
    static constexpr int kNodes = 8 * NT;
    static constexpr int kCols = kNodes < 16 ? 16 : kNodes;  // whole steps of 16
    static constexpr int kRowK = 2 * D + 64;                 // bytes of a row of k or q: 16-byte reads of 8 rows x 4 lanes meet no bank twice
    static constexpr int kRowV = 2 * D + 16;
    static constexpr int kRowF = kCols + 1;                  // floats
    static constexpr int kRowC = 2 * kCols + 16;             // bytes
    static constexpr int kGroups = D / 32;                   // of 32 state columns
    static constexpr int kAhead = NT <= 2 ? kGroups : 2;     // groups of the state in registers
    static constexpr int kK = 0, kQ = kK + kCols * kRowK, kV = kQ + kCols * kRowK, kFK = kV + kNodes * kRowV;
    static constexpr int kFQ = kFK + kCols * kRowF * 4, kC = kFQ + kCols * kRowF * 4, kCLo = kC + kNodes * kRowC;
    static constexpr int kWord = kCLo + kNodes * kRowC, kGate = kWord + kNodes * 8;
    static constexpr int kSmem = kGate + 3 * kNodes * 4;
};

// The bf16 products of tile rows [16 rt, 16 rt + 16) of `rows` and [8 ct, 8 ct + 8) of `cols`, into out[row][col].
template <int D, int NT>
__device__ __forceinline__ void products(const uint8_t *rows, const uint8_t *cols, int rt, int ct, float *out, int lane) {
    using Sh = TreeShape<D, NT>;
    const int r = lane >> 2, c = lane & 3;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int g = 0; g < Sh::kGroups; ++g) {
        const uint4 a0 = *reinterpret_cast<const uint4 *>(rows + (rt * 16 + r) * Sh::kRowK + g * 64 + c * 16);
        const uint4 a1 = *reinterpret_cast<const uint4 *>(rows + (rt * 16 + r + 8) * Sh::kRowK + g * 64 + c * 16);
        const uint4 b = *reinterpret_cast<const uint4 *>(cols + (ct * 8 + r) * Sh::kRowK + g * 64 + c * 16);
        const uint32_t f0[4] = {a0.x, a1.x, a0.y, a1.y}, f1[4] = {a0.z, a1.z, a0.w, a1.w};
        mma(acc, f0, b.x, b.y);
        mma(acc, f1, b.z, b.w);
    }
    float *p = out + (rt * 16 + r) * Sh::kRowF + ct * 8 + 2 * c;
    p[0] = acc[0];
    p[1] = acc[1];
    p[8 * Sh::kRowF] = acc[2];
    p[8 * Sh::kRowF + 1] = acc[3];
}

template <int D, int NT>
__global__ void __launch_bounds__(TreeShape<D, NT>::kThreads, 256 / D) tree_decode_kernel(const TreeDecodeArgs a) {
    using Sh = TreeShape<D, NT>;
    extern __shared__ __align__(16) uint8_t smem[];
    uint8_t *const sk = smem + Sh::kK, *const sq = smem + Sh::kQ, *const sv = smem + Sh::kV;
    float *const fk = reinterpret_cast<float *>(smem + Sh::kFK), *const fq = reinterpret_cast<float *>(smem + Sh::kFQ);
    uint8_t *const chi = smem + Sh::kC, *const clo = smem + Sh::kCLo;
    uint64_t *const word = reinterpret_cast<uint64_t *>(smem + Sh::kWord);
    float *const alpha = reinterpret_cast<float *>(smem + Sh::kGate), *const beta = alpha + Sh::kNodes, *const gamma = beta + Sh::kNodes;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, c = lane & 3;
    const int32_t req = blockIdx.x / a.h_v, head = blockIdx.x - req * a.h_v, head_k = head / (a.h_v / a.h_k);

    // Tokens behind the last request's: zeros, dealt out over the blocks.
    int32_t end = a.cu_seqlens[a.num_rows];
    if (end < 0 || end > a.num_tokens) end = static_cast<int32_t>(a.num_tokens);
    {
        const int64_t pieces = static_cast<int64_t>(a.h_v) * (D / 8);
        for (int64_t i = end * pieces + static_cast<int64_t>(blockIdx.x) * Sh::kThreads + tid; i < a.num_tokens * pieces;
             i += static_cast<int64_t>(gridDim.x) * Sh::kThreads)
            reinterpret_cast<uint4 *>(a.o)[i] = make_uint4(0, 0, 0, 0);
    }
    const int32_t b = a.cu_seqlens[req], e = a.cu_seqlens[req + 1], slot = a.src_slot[req];
    const bool range = b >= 0 && b <= e && e <= end;
    if (!range) {
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

    // 1. The state's rows 16 warp + r and + 8, in groups of 32 columns: 8 neighbouring columns a lane.
    const float *const s_row = a.state + ((static_cast<int64_t>(slot) * a.h_v + head) * D + warp * 16 + r) * D + c * 8;
    float4 s[Sh::kAhead][4];
    auto ask = [&](int g) {
        float4(&x)[4] = s[g % Sh::kAhead];
        x[0] = load_state(s_row + g * 32);
        x[1] = load_state(s_row + g * 32 + 4);
        x[2] = load_state(s_row + g * 32 + 8 * D);
        x[3] = load_state(s_row + g * 32 + 8 * D + 4);
    };
#pragma unroll
    for (int g = 0; g < Sh::kAhead; ++g) ask(g);
    for (int i = tid; i < Sh::kCols * (D / 8); i += Sh::kThreads) {
        const int u = i / (D / 8), piece = i % (D / 8);
        uint4 k = make_uint4(0, 0, 0, 0), q = k, v = k;
        if (u < m) {
            const int64_t at = static_cast<int64_t>(b) + u;
            k = __ldg(reinterpret_cast<const uint4 *>(a.k + (at * a.h_k + head_k) * D) + piece);
            q = __ldg(reinterpret_cast<const uint4 *>(a.q + (at * a.h_k + head_k) * D) + piece);
            v = __ldg(reinterpret_cast<const uint4 *>(a.v + (at * a.h_v + head) * D) + piece);
        }
        *reinterpret_cast<uint4 *>(sk + u * Sh::kRowK + piece * 16) = k;
        *reinterpret_cast<uint4 *>(sq + u * Sh::kRowK + piece * 16) = q;
        if (u < Sh::kNodes) *reinterpret_cast<uint4 *>(sv + u * Sh::kRowV + piece * 16) = v;
    }
    for (int u = tid; u < Sh::kNodes; u += Sh::kThreads) {
        const int64_t at = static_cast<int64_t>(b) + u;
        word[u] = u < m ? a.masks[at] & ((2ull << u) - 1) : 0;  // (a node's path: itself and nodes before it)
        alpha[u] = u < m ? expf(a.g[at * a.h_v + head]) : 0.f;
        beta[u] = u < m ? a.beta[at * a.h_v + head] : 0.f;
    }
    __syncthreads();

    // 2. k.k and q.k of nodes and those before them.
    {
        const int row_tiles = (m + 15) / 16;
        int task = warp;
        for (int rt = 0; rt < row_tiles; ++rt) {
            const int col_tiles = 2 * rt + 2 < NT ? 2 * rt + 2 : NT;
            for (; task < 2 * col_tiles; task += D / 16)
                if (task & 1)
                    products<D, NT>(sq, sk, rt, task >> 1, fq, lane);
                else
                    products<D, NT>(sk, sk, rt, task >> 1, fk, lane);
            task -= 2 * col_tiles;
        }
    }
    __syncthreads();

    // 3. A quad per node.  First the decays between a node and those above it.
    const int quad = tid >> 2;
    constexpr int kQuads = Sh::kThreads / 4;
    for (int u = quad; u < Sh::kNodes; u += kQuads) {
        float decay = 1.f;
        for (uint64_t left = word[u]; left; ) {
            const int w = 63 - __clzll(static_cast<long long>(left));
            left ^= 1ull << w;
            if ((w & 3) == c) {
                fk[u * Sh::kRowF + w] *= decay;
                fq[u * Sh::kRowF + w] *= decay;
            }
            decay *= alpha[w];
        }
        if (c == 0) gamma[u] = decay;
    }
    __syncthreads();
    // Then C, over q.k; a lane sums every fourth node below w on the path.
    for (int u = quad; u < Sh::kNodes; u += kQuads) {
        const uint64_t path = word[u];
        float *const row = fq + u * Sh::kRowF;
        const int steps = __reduce_max_sync(0xffffffffu, __popcll(path));
        uint64_t left = path;
        for (int i = 0; i < steps; ++i) {
            const int w = left ? 63 - __clzll(static_cast<long long>(left)) : 0;
            const bool on = left != 0;
            left &= ~(1ull << w);
            float sum = 0.f;
            if (on)
                for (uint64_t x = path & ~((2ull << w) - 1) & (0x1111111111111111ull << c); x; x &= x - 1) {
                    const int j = __ffsll(static_cast<long long>(x)) - 1;
                    sum = fmaf(row[j], fk[j * Sh::kRowF + w], sum);
                }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            if (on && c == 0) row[w] = beta[w] * (row[w] - sum);
            __syncwarp();
        }
        // As sums of two bf16; zeros off the path.
        for (int w = 2 * c; w < Sh::kCols; w += 8) {
            const float x = path >> w & 1 ? row[w] : 0.f, y = path >> w & 2 ? row[w + 1] : 0.f;
            uint32_t hi, lo;
            split2(x, y, &hi, &lo);
            *reinterpret_cast<uint32_t *>(chi + u * Sh::kRowC + w * 2) = hi;
            *reinterpret_cast<uint32_t *>(clo + u * Sh::kRowC + w * 2) = lo;
        }
    }
    __syncthreads();

    // 4. S^T [K; Q]: this warp's 16 values by the nodes.
    float y[NT][4], o[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) y[t][i] = o[t][i] = 0.f;
#pragma unroll
    for (int g = 0; g < Sh::kGroups; ++g) {
        const float4(&x)[4] = s[g % Sh::kAhead];
        uint32_t hi[2][4], lo[2][4];
        split2(x[0].x, x[0].y, &hi[0][0], &lo[0][0]);
        split2(x[0].z, x[0].w, &hi[0][2], &lo[0][2]);
        split2(x[1].x, x[1].y, &hi[1][0], &lo[1][0]);
        split2(x[1].z, x[1].w, &hi[1][2], &lo[1][2]);
        split2(x[2].x, x[2].y, &hi[0][1], &lo[0][1]);
        split2(x[2].z, x[2].w, &hi[0][3], &lo[0][3]);
        split2(x[3].x, x[3].y, &hi[1][1], &lo[1][1]);
        split2(x[3].z, x[3].w, &hi[1][3], &lo[1][3]);
        if (g + Sh::kAhead < Sh::kGroups) ask(g + Sh::kAhead);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (t * 8 >= m) break;
            const uint4 k = *reinterpret_cast<const uint4 *>(sk + (t * 8 + r) * Sh::kRowK + g * 64 + c * 16);
            const uint4 q = *reinterpret_cast<const uint4 *>(sq + (t * 8 + r) * Sh::kRowK + g * 64 + c * 16);
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

    // 5. R in y (elements 0, 1: value row r, nodes 2c and 2c + 1 of the tile; 2, 3: value row r + 8), G o in o.
    const uint16_t *const v16 = reinterpret_cast<const uint16_t *>(sv);
    constexpr int kRowV16 = Sh::kRowV / 2;
    bool bad = false;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int u = t * 8 + 2 * c + (i & 1), row = warp * 16 + r + (i & 2) * 4;
            const float g = gamma[u];
            y[t][i] = u < m ? fmaf(-g, y[t][i], bf16_bits_to_float(v16[u * kRowV16 + row])) : 0.f;
            o[t][i] *= g;
            bad |= !finite(y[t][i]);
        }
    bad = __any_sync(0xffffffffu, bad);
#pragma unroll
    for (int kt = 0; kt < (NT + 1) / 2; ++kt) {
        if (kt * 16 >= m) break;
        uint32_t hi[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (2 * kt + j < NT) {
                float x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = bad && !finite(y[2 * kt + j][i]) ? 0.f : y[2 * kt + j][i];
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
    if (bad) {  // what the product left out, to the nodes whose path it is on
#pragma unroll
        for (int t = 0; t < NT; ++t)
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
                        const int u = t2 * 8 + 2 * c + (i & 1);
                        const float x = i & 2 ? x1 : x0;
                        if (!finite(x) && (word[u] >> w & 1)) o[t2][i] = fmaf(fq[u * Sh::kRowF + w], x, o[t2][i]);
                    }
            }
    }
    // Through shared memory, over v: each lane writes where it alone has read.
    uint16_t *const o16 = reinterpret_cast<uint16_t *>(sv);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o16[(t * 8 + 2 * c + (i & 1)) * kRowV16 + warp * 16 + r + (i & 2) * 4] = float_to_bf16_bits(o[t][i] * a.scale);
    __syncthreads();
    for (int i = tid; i < m * (D / 8); i += Sh::kThreads) {
        const int u = i / (D / 8), piece = i % (D / 8);
        reinterpret_cast<uint4 *>(a.o + ((static_cast<int64_t>(b) + u) * a.h_v + head) * D)[piece] =
            *reinterpret_cast<const uint4 *>(sv + u * Sh::kRowV + piece * 16);
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
