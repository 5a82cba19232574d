// The maps of a step over the paged K/V cache, built on the device from the
// step's request lengths, and the write of the new tokens' keys and values.
//
// maps_kernel.  Everything a request needs from the others is two exclusive
// sums over the requests before it: of new tokens (its first token) and of
// new pages (its first entry of the free list).  The bytes are a few per
// request and eight per token, so the call is bound by latency: one cluster
// of up to 8 blocks runs it in one launch.  Every block scans all requests
// (1024 at a time, one per thread, sums carried in 64 bits), so no block
// waits for another's sums; the tokens and the new table entries of those
// 1024 requests are then dealt out over the cluster's threads, each finding
// its request by bisection in shared memory, so one long prompt among
// thousands of decode rows is still spread over all threads.  The cluster
// barrier orders every block's read of free_head before its update, which
// makes updating it in place sound.
//
// write_kernel.  A copy: 16-byte pieces, K and V in one launch, several
// pieces' loads in flight per thread; bound by HBM for long chunks and by the
// launch for decode steps.
#include "paged.cuh"

#include <limits.h>

namespace gdn {
namespace {

constexpr int kMapThreads = 1024;
constexpr int kMapMaxBlocks = 8;  // portable cluster size

// Exclusive sums of a and b over the block; totals in *ta, *tb.
__device__ __forceinline__ void block_scan2(long long &a, long long &b, long long *ta, long long *tb,
                                            long long (*part)[kMapThreads / 32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long ia = a, ib = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long xa = __shfl_up_sync(0xffffffffu, ia, o), xb = __shfl_up_sync(0xffffffffu, ib, o);
        if (lane >= o) {
            ia += xa;
            ib += xb;
        }
    }
    __syncthreads();  // the previous scan's readers are done with `part`
    if (lane == 31) {
        part[0][warp] = ia;
        part[1][warp] = ib;
    }
    __syncthreads();
    long long pa = part[0][lane], pb = part[1][lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long xa = __shfl_up_sync(0xffffffffu, pa, o), xb = __shfl_up_sync(0xffffffffu, pb, o);
        if (lane >= o) {
            pa += xa;
            pb += xb;
        }
    }
    *ta = __shfl_sync(0xffffffffu, pa, 31);
    *tb = __shfl_sync(0xffffffffu, pb, 31);
    const int before = warp > 0 ? warp - 1 : 0;
    const long long wa = __shfl_sync(0xffffffffu, pa, before), wb = __shfl_sync(0xffffffffu, pb, before);
    a = ia - a + (warp > 0 ? wa : 0);
    b = ib - b + (warp > 0 ? wb : 0);
}

// Last j in [0, n) with first[j] <= x (first is non-decreasing, first[0] <= x).
__device__ __forceinline__ int find_last(const int32_t *first, int n, int32_t x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

__global__ void __launch_bounds__(kMapThreads, 1) maps_kernel(const PagedMapsArgs a) {
    __shared__ int32_t s_tok[kMapThreads];    // first token of each request of the tile
    __shared__ int32_t s_page[kMapThreads];   // first of its new pages among the tile's
    __shared__ int32_t s_ctx[kMapThreads];    // context length, or -1: refused
    __shared__ int32_t s_start[kMapThreads];  // its first entry of the free list
    __shared__ long long s_part[2][kMapThreads / 32];
    __shared__ int32_t s_head;
    const int tid = threadIdx.x;
    const uint32_t rank = blockIdx.x, blocks = gridDim.x;
    const uint32_t P = static_cast<uint32_t>(a.page_size);
    const int64_t cap = a.token_capacity;
    const int32_t head_in = a.free_pages ? *a.free_head : 0;
    cluster_arrive();  // free_head has been read (the value is used below)
    // A negative head offers no page: nothing is known about the list.
    const long long head = head_in < 0 ? a.num_free : head_in;
    if (tid == 0) {
        s_head = head_in;
        if (head_in < 0 && rank == 0) report(a.dev_status, GDN_DEV_BAD_LENGTH);
    }
    long long tok0 = 0, page0 = 0;  // tokens and new pages of the tiles before
    for (int64_t base = 0; base < a.num_reqs; base += kMapThreads) {
        const int64_t i = base + tid;
        const int32_t c = i < a.num_reqs ? a.context_lens[i] : 0, m = i < a.num_reqs ? a.new_lens[i] : 0;
        const long long len = static_cast<long long>(c) + m;
        const long long mm = m > 0 ? m : 0;
        long long tok = mm, unused = 0, tile_tok, tile_page;
        block_scan2(tok, unused, &tile_tok, &tile_page, s_part);
        tok += tok0;
        bool refused = c < 0 || m < 0 || len > INT_MAX || (len + P - 1) / P > a.table_width || tok + mm > cap;
        const uint32_t have = refused ? 0 : (static_cast<uint32_t>(c) + P - 1) / P;
        const uint32_t total = refused ? 0 : static_cast<uint32_t>((len + P - 1) / P);
        const long long need = (refused || !a.free_pages) ? 0 : total - have;
        if (refused && rank == 0) report(a.dev_status, GDN_DEV_BAD_LENGTH);
        long long page = need;
        unused = 0;
        block_scan2(page, unused, &tile_page, &unused, s_part);
        const long long start = head + page0 + page;
        if (need > 0 && start + need > a.num_free) {
            refused = true;
            if (rank == 0) report(a.dev_status, GDN_DEV_NO_PAGES);
        } else if (need > 0 && rank == 0) {
            atomicMax(&s_head, static_cast<int32_t>(start + need));  // the served requests are a prefix
        }
        s_tok[tid] = static_cast<int32_t>(tok < cap ? tok : cap);
        s_page[tid] = static_cast<int32_t>(page);
        s_ctx[tid] = refused ? -1 : c;
        s_start[tid] = static_cast<int32_t>(start < INT_MAX ? start : INT_MAX);
        if (rank == 0 && i < a.num_reqs) {
            a.cu_seqlens[i] = s_tok[tid];
            a.kv_lens[i] = refused ? 0 : static_cast<int32_t>(len);
        }
        __syncthreads();
        // The tile's tokens, then its new table entries, over the cluster.
        const int64_t t0 = tok0 < cap ? tok0 : cap, t1 = tok0 + tile_tok < cap ? tok0 + tile_tok : cap;
        for (int64_t t = t0 + rank * kMapThreads + tid; t < t1; t += blocks * kMapThreads) {
            const int j = find_last(s_tok, kMapThreads, static_cast<int32_t>(t));
            int32_t pos = 0, slot = -1;
            if (s_ctx[j] >= 0) {
                pos = s_ctx[j] + static_cast<int32_t>(t - s_tok[j]);
                const uint32_t idx = static_cast<uint32_t>(pos) / P;
                const uint32_t jh = (static_cast<uint32_t>(s_ctx[j]) + P - 1) / P;
                const int32_t id = (a.free_pages && idx >= jh) ? a.free_pages[s_start[j] + (idx - jh)]
                                                               : a.block_table[(base + j) * a.table_stride + idx];
                if (id >= 0 && id < a.num_pages)
                    slot = id * a.page_size + static_cast<int32_t>(static_cast<uint32_t>(pos) - idx * P);
                else
                    report(a.dev_status, GDN_DEV_BAD_SLOT);
            }
            a.slot_map[t] = slot;
            a.positions[t] = pos;
        }
        for (int64_t e = rank * kMapThreads + tid; e < tile_page; e += blocks * kMapThreads) {
            const int j = find_last(s_page, kMapThreads, static_cast<int32_t>(e));
            if (s_ctx[j] < 0) continue;
            const int32_t k = static_cast<int32_t>(e) - s_page[j];
            const uint32_t jh = (static_cast<uint32_t>(s_ctx[j]) + P - 1) / P;
            a.block_table[(base + j) * a.table_stride + jh + k] = a.free_pages[s_start[j] + k];
        }
        tok0 += tile_tok;
        page0 += tile_page;
        __syncthreads();
    }
    const int64_t end = tok0 < cap ? tok0 : cap;
    for (int64_t t = end + rank * kMapThreads + tid; t < cap; t += blocks * kMapThreads) {
        a.slot_map[t] = -1;
        a.positions[t] = 0;
    }
    cluster_wait();  // every block has read free_head
    if (rank == 0 && tid == 0) {
        a.cu_seqlens[a.num_reqs] = static_cast<int32_t>(end);
        if (a.free_pages) *a.free_head_out = s_head;
    }
}

constexpr int kWriteThreads = 256;
constexpr int kWriteUnroll = 4;

// Piece p of 2 * num_tokens * h * (d / 8): side-major, then token, head, piece of the row.
__global__ void __launch_bounds__(kWriteThreads) write_kernel(const PagedWriteArgs a, uint32_t pieces_log2) {
    const int64_t per_side = a.num_tokens * a.h << pieces_log2;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWriteThreads;
    const PagedWriteSide &s = a.side[blockIdx.y];
    const uint32_t h = static_cast<uint32_t>(a.h), P = static_cast<uint32_t>(a.page_size);
    const int64_t slots = a.num_pages * a.page_size;
    for (int64_t p0 = static_cast<int64_t>(blockIdx.x) * kWriteThreads + threadIdx.x; p0 < per_side;
         p0 += step * kWriteUnroll) {
        uint4 val[kWriteUnroll];
        int64_t to[kWriteUnroll];
#pragma unroll
        for (int u = 0; u < kWriteUnroll; ++u) {
            const int64_t p = p0 + u * step;
            to[u] = -1;
            if (p >= per_side) continue;
            const int64_t row = p >> pieces_log2;
            const int64_t piece = p - (row << pieces_log2);
            const int64_t t = row / h;
            const int64_t head = row - t * h;
            const int32_t slot = a.slot_map[t];
            if (slot < 0) continue;
            if (slot >= slots) {
                report(a.dev_status, GDN_DEV_BAD_SLOT);
                continue;
            }
            val[u] = __ldg(reinterpret_cast<const uint4 *>(s.src + t * s.token_stride + head * s.head_stride) + piece);
            const uint32_t page = static_cast<uint32_t>(slot) / P;
            to[u] = page * s.page_stride + (static_cast<uint32_t>(slot) - page * P) * s.slot_stride +
                    head * s.dst_head_stride + piece * 8;
        }
#pragma unroll
        for (int u = 0; u < kWriteUnroll; ++u)
            if (to[u] >= 0) *reinterpret_cast<uint4 *>(s.dst + to[u]) = val[u];
    }
}

}  // namespace

cudaError_t launch_paged_maps(const PagedMapsArgs &a, cudaStream_t stream) {
    // One block for up to 2048 tokens of capacity, then one more per 2048.
    const int64_t want = (a.token_capacity + 2 * kMapThreads - 1) / (2 * kMapThreads);
    int blocks = 1;
    while (blocks < kMapMaxBlocks && blocks < want) blocks *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kMapThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = blocks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, maps_kernel, a);
}

cudaError_t launch_paged_write(const PagedWriteArgs &a, cudaStream_t stream) {
    int dev = 0, sms = 0;
    if (!current_device(&dev, &sms)) return cudaErrorInvalidDevice;
    static int cache[kMaxDevices] = {};
    const int64_t resident = static_cast<int64_t>(sms) * blocks_per_sm(write_kernel, kWriteThreads, dev, cache);
    uint32_t lg = 0;
    while ((8 << lg) < a.d) ++lg;
    const int64_t pieces = a.num_tokens * a.h << lg;
    // One piece per thread while that fits the resident blocks of one side.
    int64_t blocks = (pieces + kWriteThreads - 1) / kWriteThreads;
    if (blocks > resident / 2) blocks = resident / 2;
    write_kernel<<<dim3(static_cast<unsigned>(blocks), 2), kWriteThreads, 0, stream>>>(a, lg);
    return cudaGetLastError();
}

}  // namespace gdn
