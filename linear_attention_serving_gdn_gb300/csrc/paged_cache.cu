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
// 1024 requests are then dealt out over the cluster's threads, four tokens a
// thread and round, each finding its request by bisection in shared memory, so
// one long prompt among thousands of decode rows is still spread over all
// threads.  The cluster barrier orders every block's read of free_head before
// its update, which makes updating it in place sound.  Measured: 8 rows 4.9
// us, 1000 rows and 24 chunks (61 thousand tokens) 9.7 us (12.9 us with one
// token a thread), both in a replayed graph.
//
// write_kernel.  A copy: 16-byte pieces, K and V in one launch, four pieces'
// loads in flight per thread; bound by HBM for long chunks and by the launch
// for decode steps.  Measured: 32768 tokens of 8 x 128 43.1 us (6.2 TB/s, 0.92
// of the copy peak; 50.7 us with 64-bit index arithmetic per piece), 256
// tokens of 2 x 256 2.7 us.
#include "paged.cuh"

#include <limits.h>

namespace gdn {
namespace {

constexpr int kMapThreads = 1024;
constexpr int kMapMaxBlocks = 8;  // portable cluster size

// Exclusive sum of x over the block; the total in *total.
__device__ __forceinline__ long long block_scan(long long x, long long *total, long long *part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long sum = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
    }
    if (lane == 31) part[warp] = sum;
    __syncthreads();
    long long p = lane < static_cast<int>(blockDim.x / 32) ? part[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, p, o);
        if (lane >= o) p += y;
    }
    *total = __shfl_sync(0xffffffffu, p, 31);
    const long long before = __shfl_sync(0xffffffffu, p, warp > 0 ? warp - 1 : 0);
    return sum - x + (warp > 0 ? before : 0);
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
    __shared__ int32_t s_tok[kMapThreads + 1];  // first token of each request of the tile; the end
    __shared__ int32_t s_page[kMapThreads];     // first of its new pages among the tile's
    __shared__ int32_t s_ctx[kMapThreads];      // context length, or -1: refused
    __shared__ int32_t s_start[kMapThreads];    // its first entry of the free list
    __shared__ long long s_part[2][32];
    __shared__ int32_t s_head;
    const int tid = threadIdx.x, threads = blockDim.x;
    const uint32_t rank = blockIdx.x, blocks = gridDim.x;
    const uint32_t P = static_cast<uint32_t>(a.page_size);
    const int64_t cap = a.token_capacity;
    // The first tile's lengths are on their way while free_head is read.
    int32_t c = tid < a.num_reqs ? a.context_lens[tid] : 0, m = tid < a.num_reqs ? a.new_lens[tid] : 0;
    const int32_t head_in = a.free_pages ? *a.free_head : 0;
    if (blocks > 1) cluster_arrive();  // free_head has been read (the value is used below)
    // A negative head offers no page: nothing is known about the list.
    const long long head = head_in < 0 ? a.num_free : head_in;
    if (tid == 0) {
        s_head = head_in;
        if (head_in < 0 && rank == 0) report(a.dev_status, GDN_DEV_BAD_LENGTH);
    }
    long long tok0 = 0, page0 = 0;  // tokens and new pages of the tiles before
    for (int64_t base = 0; base < a.num_reqs; base += threads) {
        const int64_t i = base + tid;
        if (base > 0) {
            c = i < a.num_reqs ? a.context_lens[i] : 0;
            m = i < a.num_reqs ? a.new_lens[i] : 0;
        }
        const long long len = static_cast<long long>(c) + m;
        const long long mm = m > 0 ? m : 0;
        long long tile_tok, tile_page;
        const long long tok = tok0 + block_scan(mm, &tile_tok, s_part[0]);
        bool refused = c < 0 || m < 0 || len > INT_MAX || (len + P - 1) / P > a.table_width || tok + mm > cap;
        const uint32_t have = refused ? 0 : (static_cast<uint32_t>(c) + P - 1) / P;
        const uint32_t total = refused ? 0 : (static_cast<uint32_t>(len) + P - 1) / P;
        const long long need = (refused || !a.free_pages) ? 0 : total - have;
        if (refused && rank == 0) report(a.dev_status, GDN_DEV_BAD_LENGTH);
        const long long page = block_scan(need, &tile_page, s_part[1]);
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
        // The tile's tokens, four per thread and round, then its new table entries, over the cluster.
        const int64_t t0 = tok0 < cap ? tok0 : cap, t1 = tok0 + tile_tok < cap ? tok0 + tile_tok : cap;
        if (tid == 0) s_tok[threads] = static_cast<int32_t>(t1);
        __syncthreads();
        for (int64_t g = t0 / 4 + rank * threads + tid; g * 4 < t1; g += blocks * threads) {
            int32_t slot[4], where[4];
            const int64_t first = g * 4 < t0 ? t0 : g * 4;  // (a tile need not start at a multiple of four)
            int j = find_last(s_tok, threads, static_cast<int32_t>(first));
            uint32_t idx = 0, row = 0;  // page of the request and row of the token before
            int32_t id = 0;
            bool fresh = true;  // no page at hand
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t t = g * 4 + k;
                slot[k] = -1;
                where[k] = 0;
                if (t < t0 || t >= t1) continue;
                while (s_tok[j + 1] <= t) {
                    ++j;
                    fresh = true;
                }
                if (s_ctx[j] < 0) continue;
                where[k] = s_ctx[j] + static_cast<int32_t>(t - s_tok[j]);
                if (fresh) {
                    idx = static_cast<uint32_t>(where[k]) / P;
                    row = static_cast<uint32_t>(where[k]) - idx * P;
                } else if (++row == P) {
                    row = 0;
                    ++idx;
                    fresh = true;
                }
                if (fresh) {
                    const uint32_t jh = (static_cast<uint32_t>(s_ctx[j]) + P - 1) / P;
                    id = (a.free_pages && idx >= jh) ? a.free_pages[s_start[j] + (idx - jh)]
                                                     : a.block_table[(base + j) * a.table_stride + idx];
                    fresh = false;
                }
                if (id >= 0 && id < a.num_pages)
                    slot[k] = id * a.page_size + static_cast<int32_t>(row);
                else
                    report(a.dev_status, GDN_DEV_BAD_SLOT);
            }
            if (a.aligned && g * 4 >= t0 && g * 4 + 4 <= t1) {
                reinterpret_cast<int4 *>(a.slot_map)[g] = make_int4(slot[0], slot[1], slot[2], slot[3]);
                reinterpret_cast<int4 *>(a.positions)[g] = make_int4(where[0], where[1], where[2], where[3]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (g * 4 + k >= t0 && g * 4 + k < t1) {
                        a.slot_map[g * 4 + k] = slot[k];
                        a.positions[g * 4 + k] = where[k];
                    }
            }
        }
        for (int64_t e = rank * threads + tid; e < tile_page; e += blocks * threads) {
            const int j = find_last(s_page, threads, static_cast<int32_t>(e));
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
    for (int64_t t = end + rank * threads + tid; t < cap; t += blocks * threads) {
        a.slot_map[t] = -1;
        a.positions[t] = 0;
    }
    if (blocks > 1) cluster_wait();  // every block has read free_head
    if (rank == 0 && tid == 0) {
        a.cu_seqlens[a.num_reqs] = static_cast<int32_t>(end);
        if (a.free_pages) *a.free_head_out = s_head;
    }
}

constexpr int kWriteThreads = 256;
constexpr int kWriteUnroll = 4;

// A block takes kWriteThreads * kWriteUnroll consecutive pieces of 16 bytes of
// one side (blockIdx.y: K or V), counted token, head, piece of the row; only
// the first of them needs 64-bit arithmetic.
__global__ void __launch_bounds__(kWriteThreads) write_kernel(const PagedWriteArgs a, uint32_t pieces_log2) {
    const PagedWriteSide &s = a.side[blockIdx.y];
    const uint32_t per_token = static_cast<uint32_t>(a.h) << pieces_log2, mask = (1u << pieces_log2) - 1;
    const uint32_t P = static_cast<uint32_t>(a.page_size);
    const int64_t slots = a.num_pages * a.page_size, all = a.num_tokens * per_token;
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * (kWriteThreads * kWriteUnroll); first < all;
         first += static_cast<int64_t>(gridDim.x) * (kWriteThreads * kWriteUnroll)) {
        const int64_t t0 = first / per_token;
        const uint32_t skip = static_cast<uint32_t>(first - t0 * per_token);
        uint4 val[kWriteUnroll];
        uint16_t *to[kWriteUnroll];
#pragma unroll
        for (int u = 0; u < kWriteUnroll; ++u) {
            const uint32_t p = u * kWriteThreads + threadIdx.x;
            to[u] = nullptr;
            if (first + p >= all) continue;
            const uint32_t dt = (skip + p) / per_token, in = skip + p - dt * per_token;
            const uint32_t head = in >> pieces_log2, piece = in & mask;
            const int64_t t = t0 + dt;
            const int32_t slot = a.slot_map[t];
            if (slot < 0) continue;
            if (slot >= slots) {
                report(a.dev_status, GDN_DEV_BAD_SLOT);
                continue;
            }
            val[u] = __ldg(reinterpret_cast<const uint4 *>(s.src + t * s.token_stride + head * s.head_stride) + piece);
            const uint32_t page = static_cast<uint32_t>(slot) / P;
            to[u] = s.dst + page * s.page_stride + (static_cast<uint32_t>(slot) - page * P) * s.slot_stride +
                    head * s.dst_head_stride + piece * 8;
        }
#pragma unroll
        for (int u = 0; u < kWriteUnroll; ++u)
            if (to[u]) *reinterpret_cast<uint4 *>(to[u]) = val[u];
    }
}

}  // namespace

cudaError_t launch_paged_maps(const PagedMapsArgs &a, cudaStream_t stream) {
    // A block for up to 4096 tokens of capacity, then one more per 4096.
    const int64_t want = (a.token_capacity + 4 * kMapThreads - 1) / (4 * kMapThreads);
    int blocks = 1;
    while (blocks < kMapMaxBlocks && blocks < want) blocks *= 2;
    // Few requests and tokens: few warps, whose barriers cost less.
    int threads = kMapThreads;
    if (blocks == 1)
        while (threads > 32 && a.num_reqs <= threads / 2 && a.token_capacity <= 2 * threads) threads /= 2;
    PagedMapsArgs k = a;
    k.aligned = ((reinterpret_cast<uintptr_t>(a.slot_map) | reinterpret_cast<uintptr_t>(a.positions)) & 15u) == 0;
    if (blocks == 1) {  // no cluster, whose launch costs more
        maps_kernel<<<1, threads, 0, stream>>>(k);
        return cudaGetLastError();
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = blocks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, maps_kernel, k);
}

cudaError_t launch_paged_write(const PagedWriteArgs &a, cudaStream_t stream) {
    int dev = 0, sms = 0;
    if (!current_device(&dev, &sms)) return cudaErrorInvalidDevice;
    uint32_t lg = 0;
    while ((8 << lg) < a.d) ++lg;
    const int64_t pieces = a.num_tokens * a.h << lg;
    int64_t blocks = (pieces + kWriteThreads * kWriteUnroll - 1) / (kWriteThreads * kWriteUnroll);
    if (blocks > INT_MAX) blocks = INT_MAX;
    write_kernel<<<dim3(static_cast<unsigned>(blocks), 2), kWriteThreads, 0, stream>>>(a, lg);
    return cudaGetLastError();
}

}  // namespace gdn
