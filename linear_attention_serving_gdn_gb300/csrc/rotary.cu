// Rotary positions: each pair (a, b) of a head's first `rot` elements becomes
//   magnitude * (a cos - b sin, b cos + a sin),  angle = position * frequency.
//
// Angles.  A frequency is held in turns per position as a 64-bit fraction, so
// position * frequency modulo one turn is one integer product, exact for any
// int32 position: no range reduction, no 64-bit floating point.  Its upper 32
// bits are the turn's fraction to 2^-32; sincospif takes it from there.
//
// Split.  A thread takes eight pairs (two 16-byte pieces) of a token in all or
// some of its heads; with few tokens the heads are dealt out over more threads.
// A block makes the angles of its tokens once, in shared memory, while the
// first heads are on the way from memory.
// Bound by HBM for long chunks, by the launch for decode steps.
#include "paged.cuh"

#include <cuda_fp16.h>
#include <limits.h>

namespace gdn {
namespace {

constexpr int kRotaryThreads = 256;
constexpr int kRotaryUnroll = 4;  // heads whose loads are in flight at once
constexpr int kRotaryPairs = kRotaryThreads * 8;  // of a block: eight per turning thread

// Cosine and sine of a pair at a position, times the magnitude.
__device__ __forceinline__ float2 turn(const RotaryArgs &a, int64_t position, uint64_t frequency) {
    const uint64_t phase = static_cast<uint64_t>(position) * frequency;
    // (the upper half as a signed number: -1/2 to 1/2 turns, in units of 2^-32; sincospi's argument is half turns)
    const float x = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f;  // 2^-31
    float c, s;
    sincospif(x, &s, &c);
    return make_float2(c * a.magnitude, s * a.magnitude);
}

template <bool kHalf>
__device__ __forceinline__ float2 unpack(uint32_t x) {
    if (kHalf) return __half22float2(*reinterpret_cast<__half2 *>(&x));
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
template <bool kHalf>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    if (kHalf)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The heads of both sides are counted on: q's, then k's.
__device__ __forceinline__ const RotarySide &side_of(const RotaryArgs &a, int32_t *head) {
    if (*head < a.side[0].h) return a.side[0];
    *head -= a.side[0].h;
    return a.side[1];
}

// Lanes of a token: turns = rot / 16 of two pieces to turn, then those of two pieces to copy (where the output lies
// elsewhere).  `splits` threads share a lane's heads; a block takes `tokens` tokens, lanes * splits * tokens <= its threads.
template <bool kHalf, bool kInterleaved, bool kOnce>
__global__ void __launch_bounds__(kRotaryThreads, kOnce ? 4 : 3) rotary_kernel(const __grid_constant__ RotaryArgs a, int32_t turns, int32_t lanes,
                                                                   int32_t splits, int32_t tokens) {
    __shared__ float2 angle[kRotaryPairs];  // cosine and sine of the tokens' pairs
    const int32_t per_token = lanes * splits;
    const int32_t token = static_cast<int32_t>(threadIdx.x) / per_token, rest = static_cast<int32_t>(threadIdx.x) - token * per_token;
    const int32_t split = rest / lanes, lane = rest - split * lanes;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * tokens, t = first + token;
    const bool live = token < tokens && t < a.num_tokens;
    const int32_t heads = a.side[0].h + a.side[1].h;
    const bool turning = lane < turns;
    // First elements of the two pieces; a last copy lane may have only one.
    const int32_t at0 = turning ? lane * (kInterleaved ? 16 : 8) : a.rot + (lane - turns) * 16;
    const int32_t at1 = turning && !kInterleaved ? at0 + a.rot / 2 : at0 + 8;
    const bool two = at1 < a.d;
    uint4 x[kRotaryUnroll], y[kRotaryUnroll];
    auto load = [&](int32_t h0) {
#pragma unroll
        for (int k = 0; k < kRotaryUnroll; ++k) {
            int32_t h = h0 + k * splits;
            if (!live || h >= heads) continue;
            const RotarySide &side = side_of(a, &h);
            if (!turning && side.src == side.dst) continue;
            const uint16_t *p = side.src + t * side.token_stride + h * side.head_stride;
            x[k] = *reinterpret_cast<const uint4 *>(p + at0);
            if (two) y[k] = *reinterpret_cast<const uint4 *>(p + at1);
        }
    };
    if (kOnce) load(split);  // (on the way while the angles are made)
    const int32_t pairs = a.rot / 2;
    for (int32_t i = threadIdx.x; i < tokens * pairs; i += kRotaryThreads) {
        const int32_t of = i / pairs;
        if (first + of < a.num_tokens)
            angle[i] = turn(a, a.positions[first + of], a.frequencies[i - of * pairs]);
    }
    __syncthreads();
    float c[8], s[8];
    if (turning && live)
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const float4 cs = *reinterpret_cast<const float4 *>(angle + token * pairs + lane * 8 + j);
            c[j] = cs.x, s[j] = cs.y, c[j + 1] = cs.z, s[j + 1] = cs.w;
        }
#pragma unroll 1
    for (int32_t h0 = split; live && h0 < heads; h0 += splits * kRotaryUnroll) {
        if (!kOnce) load(h0);
#pragma unroll
        for (int k = 0; k < kRotaryUnroll; ++k) {
            int32_t h = h0 + k * splits;
            if (h >= heads) continue;
            const RotarySide &side = side_of(a, &h);
            if (!turning && side.src == side.dst) continue;
            if (turning) {
                uint32_t u[8] = {x[k].x, x[k].y, x[k].z, x[k].w, y[k].x, y[k].y, y[k].z, y[k].w};
                if (kInterleaved) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 v = unpack<kHalf>(u[j]);
                        u[j] = pack<kHalf>(v.x * c[j] - v.y * s[j], v.y * c[j] + v.x * s[j]);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 v = unpack<kHalf>(u[j]), w = unpack<kHalf>(u[j + 4]);
                        u[j] = pack<kHalf>(v.x * c[2 * j] - w.x * s[2 * j], v.y * c[2 * j + 1] - w.y * s[2 * j + 1]);
                        u[j + 4] = pack<kHalf>(w.x * c[2 * j] + v.x * s[2 * j], w.y * c[2 * j + 1] + v.y * s[2 * j + 1]);
                    }
                }
                x[k] = make_uint4(u[0], u[1], u[2], u[3]);
                y[k] = make_uint4(u[4], u[5], u[6], u[7]);
            }
            uint16_t *p = side.dst + t * side.dst_token_stride + h * side.dst_head_stride;
            *reinterpret_cast<uint4 *>(p + at0) = x[k];
            if (two) *reinterpret_cast<uint4 *>(p + at1) = y[k];
        }
        if (kOnce) break;
    }
}

// Any head size, rotary size, stride and alignment: a pair, or a copied element, per lane.
template <bool kHalf>
__global__ void __launch_bounds__(kRotaryThreads) rotary_any_kernel(const __grid_constant__ RotaryArgs a, int32_t turns,
                                                                    int32_t lanes, int32_t splits) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kRotaryThreads + threadIdx.x;
    const uint32_t per_token = static_cast<uint32_t>(lanes) * static_cast<uint32_t>(splits);
    const int64_t t = i / per_token;
    if (t >= a.num_tokens) return;
    const uint32_t rest = static_cast<uint32_t>(i - t * per_token);
    const int32_t split = static_cast<int32_t>(rest / static_cast<uint32_t>(lanes));
    const int32_t lane = static_cast<int32_t>(rest) - split * lanes;
    const int32_t heads = a.side[0].h + a.side[1].h;
    const bool turning = lane < turns;
    int32_t at0 = a.rot + lane - turns, at1 = at0;
    float c = 1.f, s = 0.f;
    if (turning) {
        at0 = a.interleaved ? 2 * lane : lane;
        at1 = a.interleaved ? at0 + 1 : lane + a.rot / 2;
        const float2 cs = turn(a, a.positions[t], a.frequencies[lane]);
        c = cs.x;
        s = cs.y;
    }
    for (int32_t h0 = split; h0 < heads; h0 += splits) {
        int32_t h = h0;
        const RotarySide &side = side_of(a, &h);
        if (!turning && side.src == side.dst) continue;
        const uint16_t *p = side.src + t * side.token_stride + h * side.head_stride;
        uint16_t *to = side.dst + t * side.dst_token_stride + h * side.dst_head_stride;
        if (!turning) {
            to[at0] = p[at0];
            continue;
        }
        const float2 v = unpack<kHalf>(p[at0] | static_cast<uint32_t>(p[at1]) << 16);
        const uint32_t out = pack<kHalf>(v.x * c - v.y * s, v.y * c + v.x * s);
        to[at0] = static_cast<uint16_t>(out);
        to[at1] = static_cast<uint16_t>(out >> 16);
    }
}

using RotaryKernel = void (*)(const RotaryArgs, int32_t, int32_t, int32_t, int32_t);
template <bool kHalf, bool kInterleaved>
RotaryKernel pick_once(bool once) {
    return once ? rotary_kernel<kHalf, kInterleaved, true> : rotary_kernel<kHalf, kInterleaved, false>;
}
RotaryKernel pick(bool half, bool interleaved, bool once) {
    if (half) return interleaved ? pick_once<true, true>(once) : pick_once<true, false>(once);
    return interleaved ? pick_once<false, true>(once) : pick_once<false, false>(once);
}

bool pieces16(const RotarySide &s) {
    return ((reinterpret_cast<uintptr_t>(s.src) | reinterpret_cast<uintptr_t>(s.dst)) & 15u) == 0 &&
           ((s.token_stride | s.head_stride | s.dst_token_stride | s.dst_head_stride) & 7) == 0;
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs &a, cudaStream_t stream) {
    int dev = 0, sms = 0;
    if (!current_device(&dev, &sms)) return cudaErrorInvalidDevice;
    const bool copies = a.side[0].src != a.side[0].dst || a.side[1].src != a.side[1].dst;
    const bool wide = a.rot % 16 == 0 && a.d % 8 == 0 && pieces16(a.side[0]) && pieces16(a.side[1]) &&
                      (reinterpret_cast<uintptr_t>(a.frequencies) & 15u) == 0;
    const int32_t turns = wide ? a.rot / 16 : a.rot / 2;
    const int32_t lanes = turns + (!copies ? 0 : wide ? (a.d - a.rot + 15) / 16 : a.d - a.rot);
    // Heads are dealt out until the GPU's threads are all used: each keeps as many as it can, for the angles' sake.
    const int32_t heads = a.side[0].h + a.side[1].h;
    const int64_t have = a.num_tokens * lanes, want = static_cast<int64_t>(sms) * 2048;
    int64_t splits = (want + have - 1) / have;
    if (splits > heads) splits = heads;
    const bool half = a.dtype == GDN_FP16;
    if (!wide) {
        const int64_t blocks = (have * splits + kRotaryThreads - 1) / kRotaryThreads;
        if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
        (half ? rotary_any_kernel<true> : rotary_any_kernel<false>)<<<static_cast<unsigned>(blocks), kRotaryThreads, 0, stream>>>(
            a, turns, lanes, static_cast<int32_t>(splits));
        return cudaGetLastError();
    }
    if (splits * lanes > kRotaryThreads) splits = kRotaryThreads / lanes;  // (at most 64 lanes: d <= 1024)
    const int32_t n = static_cast<int32_t>(splits), tokens = kRotaryThreads / (lanes * n);
    const dim3 grid(static_cast<unsigned>((a.num_tokens + tokens - 1) / tokens));
    const auto kernel = pick(half, a.interleaved, n * kRotaryUnroll >= heads);
    kernel<<<grid, kRotaryThreads, 0, stream>>>(a, turns, lanes, n, tokens);
    return cudaGetLastError();
}

}  // namespace gdn
