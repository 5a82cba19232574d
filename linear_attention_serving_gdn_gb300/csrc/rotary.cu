// Rotary positions: each pair (a, b) of a head's first `rot` elements becomes
//   magnitude * (a cos - b sin, b cos + a sin),  angle = position * frequency.
//
// Angles.  A frequency is held in turns per position as a 64-bit fraction, so
// position * frequency modulo one turn is one integer product, exact for any
// int32 position: no range reduction, no 64-bit floating point.  Its upper 32
// bits are the turn's fraction to 2^-32; sincospif takes it from there.
//
// Split.  A thread takes eight pairs (two 16-byte pieces; four or two, or a
// pair alone, where sizes, strides or addresses do not allow them) of a token
// in all or some of its heads; with few tokens the heads are dealt out over
// more threads, and a thread that has four heads at most asks for all of them
// before the angles are made.  A block makes its tokens' angles once, in shared
// memory: two integer products and a sincospif each, for all heads.
//
// What bounds it: HBM for chunks (32768 tokens, 40 heads of 128: 671 MB in
// 105 us, 0.94 of the copy peak; 200000 tokens, 6 heads of 80 by 4-byte pieces
// 102 us, pair by pair 245); for a step of some thousand tokens the launch and a
// block's chain of loads, angles and stores as well (4096 tokens, 18 heads of 256,
// 64 of them turned: 75 MB in 16.4 us, 0.68; angles made by each thread for
// itself 19 us); the host's call for decode steps (8 tokens: 2.3 us on the GPU).
#include "paged.cuh"

#include <cuda_fp16.h>
#include <limits.h>

namespace gdn {
namespace {

constexpr int kRotaryThreads = 256;
constexpr int kRotaryUnroll = 4;  // heads whose loads are in flight at once

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

// The pair (a, b), turned; written out so that every kernel gives the same bits.
__device__ __forceinline__ float2 rotate(float a, float b, float2 cs) {
    return make_float2(fmaf(a, cs.x, -(b * cs.y)), fmaf(b, cs.x, a * cs.y));
}

// The heads of both sides are counted on: q's, then k's.
__device__ __forceinline__ const RotarySide &side_of(const RotaryArgs &a, int32_t *head) {
    if (*head < a.side[0].h) return a.side[0];
    *head -= a.side[0].h;
    return a.side[1];
}

// A piece of kWide elements.
template <int kWide>
struct Piece {
    uint32_t w[kWide / 2];
};
template <int kWide>
__device__ __forceinline__ Piece<kWide> load_piece(const uint16_t *p) {
    Piece<kWide> x;
    if constexpr (kWide == 8) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        x.w[0] = v.x, x.w[1] = v.y, x.w[2] = v.z, x.w[3] = v.w;
    } else if constexpr (kWide == 4) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        x.w[0] = v.x, x.w[1] = v.y;
    } else {
        x.w[0] = *reinterpret_cast<const uint32_t *>(p);
    }
    return x;
}
template <int kWide>
__device__ __forceinline__ void store_piece(uint16_t *p, const Piece<kWide> &x) {
    if constexpr (kWide == 8)
        *reinterpret_cast<uint4 *>(p) = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
    else if constexpr (kWide == 4)
        *reinterpret_cast<uint2 *>(p) = make_uint2(x.w[0], x.w[1]);
    else
        *reinterpret_cast<uint32_t *>(p) = x.w[0];
}

// Lanes of a token: turns = rot / (2 kWide) of two pieces to turn, then those of two pieces to copy (where the output lies
// elsewhere).  `splits` threads share a lane's heads; a block takes `tokens` tokens, lanes * splits * tokens <= its threads.
// With kOnce a thread's heads are all asked for at once, before the angles are made.
template <int kWide, bool kHalf, bool kInterleaved, bool kOnce>
__global__ void __launch_bounds__(kRotaryThreads, kOnce ? 4 : 3) rotary_kernel(const __grid_constant__ RotaryArgs a, int32_t turns,
                                                                              int32_t lanes, int32_t splits, int32_t tokens) {
    __shared__ float2 angle[kRotaryThreads * kWide];  // cosine and sine of the tokens' pairs
    const int32_t per_token = lanes * splits;
    const int32_t token = static_cast<int32_t>(threadIdx.x) / per_token, rest = static_cast<int32_t>(threadIdx.x) - token * per_token;
    const int32_t split = rest / lanes, lane = rest - split * lanes;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * tokens, t = first + token;
    const bool live = token < tokens && t < a.num_tokens;
    const int32_t heads = a.side[0].h + a.side[1].h;
    const bool turning = lane < turns;
    // First elements of the two pieces; a last copy lane may have only one.
    const int32_t at0 = turning ? lane * (kInterleaved ? 2 * kWide : kWide) : a.rot + (lane - turns) * (2 * kWide);
    const int32_t at1 = turning && !kInterleaved ? at0 + a.rot / 2 : at0 + kWide;
    const bool two = at1 < a.d;
    Piece<kWide> x[kRotaryUnroll], y[kRotaryUnroll];
    auto load = [&](int32_t h0) {
#pragma unroll
        for (int k = 0; k < kRotaryUnroll; ++k) {
            int32_t h = h0 + k * splits;
            if (!live || h >= heads) continue;
            const RotarySide &side = side_of(a, &h);
            if (!turning && side.src == side.dst) continue;
            const uint16_t *p = side.src + t * side.token_stride + h * side.head_stride;
            x[k] = load_piece<kWide>(p + at0);
            if (two) y[k] = load_piece<kWide>(p + at1);
        }
    };
    if (kOnce) load(split);
    const int32_t pairs = a.rot / 2;
    for (int32_t i = threadIdx.x; i < tokens * pairs; i += kRotaryThreads) {
        const int32_t of = i / pairs;
        if (first + of < a.num_tokens)
            angle[i] = turn(a, a.positions[first + of], a.frequencies[i - of * pairs]);
    }
    __syncthreads();
    float2 cs[kWide];
    if (turning && live)
#pragma unroll
        for (int j = 0; j < kWide; ++j) cs[j] = angle[token * pairs + lane * kWide + j];
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
#pragma unroll
                for (int j = 0; j < kWide / 2; ++j) {
                    const float2 v = unpack<kHalf>(x[k].w[j]), w = unpack<kHalf>(y[k].w[j]);
                    if (kInterleaved) {
                        const float2 e = rotate(v.x, v.y, cs[j]), f = rotate(w.x, w.y, cs[kWide / 2 + j]);
                        x[k].w[j] = pack<kHalf>(e.x, e.y);
                        y[k].w[j] = pack<kHalf>(f.x, f.y);
                    } else {
                        const float2 e = rotate(v.x, w.x, cs[2 * j]), f = rotate(v.y, w.y, cs[2 * j + 1]);
                        x[k].w[j] = pack<kHalf>(e.x, f.x);
                        y[k].w[j] = pack<kHalf>(e.y, f.y);
                    }
                }
            }
            uint16_t *p = side.dst + t * side.dst_token_stride + h * side.dst_head_stride;
            store_piece<kWide>(p + at0, x[k]);
            if (two) store_piece<kWide>(p + at1, y[k]);
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
    float2 cs = make_float2(1.f, 0.f);
    if (turning) {
        at0 = a.interleaved ? 2 * lane : lane;
        at1 = a.interleaved ? at0 + 1 : lane + a.rot / 2;
        cs = turn(a, a.positions[t], a.frequencies[lane]);
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
        const float2 e = rotate(v.x, v.y, cs);
        const uint32_t out = pack<kHalf>(e.x, e.y);
        to[at0] = static_cast<uint16_t>(out);
        to[at1] = static_cast<uint16_t>(out >> 16);
    }
}

using RotaryKernel = void (*)(const RotaryArgs, int32_t, int32_t, int32_t, int32_t);
template <int kWide, bool kHalf, bool kInterleaved>
RotaryKernel pick_once(bool once) {
    return once ? rotary_kernel<kWide, kHalf, kInterleaved, true> : rotary_kernel<kWide, kHalf, kInterleaved, false>;
}
template <int kWide>
RotaryKernel pick(bool half, bool interleaved, bool once) {
    if (half) return interleaved ? pick_once<kWide, true, true>(once) : pick_once<kWide, true, false>(once);
    return interleaved ? pick_once<kWide, false, true>(once) : pick_once<kWide, false, false>(once);
}

// Whether pieces of `wide` elements lie at multiples of their size.
bool pieces_of(const RotarySide &s, int32_t wide) {
    return ((reinterpret_cast<uintptr_t>(s.src) | reinterpret_cast<uintptr_t>(s.dst)) & (2 * wide - 1)) == 0 &&
           ((s.token_stride | s.head_stride | s.dst_token_stride | s.dst_head_stride) & (wide - 1)) == 0;
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs &a, cudaStream_t stream) {
    int dev = 0, sms = 0;
    if (!current_device(&dev, &sms)) return cudaErrorInvalidDevice;
    const bool copies = a.side[0].src != a.side[0].dst || a.side[1].src != a.side[1].dst;
    int32_t wide = 8;  // elements of a piece, 1: single pairs
    while (wide > 1 && (a.rot % (2 * wide) != 0 || a.d % wide != 0 || !pieces_of(a.side[0], wide) || !pieces_of(a.side[1], wide)))
        wide /= 2;
    const int32_t turns = a.rot / (2 * wide);
    const int32_t lanes = turns + (!copies ? 0 : wide > 1 ? (a.d - a.rot + 2 * wide - 1) / (2 * wide) : a.d - a.rot);
    // Heads are dealt out until the GPU's threads are all used: each keeps as many as it can, for the angles' sake.
    const int32_t heads = a.side[0].h + a.side[1].h;
    const int64_t have = a.num_tokens * lanes, want = static_cast<int64_t>(sms) * 2048;
    int64_t splits = (want + have - 1) / have;
    if (splits > heads) splits = heads;
    const bool half = a.dtype == GDN_FP16;
    if (wide == 1) {
        const int64_t blocks = (have * splits + kRotaryThreads - 1) / kRotaryThreads;
        if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
        (half ? rotary_any_kernel<true> : rotary_any_kernel<false>)<<<static_cast<unsigned>(blocks), kRotaryThreads, 0, stream>>>(
            a, turns, lanes, static_cast<int32_t>(splits));
        return cudaGetLastError();
    }
    if (splits * lanes > kRotaryThreads) splits = kRotaryThreads / lanes;  // (at most 256 lanes: d <= 1024)
    const int32_t n = static_cast<int32_t>(splits), tokens = kRotaryThreads / (lanes * n);
    const bool once = n * kRotaryUnroll >= heads;
    const RotaryKernel kernel = wide == 8   ? pick<8>(half, a.interleaved, once)
                                : wide == 4 ? pick<4>(half, a.interleaved, once)
                                            : pick<2>(half, a.interleaved, once);
    kernel<<<static_cast<unsigned>((a.num_tokens + tokens - 1) / tokens), kRotaryThreads, 0, stream>>>(a, turns, lanes, n, tokens);
    return cudaGetLastError();
}

}  // namespace gdn
