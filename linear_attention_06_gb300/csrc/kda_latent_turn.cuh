// kda_latent_turn.cuh -- the position rotation of the latent cache's appends, and the sequence that a token belongs to.
//
// The angle of pair i is p * f_i.  In fp32 the product of a position near 10^6 and f_0 = 1 is off by
// 0.03 rad.  So f_i / 2 pi is taken in fp64, once a block, as a fraction of a turn in 64-bit fixed point, and
// p times it modulo 2^64 is the reduced angle: exact but for the fraction's own 53 bits (2^-25 turns at p = 2^31).
// Sine and cosine of the fp32 remainder are then good to about 2^-22.  (An fp64 product and reduction for every
// token and pair took 3.5 us of 8000 tokens on this card, whose fp64 rate is a few operations a cycle and SM.)
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_latent_common.cuh"

namespace kda {
namespace latent {

struct Turn {
    float c, s;
};

// A position's share of a turn at frequency f, in 2^-64; sine and cosine at position p.
__device__ __forceinline__ uint64_t share_of_turn(float f) {
    const double turn = (double)f * 0.15915494309189533577;                                   // / 2 pi
    return (uint64_t)((turn - floor(turn)) * 18446744073709551616.0);                         // * 2^64
}
__device__ __forceinline__ Turn turn_at(int64_t p, uint64_t share) {
    const uint64_t angle = (uint64_t)p * share;
    Turn t;
    sincospif((float)(int32_t)(angle >> 32) * 0x1p-31f, &t.s, &t.c);                          // half turns in [-1, 1]
    return t;
}

// What happens to a row's rotated part: copied, pairs (i, i + 32) turned, pairs (2i, 2i + 1) turned.  A copy keeps every
// bit: a product with (1, 0) would turn an infinite channel's partner into NaN and could lose the sign of a zero.
enum Turning { kCopied, kHalves, kInterleaved };

// Eight pairs of one 64-channel row: the two 16-byte chunks that unit u (0..3) of the row owns, i.e.
// channels 8u.. and 8u + 32.. (pairs i, i + 32), or 16u..16u + 15 (interleaved pairs).
struct Unit {
    uint4 x0, x1;
};
template <Turning TURN>
__device__ __forceinline__ Unit load_unit(const __nv_bfloat16* src, int u) {
    const uint4* p = reinterpret_cast<const uint4*>(src);
    return {p[TURN == kInterleaved ? 2 * u : u], p[TURN == kInterleaved ? 2 * u + 1 : u + 4]};
}
template <Turning TURN>
__device__ __forceinline__ void store_unit(uint4 y0, uint4 y1, __nv_bfloat16* dst, int u) {
    reinterpret_cast<uint4*>(dst)[TURN == kInterleaved ? 2 * u : u] = y0;
    reinterpret_cast<uint4*>(dst)[TURN == kInterleaved ? 2 * u + 1 : u + 4] = y1;
}
template <Turning TURN>
__device__ __forceinline__ void rotate_unit(const Unit& x, __nv_bfloat16* dst, int u, const Turn* turn) {
    if constexpr (TURN == kCopied) return store_unit<TURN>(x.x0, x.x1, dst, u);
    const __nv_bfloat162* a = reinterpret_cast<const __nv_bfloat162*>(&x.x0);
    const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(&x.x1);
    uint4 y0, y1;
    __nv_bfloat162* ya = reinterpret_cast<__nv_bfloat162*>(&y0);
    __nv_bfloat162* yb = reinterpret_cast<__nv_bfloat162*>(&y1);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 fa = __bfloat1622float2(a[k]), fb = __bfloat1622float2(b[k]);
        if constexpr (TURN == kInterleaved) {   // fa, fb are pairs 8u + k and 8u + 4 + k
            const Turn t = turn[8 * u + k], v = turn[8 * u + 4 + k];
            ya[k] = __floats2bfloat162_rn(fa.x * t.c - fa.y * t.s, fa.x * t.s + fa.y * t.c);
            yb[k] = __floats2bfloat162_rn(fb.x * v.c - fb.y * v.s, fb.x * v.s + fb.y * v.c);
        } else {                                // pairs 8u + 2k and 8u + 2k + 1
            const Turn t = turn[8 * u + 2 * k], v = turn[8 * u + 2 * k + 1];
            ya[k] = __floats2bfloat162_rn(fa.x * t.c - fb.x * t.s, fa.y * v.c - fb.y * v.s);
            yb[k] = __floats2bfloat162_rn(fa.x * t.s + fb.x * t.c, fa.y * v.s + fb.y * v.c);
        }
    }
    store_unit<TURN>(y0, y1, dst, u);
}

// find_seq by a whole warp: 32 offsets a step instead of one, since each step waits for memory.
__device__ __forceinline__ int find_seq_warp(const int32_t* cu, int num_seqs, int64_t total, int64_t t, int64_t& b,
                                             int64_t& e) {
    if (!cu) return find_seq(cu, num_seqs, total, t, b, e);
    const int lane = threadIdx.x & 31;
    int lo = 0, count = num_seqs;               // the last n in [lo, lo + count) with cu[n] <= t
    while (count > 1) {
        const int step = (count + 31) / 32, at = lane * step;
        const uint32_t mask = __ballot_sync(0xffffffffu, at < count && (lane == 0 || (int64_t)cu[lo + at] <= t));
        const int skip = (31 - __clz(mask)) * step;
        lo += skip;
        count = count - skip < step ? count - skip : step;
    }
    bounds(cu, lo, num_seqs, total, b, e);
    return t >= b && t < e ? lo : -1;
}

}  // namespace latent
}  // namespace kda
