// kda_latent_cache.cu -- the latent cache of kda.h: rows in (with the position rotation) and rows out.
//
// Append, token t at position p:  cache[row(p)] = [ c_t | R(p) r_t ],  q'_th = R(p) q_th.
// Gather:                         c_t, r_t = cache[row(p)].
// Both move every byte once and compute next to nothing, so memory bounds them (and, for a step of
// few tokens, the launch and two dependent loads: the sequence's bounds, then the page).
//
// The angle of pair i is p * f_i.  In fp32 the product of a position near 10^6 and f_0 = 1 is off by
// 0.03 rad.  So f_i / 2 pi is taken in fp64, once a block, as a fraction of a turn in 64-bit fixed point, and
// p times it modulo 2^64 is the reduced angle: exact but for the fraction's own 53 bits (2^-25 turns at p = 2^31).
// Sine and cosine of the fp32 remainder are then good to about 2^-22.  (An fp64 product and reduction for every
// token and pair took 3.5 us of 8000 tokens on this card, whose fp64 rate is a few operations a cycle and SM.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_internal.h"
#include "kda_latent_common.cuh"

namespace kda {
namespace {

using namespace latent;

constexpr int kThreads = 256;

struct Turn {
    float c, s;
};

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

// TOK tokens a block.  The rows to copy and to rotate are requested before anything else: they arrive while the
// block finds its tokens' sequences, pages and angles.  A thread's first kQ units of queries take part in that;
// queries of more heads follow in a loop.
template <int TOK, Turning TURN>
__global__ void __launch_bounds__(kThreads, 3) append_kernel(const LatentAppendArgs a) {
    constexpr int kChunks = kLatent / 8, kLat = (TOK * kChunks + kThreads - 1) / kThreads, kQ = 4;
    __shared__ int64_t row_s[TOK], pos_s[TOK];
    __shared__ int live_s[TOK];
    __shared__ Turn turn_s[TOK][kRope / 2];
    __shared__ uint64_t step_s[kRope / 2];      // a position's share of a turn, in 2^-64
    const int tid = threadIdx.x, lane = tid & 31;
    const int64_t t0 = (int64_t)blockIdx.x * TOK;
    const int count = (int)(a.total_tokens - t0 < TOK ? a.total_tokens - t0 : TOK);
    const int width = kLatent + a.c.rope_dim;
    const __nv_bfloat16* latent = static_cast<const __nv_bfloat16*>(a.latent);
    const __nv_bfloat16* k_rope = static_cast<const __nv_bfloat16*>(a.k_rope);
    const __nv_bfloat16* q_rope = static_cast<const __nv_bfloat16*>(a.q_rope);
    const int units = q_rope ? 4 * a.H : 0;
    uint4 lat[kLat];
    Unit key{}, q[kQ];
    allow_next();
    wait_before();
#pragma unroll
    for (int k = 0; k < kLat; ++k) {
        const int i = tid + k * kThreads;
        if (i < count * kChunks)
            lat[k] = reinterpret_cast<const uint4*>(latent + (t0 + i / kChunks) * a.latent_stride)[i % kChunks];
    }
    if (k_rope && tid < count * 4) key = load_unit<TURN>(k_rope + (t0 + (tid >> 2)) * a.k_rope_stride, tid & 3);
#pragma unroll
    for (int k = 0; k < kQ; ++k) {
        const int i = tid + k * kThreads;
        if (i < count * units) q[k] = load_unit<TURN>(q_rope + (t0 * a.H + (i >> 2)) * a.q_stride, i & 3);
    }
    if (TURN != kCopied && tid >= kThreads - kRope / 2) {
        const int k = tid - (kThreads - kRope / 2);
        const double turn = (double)a.inv_freq[k] * 0.15915494309189533577;                   // / 2 pi
        step_s[k] = (uint64_t)((turn - floor(turn)) * 18446744073709551616.0);                // * 2^64
    }
    for (int j = tid >> 5; j < count; j += kThreads / 32) {
        int64_t b, e;
        const int n = find_seq_warp(a.cu_seqlens, a.num_seqs, a.total_tokens, t0 + j, b, e);
        if (lane == 0) {
            const int64_t p = n < 0 ? 0 : (int64_t)a.seq_lens[n] - (e - (t0 + j));
            live_s[j] = n >= 0;
            pos_s[j] = p;
            int64_t row = n < 0 ? -1 : cache_row(a.c, n, p);
            if (row >= 0 && !KDA_INDEX_OK(row, (int64_t)a.c.num_pages * a.c.page_size, a.status)) row = -1;
            row_s[j] = row;
        }
    }
    __syncthreads();
    if (TURN != kCopied) {
        for (int i = tid; i < count * (kRope / 2); i += kThreads) {
            const int j = i / (kRope / 2), k = i % (kRope / 2);
            const uint64_t angle = (uint64_t)pos_s[j] * step_s[k];
            Turn t;
            sincospif((float)(int32_t)(angle >> 32) * 0x1p-31f, &t.s, &t.c);                  // half turns in [-1, 1]
            turn_s[j][k] = t;
        }
        __syncthreads();
    }
    __nv_bfloat16* cache = static_cast<__nv_bfloat16*>(a.c.cache);
#pragma unroll
    for (int k = 0; k < kLat; ++k) {
        const int i = tid + k * kThreads, j = i / kChunks;
        if (i < count * kChunks && row_s[j] >= 0) reinterpret_cast<uint4*>(cache + row_s[j] * width)[i % kChunks] = lat[k];
    }
    if (k_rope && tid < count * 4 && row_s[tid >> 2] >= 0)
        rotate_unit<TURN>(key, cache + row_s[tid >> 2] * width + kLatent, tid & 3, turn_s[tid >> 2]);
    auto turn_q = [&](int i, const Unit& x) {
        const int j = i / units;
        if (live_s[j])
            rotate_unit<TURN>(x, static_cast<__nv_bfloat16*>(a.q_out) + (t0 * a.H + (i >> 2)) * a.q_out_stride, i & 3,
                                     turn_s[j]);
    };
#pragma unroll
    for (int k = 0; k < kQ; ++k) {
        const int i = tid + k * kThreads;
        if (i < count * units) turn_q(i, q[k]);
    }
    for (int i = tid + kQ * kThreads; i < count * units; i += kThreads)
        turn_q(i, load_unit<TURN>(q_rope + (t0 * a.H + (i >> 2)) * a.q_stride, i & 3));
}

// ROWS rows a block, a 16-byte chunk a thread and step, all of a thread's loads before its stores.  The rows are read
// once, past L1 and never as read-only data: an overlapped block starts while the append before it may still write them.
template <int ROWS, int CHUNKS>
__global__ void __launch_bounds__(kThreads) gather_kernel(const LatentGatherArgs a) {
    __shared__ int64_t row_s[ROWS];             // -1: zeros, -2: no sequence's
    const int tid = threadIdx.x;
    const int64_t t0 = (int64_t)blockIdx.x * ROWS;
    allow_next();
    wait_before();
    if (tid < ROWS) {
        int64_t r = -2;
        if (t0 + tid < a.total_tokens) {
            int64_t b, e;
            const int n = find_seq(a.cu_seqlens, a.num_seqs, a.total_tokens, t0 + tid, b, e);
            if (n >= 0) r = cache_row(a.c, n, t0 + tid - b + (a.starts ? a.starts[n] : 0));
        }
        row_s[tid] = r;
    }
    __syncthreads();
    constexpr int kSteps = (ROWS * CHUNKS + kThreads - 1) / kThreads, kLat = kLatent / 8;
    const uint4* cache = static_cast<const uint4*>(a.c.cache);
    uint4 x[kSteps];
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
        const int i = tid + k * kThreads, j = i / CHUNKS, c = i % CHUNKS;
        x[k] = make_uint4(0, 0, 0, 0);
        if (i < ROWS * CHUNKS && row_s[j] >= 0 &&
            KDA_INDEX_OK(row_s[j], (int64_t)a.c.num_pages * a.c.page_size, a.status))
            x[k] = __ldcg(cache + row_s[j] * CHUNKS + c);
    }
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
        const int i = tid + k * kThreads, j = i / CHUNKS, c = i % CHUNKS;
        if (i >= ROWS * CHUNKS || row_s[j] < -1) continue;
        if (c < kLat)
            static_cast<uint4*>(a.latent)[(t0 + j) * kLat + c] = x[k];
        else
            static_cast<uint4*>(a.k_rope)[(t0 + j) * (CHUNKS - kLat) + c - kLat] = x[k];
    }
}

// Calls of few tokens take few rows a block, so that every SM has some; they end sooner than the host makes the
// next call, so an overlapped launch (about 1 us more of the host) only helps the others.
template <int TOK>
cudaError_t append(const LatentAppendArgs& a, bool overlapped, cudaStream_t s) {
    const unsigned blocks = (unsigned)((a.total_tokens + TOK - 1) / TOK);
    const auto kernel = !a.inv_freq ? append_kernel<TOK, kCopied>
                        : a.interleaved ? append_kernel<TOK, kInterleaved> : append_kernel<TOK, kHalves>;
    if (overlapped) return launch_overlapped(kernel, blocks, kThreads, 0, s, a);
    kernel<<<blocks, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <int ROWS>
cudaError_t gather(const LatentGatherArgs& a, bool overlapped, cudaStream_t s) {
    const unsigned blocks = (unsigned)((a.total_tokens + ROWS - 1) / ROWS);
    const auto kernel = a.c.rope_dim ? gather_kernel<ROWS, (kLatent + kRope) / 8> : gather_kernel<ROWS, kLatent / 8>;
    if (overlapped) return launch_overlapped(kernel, blocks, kThreads, 0, s, a);
    kernel<<<blocks, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_latent_append(const LatentAppendArgs& a, cudaStream_t s) {
    return a.total_tokens < 2048 ? append<1>(a, false, s) : append<8>(a, true, s);
}

cudaError_t launch_latent_gather(const LatentGatherArgs& a, cudaStream_t s) {
    return a.total_tokens < 8192 ? gather<4>(a, false, s) : gather<32>(a, true, s);
}

}  // namespace kda
