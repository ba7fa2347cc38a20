// kda_latent_cache_q8.cu -- the 8-bit latent cache of kda.h: rows quantised in (with the position rotation), rows out.
//
// Append, token t at position p:  x = [ c_t | R(p) r_t ],  cache[row(p)] = e4m3(x 2^-e), scales[row(p)] = e,
//                                 q'_th = R(p) q_th.
// Gather:                         [ c_t | r_t ] = cache[row(p)] 2^scales[row(p)].
// (the format: kda_latent_q8.cuh)  The rotated part stays in fp32 until it is quantised: one rounding.  Both move every
// byte once, and memory bounds them; a step of few tokens is bound by the launch and its chain of dependent loads.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_internal.h"
#include "kda_latent_common.cuh"
#include "kda_latent_q8.cuh"
#include "kda_latent_turn.cuh"

namespace kda {
namespace {

using namespace latent;

constexpr int kThreads = 256, kWarps = kThreads / 32;

__device__ __forceinline__ float2 floats(uint32_t pair) {
    return make_float2(__uint_as_float(pair << 16), __uint_as_float(pair & 0xffff0000u));
}
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// TOK tokens a block, a warp a row: a lane has two chunks of eight latent channels and one pair of rotated ones, so that
// a row's largest magnitude is one reduction of the warp.  As in the bf16 append, rows and queries are requested before
// anything else and arrive while the block finds its tokens' sequences, pages and angles.  Four blocks an SM (8 x
// 1000 tokens, 32 heads: 12.8 us; 13.9 with three, 15.9 with five).
template <int TOK, Turning TURN>
__global__ void __launch_bounds__(kThreads, 4) append_kernel(const LatentAppendArgs a) {
    static_assert(TOK <= kWarps, "a warp a token");
    constexpr int kQ = 4;
    __shared__ Turn turn_s[TOK][kRope / 2];
    __shared__ uint64_t step_s[kRope / 2];      // a position's share of a turn, in 2^-64
    __shared__ int64_t pos_s[TOK];
    __shared__ int live_s[TOK];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t t0 = (int64_t)blockIdx.x * TOK;
    const int count = (int)(a.total_tokens - t0 < TOK ? a.total_tokens - t0 : TOK);
    const int width = kLatent + a.c.rope_dim;
    const __nv_bfloat16* q_rope = static_cast<const __nv_bfloat16*>(a.q_rope);
    const int units = q_rope ? 4 * a.H : 0;
    const bool mine = warp < count;             // this warp has a row
    uint4 lat[2];
    uint32_t key = 0;
    Unit q[kQ];
    allow_next();
    wait_before();
    if (mine) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.latent) + (t0 + warp) * a.latent_stride);
        lat[0] = p[lane];
        lat[1] = p[lane + 32];
        if (a.k_rope) {
            const uint16_t* r = reinterpret_cast<const uint16_t*>(a.k_rope) + (t0 + warp) * a.k_rope_stride;
            key = TURN == kInterleaved ? reinterpret_cast<const uint32_t*>(r)[lane] : r[lane] | (uint32_t)r[lane + 32] << 16;
        }
    }
#pragma unroll
    for (int k = 0; k < kQ; ++k) {
        const int i = tid + k * kThreads;
        if (i < count * units) q[k] = load_unit<TURN>(q_rope + (t0 * a.H + (i >> 2)) * a.q_stride, i & 3);
    }
    if (TURN != kCopied && tid >= kThreads - kRope / 2) {
        const int k = tid - (kThreads - kRope / 2);
        step_s[k] = share_of_turn(a.inv_freq[k]);
    }
    int64_t row = -1;
    if (mine) {
        int64_t b, e;
        const int n = find_seq_warp(a.cu_seqlens, a.num_seqs, a.total_tokens, t0 + warp, b, e);
        const int64_t p = n < 0 ? 0 : (int64_t)a.seq_lens[n] - (e - (t0 + warp));
        if (n >= 0) row = cache_row(a.c, n, p);
        if (row >= 0 && !KDA_INDEX_OK(row, (int64_t)a.c.num_pages * a.c.page_size, a.status)) row = -1;
        if (lane == 0) {
            live_s[warp] = n >= 0;
            pos_s[warp] = p;
        }
    }
    __syncthreads();
    if (TURN != kCopied) {
        for (int i = tid; i < count * (kRope / 2); i += kThreads) {
            const int j = i / (kRope / 2), k = i % (kRope / 2);
            turn_s[j][k] = turn_at(pos_s[j], step_s[k]);
        }
        __syncthreads();
    }
    if (mine) {
        float2 k = floats(key);
        if constexpr (TURN != kCopied) {
            const Turn t = turn_s[warp][lane];
            k = make_float2(k.x * t.c - k.y * t.s, k.x * t.s + k.y * t.c);
        }
        const uint32_t* x = reinterpret_cast<const uint32_t*>(lat);
        uint32_t most = max(magnitude(k.x), magnitude(k.y));
#pragma unroll
        for (int i = 0; i < 8; ++i) most = max(most, max(x[i] << 16 & 0x7fff0000u, x[i] & 0x7fff0000u));
        const int e = power_for(__reduce_max_sync(0xffffffffu, most));
        const float f = two_to(-e);
        if (row >= 0) {
            uint8_t* out = static_cast<uint8_t*>(a.c.cache) + row * width;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t y[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 u = floats(x[4 * h + 2 * i]), v = floats(x[4 * h + 2 * i + 1]);
                    y[i] = to_e4m3x4(u.x * f, u.y * f, v.x * f, v.y * f);
                }
                reinterpret_cast<uint2*>(out)[lane + 32 * h] = make_uint2(y[0], y[1]);
            }
            if (a.c.rope_dim) {
                const uint32_t y = to_e4m3x2(k.x * f, k.y * f);
                if constexpr (TURN == kInterleaved) {
                    reinterpret_cast<uint16_t*>(out + kLatent)[lane] = (uint16_t)y;
                } else {
                    out[kLatent + lane] = (uint8_t)y;
                    out[kLatent + kRope / 2 + lane] = (uint8_t)(y >> 8);
                }
            }
            if (lane == 0) a.c.scales[row] = power_byte(e);
        }
    }
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

// ROWS rows a block, eight numbers a thread and step: a warp's loads (256 bytes) and stores (512) are whole lines.  All
// of a thread's loads come before its stores; rows are read past L1 and never as read-only data: an overlapped block
// starts while the append before it may still write them.
template <int ROWS, int CHUNKS>
__global__ void __launch_bounds__(kThreads) gather_kernel(const LatentGatherArgs a) {
    __shared__ int64_t row_s[ROWS];             // -1: zeros, -2: no sequence's
    __shared__ float scale_s[ROWS];
    const int tid = threadIdx.x;
    const int64_t t0 = (int64_t)blockIdx.x * ROWS;
    allow_next();
    wait_before();
    int64_t mine = -2;
    if (tid < ROWS) {
        if (t0 + tid < a.total_tokens) {
            int64_t b, e;
            const int n = find_seq(a.cu_seqlens, a.num_seqs, a.total_tokens, t0 + tid, b, e);
            if (n >= 0) mine = cache_row(a.c, n, t0 + tid - b + (a.starts ? a.starts[n] : 0));
        }
        if (mine >= 0 && !KDA_INDEX_OK(mine, (int64_t)a.c.num_pages * a.c.page_size, a.status)) mine = -1;
        row_s[tid] = mine;
    }
    __syncthreads();
    constexpr int kSteps = (ROWS * CHUNKS + kThreads - 1) / kThreads, kLat = kLatent / 8;
    const uint2* cache = static_cast<const uint2*>(a.c.cache);
    uint2 x[kSteps];
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
        const int i = tid + k * kThreads, j = i / CHUNKS, c = i % CHUNKS;
        x[k] = make_uint2(0, 0);
        if (i < ROWS * CHUNKS && row_s[j] >= 0) x[k] = __ldcg(cache + row_s[j] * CHUNKS + c);
    }
    if (tid < ROWS) scale_s[tid] = mine >= 0 ? two_to(power_of(__ldcg(a.c.scales + mine))) : 1.f;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
        const int i = tid + k * kThreads, j = i / CHUNKS, c = i % CHUNKS;
        if (i >= ROWS * CHUNKS || row_s[j] < -1) continue;
        const float f = scale_s[j];
        uint32_t y[4];
        e4m3x4_to_f16(x[k].x, y[0], y[1]);
        e4m3x4_to_f16(x[k].y, y[2], y[3]);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const float2 v = f16x2_to_floats(y[h]);
            const __nv_bfloat162 b = __floats2bfloat162_rn(v.x * f, v.y * f);                 // exact
            y[h] = *reinterpret_cast<const uint32_t*>(&b);
        }
        const uint4 row = make_uint4(y[0], y[1], y[2], y[3]);
        if (c < kLat)
            static_cast<uint4*>(a.latent)[(t0 + j) * kLat + c] = row;
        else
            static_cast<uint4*>(a.k_rope)[(t0 + j) * (CHUNKS - kLat) + c - kLat] = row;
    }
}

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

// As in bf16: calls of few tokens take few rows a block, so that every SM has some, and are launched plainly; they end
// sooner than the host makes the next call.  Tokens a block of an append, 32 heads: 1024 tokens take 6.3 us with 8, 9.8 with
// one, 1536 8.3 and 12.4, 8000 13.1 and 39.8; up to 512 the host's 6.3 us bound both.  Rows a block of a gather: 140000 take
// 38.4 us with 16, 45.1 with 8, 39.8 with 32, 63.6 with 4; 16000 5.8 with 16, 7.7 with 4; 4096 3.5 with either.
cudaError_t launch_latent_append_q8(const LatentAppendArgs& a, cudaStream_t s) {
    return a.total_tokens < 1024 ? append<1>(a, false, s) : append<8>(a, true, s);
}

cudaError_t launch_latent_gather_q8(const LatentGatherArgs& a, cudaStream_t s) {
    return a.total_tokens < 4096 ? gather<4>(a, false, s) : gather<16>(a, true, s);
}

}  // namespace kda
