// kda_latent_cache.cu -- the latent cache of kda.h: rows in (with the position rotation) and rows out.
//
// Append, token t at position p:  cache[row(p)] = [ c_t | R(p) r_t ],  q'_th = R(p) q_th.
// Gather:                         c_t, r_t = cache[row(p)].
// Both move every byte once and compute next to nothing, so memory bounds them (and, for a step of
// few tokens, the launch and two dependent loads: the sequence's bounds, then the page).
//
// The angle of pair i is p * f_i.  In fp32 the product of a position near 10^6 and f_0 = 1 is off by
// 0.03 rad, so the turns p * f_i / 2 pi are formed and reduced to [-1/2, 1/2] in fp64 (32 values a
// token, shared by all heads); sine and cosine of the fp32 remainder are then good to about 2^-22.
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

// Eight pairs of one 64-channel row: the two 16-byte chunks that unit u (0..3) of the row owns, i.e.
// channels 8u.. and 8u + 32.. (pairs i, i + 32), or 16u..16u + 15 (interleaved pairs).
template <bool INTERLEAVED>
__device__ __forceinline__ void rotate_unit(const __nv_bfloat16* src, __nv_bfloat16* dst, int u, const Turn* turn) {
    const int first = INTERLEAVED ? 2 * u : u, second = INTERLEAVED ? 2 * u + 1 : u + 4;
    const uint4 x0 = reinterpret_cast<const uint4*>(src)[first], x1 = reinterpret_cast<const uint4*>(src)[second];
    const __nv_bfloat162* a = reinterpret_cast<const __nv_bfloat162*>(&x0);
    const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(&x1);
    uint4 y0, y1;
    __nv_bfloat162* ya = reinterpret_cast<__nv_bfloat162*>(&y0);
    __nv_bfloat162* yb = reinterpret_cast<__nv_bfloat162*>(&y1);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 fa = __bfloat1622float2(a[k]), fb = __bfloat1622float2(b[k]);
        if constexpr (INTERLEAVED) {            // fa, fb are pairs 8u + k and 8u + 4 + k
            const Turn t = turn[8 * u + k], v = turn[8 * u + 4 + k];
            ya[k] = __floats2bfloat162_rn(fa.x * t.c - fa.y * t.s, fa.x * t.s + fa.y * t.c);
            yb[k] = __floats2bfloat162_rn(fb.x * v.c - fb.y * v.s, fb.x * v.s + fb.y * v.c);
        } else {                                // pairs 8u + 2k and 8u + 2k + 1
            const Turn t = turn[8 * u + 2 * k], v = turn[8 * u + 2 * k + 1];
            ya[k] = __floats2bfloat162_rn(fa.x * t.c - fb.x * t.s, fa.y * v.c - fb.y * v.s);
            yb[k] = __floats2bfloat162_rn(fa.x * t.s + fb.x * t.c, fa.y * v.s + fb.y * v.c);
        }
    }
    reinterpret_cast<uint4*>(dst)[first] = y0;
    reinterpret_cast<uint4*>(dst)[second] = y1;
}

// TOK tokens a block.
template <int TOK, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) append_kernel(const LatentAppendArgs a) {
    __shared__ int64_t row_s[TOK], pos_s[TOK];
    __shared__ int live_s[TOK];
    __shared__ Turn turn_s[TOK][kRope / 2];
    const int tid = threadIdx.x;
    const int64_t t0 = (int64_t)blockIdx.x * TOK;
    const int count = (int)(a.total_tokens - t0 < TOK ? a.total_tokens - t0 : TOK);
    const int width = kLatent + a.c.rope_dim;
    const int64_t cache_rows = (int64_t)a.c.num_pages * a.c.page_size;
    if (tid < count) {
        int64_t b, e;
        const int n = find_seq(a.cu_seqlens, a.num_seqs, a.total_tokens, t0 + tid, b, e);
        const int64_t p = n < 0 ? 0 : (int64_t)clamped_len(a.c, a.seq_lens, n) - (e - (t0 + tid));
        live_s[tid] = n >= 0;
        pos_s[tid] = p;
        row_s[tid] = n < 0 ? -1 : cache_row(a.c, n, p);
    }
    __syncthreads();
    if (a.inv_freq) {
        for (int i = tid; i < count * (kRope / 2); i += kThreads) {
            const int j = i / (kRope / 2), k = i % (kRope / 2);
            const double turns = (double)pos_s[j] * ((double)a.inv_freq[k] * 0.15915494309189533577);  // 1 / 2 pi
            const float x = (float)(turns - rint(turns));
            Turn t;
            sincospif(2.f * x, &t.s, &t.c);
            turn_s[j][k] = t;
        }
    } else {
        for (int i = tid; i < count * (kRope / 2); i += kThreads)
            turn_s[i / (kRope / 2)][i % (kRope / 2)] = Turn{1.f, 0.f};
    }
    __nv_bfloat16* cache = static_cast<__nv_bfloat16*>(a.c.cache);
    constexpr int kChunks = kLatent / 8;
    for (int i = tid; i < count * kChunks; i += kThreads) {
        const int j = i / kChunks, k = i % kChunks;
        if (row_s[j] < 0 || !KDA_INDEX_OK(row_s[j], cache_rows, a.status)) continue;
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.latent) + (t0 + j) * a.latent_stride;
        reinterpret_cast<uint4*>(cache + row_s[j] * width)[k] = reinterpret_cast<const uint4*>(src)[k];
    }
    if (!a.c.rope_dim) return;
    __syncthreads();
    for (int i = tid; i < count * 4; i += kThreads) {
        const int j = i >> 2, u = i & 3;
        if (row_s[j] < 0 || !KDA_INDEX_OK(row_s[j], cache_rows, a.status)) continue;
        rotate_unit<INTERLEAVED>(static_cast<const __nv_bfloat16*>(a.k_rope) + (t0 + j) * a.k_rope_stride,
                                 cache + row_s[j] * width + kLatent, u, turn_s[j]);
    }
    if (!a.q_rope) return;
    const int units = 4 * a.H;
#pragma unroll 4
    for (int i = tid; i < count * units; i += kThreads) {
        const int j = i / units, r = i - j * units, h = r >> 2, u = r & 3;
        if (!live_s[j]) continue;
        const int64_t row = (t0 + j) * a.H + h;
        rotate_unit<INTERLEAVED>(static_cast<const __nv_bfloat16*>(a.q_rope) + row * a.q_stride,
                                 static_cast<__nv_bfloat16*>(a.q_out) + row * a.q_out_stride, u, turn_s[j]);
    }
}

// ROWS rows a block, a 16-byte chunk a thread and step, all of a thread's loads before its stores.
template <int ROWS, int CHUNKS>
__global__ void __launch_bounds__(kThreads) gather_kernel(const LatentGatherArgs a) {
    __shared__ int64_t row_s[ROWS];             // -1: zeros, -2: no sequence's
    const int tid = threadIdx.x;
    const int64_t t0 = (int64_t)blockIdx.x * ROWS;
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
            x[k] = __ldg(cache + row_s[j] * CHUNKS + c);
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

template <int TOK>
void append(const LatentAppendArgs& a, cudaStream_t s) {
    const unsigned blocks = (unsigned)((a.total_tokens + TOK - 1) / TOK);
    if (a.interleaved)
        append_kernel<TOK, true><<<blocks, kThreads, 0, s>>>(a);
    else
        append_kernel<TOK, false><<<blocks, kThreads, 0, s>>>(a);
}

template <int ROWS>
void gather(const LatentGatherArgs& a, cudaStream_t s) {
    const unsigned blocks = (unsigned)((a.total_tokens + ROWS - 1) / ROWS);
    if (a.c.rope_dim)
        gather_kernel<ROWS, (kLatent + kRope) / 8><<<blocks, kThreads, 0, s>>>(a);
    else
        gather_kernel<ROWS, kLatent / 8><<<blocks, kThreads, 0, s>>>(a);
}

}  // namespace

cudaError_t launch_latent_append(const LatentAppendArgs& a, cudaStream_t s) {
    if (a.total_tokens < 2048)
        append<1>(a, s);
    else
        append<8>(a, s);
    return cudaGetLastError();
}

cudaError_t launch_latent_gather(const LatentGatherArgs& a, cudaStream_t s) {
    if (a.total_tokens < 8192)
        gather<4>(a, s);
    else
        gather<32>(a, s);
    return cudaGetLastError();
}

}  // namespace kda
