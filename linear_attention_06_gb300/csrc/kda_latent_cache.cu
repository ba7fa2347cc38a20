// kda_latent_cache.cu -- the latent cache of kda.h: rows in (with the position rotation) and rows out.
//
// Append, token t at position p:  cache[row(p)] = [ c_t | R(p) r_t ],  q'_th = R(p) q_th.
// Gather:                         c_t, r_t = cache[row(p)].
// Both move every byte once and compute next to nothing, so memory bounds them (and, for a step of
// few tokens, the launch and two dependent loads: the sequence's bounds, then the page).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_internal.h"
#include "kda_latent_common.cuh"
#include "kda_latent_turn.cuh"

namespace kda {
namespace {

using namespace latent;

constexpr int kThreads = 256;

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
        step_s[k] = share_of_turn(a.inv_freq[k]);
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
            turn_s[j][k] = turn_at(pos_s[j], step_s[k]);
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
