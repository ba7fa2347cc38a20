// kda_latent_common.cuh -- what the latent-attention kernels share: sequence bounds of a packed
// batch and the paged cache's row lookup.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_internal.h"

namespace kda {
namespace latent {

constexpr int kLatent = 512;   // channels of the latent (the cache row's first part)
constexpr int kRope = 64;      // channels of the rotated part, where there is one
constexpr int kHead = 128;     // per-head channels of the expanded form

// A kernel launched with launch_overlapped may start while the kernel before it in the stream still runs; nothing
// of that kernel, and of all before it, may be read or overwritten until wait_before().  allow_next() lets the next
// such kernel start; it waits in the same way, so a kernel that calls both keeps the order of all memory.
__device__ __forceinline__ void wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void allow_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <typename... Params, typename... Args>
cudaError_t launch_overlapped(void (*kernel)(Params...), unsigned blocks, unsigned threads, size_t smem, cudaStream_t s,
                              const Args&... args) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// 2^x by the special function unit (2 units in the last place; results below 2^-126 become zero).
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Tokens [b, e) of sequence n; a table's offsets are clamped into [0, total] and a reversed range
// is empty, so that no table leads outside the batch.
__device__ __forceinline__ void bounds(const int32_t* cu, int n, int num_seqs, int64_t total, int64_t& b, int64_t& e) {
    if (cu) {
        b = cu[n];
        e = cu[n + 1];
        b = b < 0 ? 0 : (b > total ? total : b);
        e = e < b ? b : (e > total ? total : e);
    } else {
        const int64_t each = total / num_seqs;
        b = n * each;
        e = b + each;
    }
}

// The sequence that token t of a packed batch belongs to, with its bounds; -1 if none does.
__device__ __forceinline__ int find_seq(const int32_t* cu, int num_seqs, int64_t total, int64_t t, int64_t& b,
                                        int64_t& e) {
    int n;
    if (cu) {
        int lo = 0, hi = num_seqs;              // the last n with cu[n] <= t (empty sequences before it are passed)
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if ((int64_t)cu[mid] <= t) lo = mid; else hi = mid;
        }
        n = lo;
    } else {
        n = (int)(t / (total / num_seqs));
    }
    bounds(cu, n, num_seqs, total, b, e);
    return t >= b && t < e ? n : -1;
}

// The cache row (page * page_size + offset) of position p of sequence n; -1 outside the table or the cache.
__device__ __forceinline__ int64_t cache_row(const LatentCache& c, int n, int64_t p) {
    if (p < 0 || p >= (int64_t)c.max_pages * c.page_size) return -1;
    const int shift = 31 - __clz(c.page_size);  // a power of two
    const int page = c.block_table[(int64_t)n * c.max_pages + (p >> shift)];
    if (page < 0 || page >= c.num_pages) return -1;
    return ((int64_t)page << shift) + (p & (c.page_size - 1));
}

__device__ __forceinline__ int clamped_len(const LatentCache& c, const int32_t* seq_lens, int n) {
    const int64_t most = (int64_t)c.max_pages * c.page_size;
    const int64_t len = seq_lens[n];
    return (int)(len < 0 ? 0 : (len > most ? most : len));
}

}  // namespace latent
}  // namespace kda
