// kda_latent_decode_q8.cu -- absorbed latent attention over the 8-bit paged cache (kda_latent_decode_q8).
//
// For a query row x = [q_latent | q_rope] and the cached rows y_j 2^{e_j} (the first 512 channels c_j are the values):
//
//     s_j = scale 2^{e_j} x . y_j,   p_j = e^{s_j - m},   o = sum_j p_j 2^{e_j} c_j / sum_j p_j.
//
// The plain form: a block a query row, a thread a cached row of a tile for the scores, four channels for the output.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kda_internal.h"
#include "kda_latent_common.cuh"
#include "kda_latent_q8.cuh"

namespace kda {
namespace {

using namespace latent;

constexpr int kThreads = 128;

__global__ void __launch_bounds__(kThreads) decode_q8_kernel(const LatentDecodeArgs a) {
    __shared__ float q_s[kLatent + kRope], p_s[kThreads], red_s[kThreads / 32];
    __shared__ int64_t row_s[kThreads];
    const int tid = threadIdx.x, width = kLatent + a.c.rope_dim;
    const int64_t q = blockIdx.x;
    const int R = a.tokens_per_seq * a.H, n = (int)(q / R), t = (int)(q % R) / a.H;
    for (int i = tid; i < width; i += kThreads)
        q_s[i] = __bfloat162float(i < kLatent ? static_cast<const __nv_bfloat16*>(a.q_latent)[q * kLatent + i]
                                              : static_cast<const __nv_bfloat16*>(a.q_rope)[q * kRope + i - kLatent]);
    const int seen = clamped_len(a.c, a.seq_lens, n) - a.tokens_per_seq + 1 + t;
    const uint8_t* cache = static_cast<const uint8_t*>(a.c.cache);
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    auto block_reduce = [&](float x, bool sum) {
        for (int d = 16; d; d >>= 1) {
            const float y = __shfl_xor_sync(0xffffffffu, x, d);
            x = sum ? x + y : fmaxf(x, y);
        }
        __syncthreads();
        if ((tid & 31) == 0) red_s[tid >> 5] = x;
        __syncthreads();
        x = red_s[0];
        for (int w = 1; w < kThreads / 32; ++w) x = sum ? x + red_s[w] : fmaxf(x, red_s[w]);
        return x;
    };
    for (int base = 0; base < seen; base += kThreads) {
        const int j = base + tid;
        const int64_t row = j < seen ? cache_row(a.c, n, j) : -1;
        const float f = row >= 0 ? two_to(power_of(a.c.scales[row])) : 0.f;
        float s = 0.f;
        __syncthreads();
        row_s[tid] = row;
        if (row >= 0)
            for (int i = 0; i < width; i += 4) {
                const uint32_t y = *reinterpret_cast<const uint32_t*>(cache + row * width + i);
                const float2 u = from_e4m3x2(y), v = from_e4m3x2(y >> 16);
                s += q_s[i] * u.x + q_s[i + 1] * u.y + q_s[i + 2] * v.x + q_s[i + 3] * v.y;
            }
        s = j < seen ? s * f * a.scale : -INFINITY;
        const float mx = fmaxf(m, block_reduce(s, false));
        const float p = expf(s - mx), r = expf(m - mx);
        l = l * r + block_reduce(p, true);
        p_s[tid] = p * f;
        m = mx;
        __syncthreads();
        for (int k = 0; k < 4; ++k) o[k] *= r;
        for (int i = 0; i < kThreads; ++i) {
            if (row_s[i] < 0) continue;
            const uint32_t y = *reinterpret_cast<const uint32_t*>(cache + row_s[i] * width + 4 * tid);
            const float2 u = from_e4m3x2(y), v = from_e4m3x2(y >> 16);
            o[0] += p_s[i] * u.x; o[1] += p_s[i] * u.y; o[2] += p_s[i] * v.x; o[3] += p_s[i] * v.y;
        }
    }
    const float f = l == 0.f ? 0.f : 1.f / l;
    for (int k = 0; k < 4; ++k)
        static_cast<__nv_bfloat16*>(a.out)[q * kLatent + 4 * tid + k] = __float2bfloat16_rn(o[k] * f);
    if (a.lse && tid == 0) a.lse[q] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

size_t latent_decode_q8_workspace_bytes(int, int) { return 256; }

cudaError_t launch_latent_decode_q8(const LatentDecodeArgs& a, cudaStream_t s) {
    decode_q8_kernel<<<(unsigned)(a.num_seqs * a.tokens_per_seq * a.H), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace kda
