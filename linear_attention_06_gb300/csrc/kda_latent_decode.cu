// kda_latent_decode.cu -- absorbed latent attention over the paged cache (kda_latent_decode).
//
// First form: one block per (sequence, token, head), its warps taking every eighth cached row with a
// softmax of their own, joined at the end.  Right for every shape; it reads the cache once a head.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kda_internal.h"
#include "kda_latent_common.cuh"

namespace kda {
namespace {

using namespace latent;

constexpr int kThreads = 256, kWarps = kThreads / 32;

__global__ void __launch_bounds__(kThreads) decode_simple_kernel(const LatentDecodeArgs a) {
    __shared__ float acc_s[kWarps][kLatent];
    __shared__ float m_s[kWarps], l_s[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * a.H + blockIdx.y;
    const int n = blockIdx.x / a.tokens_per_seq, t = blockIdx.x % a.tokens_per_seq;
    const int seen = clamped_len(a.c, a.seq_lens, n) - a.tokens_per_seq + 1 + t;
    const int width = kLatent + a.c.rope_dim, steps = width / 32;
    float q[18], acc[16];
    for (int k = 0; k < 16; ++k) {
        acc[k] = 0.f;
        q[k] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.q_latent)[row * kLatent + k * 32 + lane]);
    }
    for (int k = 16; k < steps; ++k)
        q[k] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.q_rope)[row * kRope + (k - 16) * 32 + lane]);
    float m = -INFINITY, l = 0.f;
    for (int p = warp; p < seen; p += kWarps) {
        const int64_t r = cache_row(a.c, n, p);
        const __nv_bfloat16* c = static_cast<const __nv_bfloat16*>(a.c.cache) + r * width;
        float x[18], s = 0.f;
        for (int k = 0; k < steps; ++k) {
            x[k] = r < 0 ? 0.f : __bfloat162float(c[k * 32 + lane]);
            s += x[k] * q[k];
        }
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        s *= a.scale;
        const float mn = fmaxf(m, s), f = expf(m - mn), w = expf(s - mn);
        l = l * f + w;
        for (int k = 0; k < 16; ++k) acc[k] = acc[k] * f + w * x[k];
        m = mn;
    }
    for (int k = 0; k < 16; ++k) acc_s[warp][k * 32 + lane] = acc[k];
    if (lane == 0) { m_s[warp] = m; l_s[warp] = l; }
    __syncthreads();
    float mx = -INFINITY, sum = 0.f;
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, m_s[w]);
    for (int w = 0; w < kWarps; ++w) sum += m_s[w] == -INFINITY ? 0.f : l_s[w] * expf(m_s[w] - mx);
    for (int i = threadIdx.x; i < kLatent; i += kThreads) {
        float o = 0.f;
        for (int w = 0; w < kWarps; ++w) o += m_s[w] == -INFINITY ? 0.f : acc_s[w][i] * expf(m_s[w] - mx);
        static_cast<__nv_bfloat16*>(a.out)[row * kLatent + i] = __float2bfloat16_rn(seen > 0 ? o / sum : 0.f);
    }
    if (a.lse && threadIdx.x == 0) a.lse[row] = seen > 0 ? mx + logf(sum) : -INFINITY;
}

}  // namespace

size_t latent_decode_workspace_bytes(int, int) { return 256; }

cudaError_t launch_latent_decode(const LatentDecodeArgs& a, cudaStream_t s) {
    decode_simple_kernel<<<dim3((unsigned)(a.num_seqs * a.tokens_per_seq), (unsigned)a.H), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace kda
