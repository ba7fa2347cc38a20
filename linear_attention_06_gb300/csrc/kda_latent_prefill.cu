// kda_latent_prefill.cu -- expanded latent attention over packed sequences (kda_latent_prefill).
//
// First form: one block per (query, head), its warps taking every fourth key with a softmax of their
// own, joined at the end.  Right for every shape; it reads the keys once a query.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kda_internal.h"
#include "kda_latent_common.cuh"

namespace kda {
namespace {

using namespace latent;

constexpr int kThreads = 128, kWarps = kThreads / 32;

__global__ void __launch_bounds__(kThreads) prefill_simple_kernel(const LatentPrefillArgs a) {
    __shared__ float acc_s[kWarps][kHead];
    __shared__ float m_s[kWarps], l_s[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = blockIdx.x;
    const int h = blockIdx.y;
    int64_t qb, qe, kb, ke;
    const int n = find_seq(a.cu_q, a.num_seqs, a.total_q, t, qb, qe);
    if (n < 0) return;
    bounds(a.cu_k, n, a.num_seqs, a.total_kv, kb, ke);
    const int64_t seen = (ke - kb) - (qe - qb) + (t - qb) + 1;
    const int64_t row = t * a.H + h;
    const int steps = a.dk / 32;
    float q[6], acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < steps; ++k)
        q[k] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[row * a.dk + k * 32 + lane]);
    float m = -INFINITY, l = 0.f;
    for (int64_t p = warp; p < seen; p += kWarps) {
        const __nv_bfloat16* k_row = static_cast<const __nv_bfloat16*>(a.k) + ((kb + p) * a.H + h) * a.kv_stride;
        const __nv_bfloat16* v_row = static_cast<const __nv_bfloat16*>(a.v) + ((kb + p) * a.H + h) * a.kv_stride;
        float s = 0.f;
        for (int k = 0; k < 4; ++k) s += q[k] * __bfloat162float(k_row[k * 32 + lane]);
        for (int k = 4; k < steps; ++k)
            s += q[k] * __bfloat162float(
                            static_cast<const __nv_bfloat16*>(a.k_rope)[(kb + p) * kRope + (k - 4) * 32 + lane]);
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        s *= a.scale;
        const float mn = fmaxf(m, s), f = expf(m - mn), w = expf(s - mn);
        l = l * f + w;
        for (int k = 0; k < 4; ++k) acc[k] = acc[k] * f + w * __bfloat162float(v_row[k * 32 + lane]);
        m = mn;
    }
    for (int k = 0; k < 4; ++k) acc_s[warp][k * 32 + lane] = acc[k];
    if (lane == 0) { m_s[warp] = m; l_s[warp] = l; }
    __syncthreads();
    float mx = -INFINITY, sum = 0.f;
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, m_s[w]);
    for (int w = 0; w < kWarps; ++w) sum += m_s[w] == -INFINITY ? 0.f : l_s[w] * expf(m_s[w] - mx);
    float o = 0.f;
    for (int w = 0; w < kWarps; ++w) o += m_s[w] == -INFINITY ? 0.f : acc_s[w][threadIdx.x] * expf(m_s[w] - mx);
    static_cast<__nv_bfloat16*>(a.out)[row * kHead + threadIdx.x] = __float2bfloat16_rn(seen > 0 ? o / sum : 0.f);
    if (a.lse && threadIdx.x == 0) a.lse[row] = seen > 0 ? mx + logf(sum) : -INFINITY;
}

}  // namespace

cudaError_t launch_latent_prefill(const LatentPrefillArgs& a, cudaStream_t s) {
    prefill_simple_kernel<<<dim3((unsigned)a.total_q, (unsigned)a.H), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace kda
