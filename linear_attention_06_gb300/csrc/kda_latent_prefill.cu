// kda_latent_prefill.cu -- expanded latent attention over packed sequences (kda_latent_prefill).
//
// For one head and query i of a sequence with nq queries and nk keys, over the keys j <= nk - nq + i:
//
//     s_ij = scale (q_i[:128] . k_j + q_i[128:] . r_j),   o_i = sum_j e^{s_ij - m_i} v_j / sum_j e^{s_ij - m_i}.
//
// One pass over the keys with the running maximum and sum.  2 (192 + 128) flop a visible pair against 2 (128 + 128)
// bytes a key and head, read once for 256 queries: the tensor cores bound it.
//
// Block: 256 queries of one head as two tiles of 128, A and B, that take turns: while the tensor core works on
// one, eight warps turn the other's scores into weights.  Per tile of 128 keys and query tile X:
//   S_X [128 x 128]  = Q_X K^T     both from shared memory (128-byte swizzle), K = 192 or 128
//   O_X [128 x 128] += P_X V       P_X bf16 in tensor memory, over the columns that held S_X
// S_A, S_B, O_A, O_B are all of tensor memory's 512 columns, so a tile's chain (scores, weights, value product,
// next scores) cannot overlap itself: two threads share a query's row, 64 keys each, which shortens it, and hand the
// weights over in halves.  The maximum is raised only when a score exceeds it by more than 2^8 (weights stay below
// 2^8 in bf16, whose precision does not depend on the exponent; sums are fp32), so O is rarely rescaled; when it is,
// its last product is done already: S_X was issued behind it.
//
// Few queries over many keys leave SMs idle: then up to eight blocks, a cluster, take a share of the same queries' keys
// each, leave O in fp32 in their shared memory, where queries, keys and values were, and join it by reading one another's.
//
// Keys stream through a ring of 16 KB slices of 64 channels, each handed back when B's product has read it, values
// through two stages of 32 KB.
//
// Measured (GB300): 4 x 8192 tokens x 32 heads, dk = 192: 1.70 ms, 1.62 PFLOP/s, 0.93 of the sustained cuBLAS rate,
// under the power cap (1.7 GHz; 1.51 ms in a short run before it; the tensor pipe computes for 0.81 of a launch).
// dk = 128, 2 x 1024 queries over 17408 keys: 390 us, 1.45 PFLOP/s: about 2800 cycles for 2048 of products, the chain
// of one tile, and 256 blocks for 152 SMs.  A thread a query with 128 registers of scores was 1% slower in both (1.78
// against 1.76 ms, 420 against 416 us, before the last steps).
#include <atomic>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <math.h>
#include <stdint.h>
#include <type_traits>

#include "kda_internal.h"
#include "kda_latent_common.cuh"
#include "kda_latent_split.h"
#include "sm103_primitives.cuh"

namespace kda {
namespace {

using namespace latent;
using namespace sm103;

constexpr int kM = 128, kBlockQ = 2 * kM, kN = 128;   // queries a tile and a block, keys a tile
constexpr int kSoft = 256;                            // threads of a query tile: two for each query
constexpr int kThreads = 2 * kSoft + 64;              // warps 0-7: A, 8-15: B, 16: producer, 17: issuer
constexpr int64_t kKeysInL2 = (int64_t)40 << 20;      // bytes of keys and values of the heads that run together
constexpr float kRaise = 8.f;                         // log2 of how far a score may exceed the running maximum
constexpr uint64_t kWaitNs = 4000000000ull;           // bound of every wait

template <int DK>
struct Cfg {
    static constexpr uint32_t kSlices = DK / 64;                  // of queries and keys
    static constexpr uint32_t kQ = 0, kV = 2 * kSlices * 16384;   // queries [A, B][slice][128][64], values [2][2][128][64]
    static constexpr uint32_t kK = kV + 65536;
    static constexpr uint32_t kKSlots = DK == 192 ? 4 : 6;
    static constexpr uint32_t kSmall = kK + kKSlots * 16384;
    static constexpr uint32_t kBytes = kSmall + 2560;
    static_assert(kBytes <= 232448, "shared memory");
};

struct Place {                                // a block's sequence, 256 queries and head
    int n, h;
    int64_t qb, q0, kb;                       // sequence's first query, this tile's first query in it, first key
    int nq, nk;
};

struct Small {
    uint64_t q_full[2], k_full[6], k_empty[6], v_full[2], v_empty[2], s_full[2], p_half[2], p_full[2], o_done[2], drain;
    uint32_t tmem;
    int count[2];                             // key tiles of A and B, as one thread read them
    float best[2][2][kM];                     // [X][half of the keys][query]: maxima
};
static_assert(sizeof(Small) <= 2560, "small area");

struct Maps {
    CUtensorMap q, k, v, r;
};

__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) { return mbar_wait_parked(bar, parity, kWaitNs); }
// The same for a converged warp, whose lanes agree on whether all of them saw the phase end in time.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_parked(bar, parity, kWaitNs));
}

// OR of a predicate over the warps of query tile X; also a barrier between them.
__device__ __forceinline__ bool tile_or(int X, bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "bar.red.or.pred p, %2, %3, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)pred), "r"(1 + X), "n"(kSoft)
        : "memory");
    return r != 0;
}
// A barrier of both query tiles' warps.
__device__ __forceinline__ void soft_meet() { asm volatile("bar.sync 3, %0;" ::"n"(2 * kSoft) : "memory"); }
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// Two fp32 in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return d;
}

// Clusters: this block's number in its own; all threads meet, what they wrote before seen by all behind it (blocks that
// ended count as there); reads of another block's shared memory.
__device__ __forceinline__ int cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return (int)r;
}
__device__ __forceinline__ void cluster_meet() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(uint32_t smem, int rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem), "r"(rank));
    return a;
}
__device__ __forceinline__ float cluster_load(uint32_t addr) {
    float x;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
    return x;
}
__device__ __forceinline__ float4 cluster_load4(uint32_t addr) {
    float4 x;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(addr) : "memory");
    return x;
}

// The block's sequence, 256-query tile and head.  Tile slots: sequence n's start at floor(b_n / 256) + n, so that
// ceil(T / 256) + N - 1 slots hold any lengths and a block finds its own by bisection.  Heads go in groups whose keys
// stay in L2, and slots from the last (the longest rows of a sequence) down, so that the lightest end the launch.
__device__ __forceinline__ bool find_place(const LatentPrefillArgs& a, int64_t slots, int group, int64_t b, Place& x) {
    const int64_t per = slots * group;
    const int first = (int)(b / per) * group;
    const int together = a.H - first < group ? a.H - first : group;
    const int64_t rem = b % per, slot = slots - 1 - rem / together;
    x.h = first + (int)(rem % together);
    int lo = 0, hi = a.num_seqs;              // the last n whose first slot is <= slot
    auto first_slot = [&](int n) {
        int64_t s, e;
        bounds(a.cu_q, n, a.num_seqs, a.total_q, s, e);
        return s / kBlockQ + n;
    };
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first_slot(mid) <= slot) lo = mid; else hi = mid;
    }
    int64_t qe, ke;
    x.n = lo;
    bounds(a.cu_q, lo, a.num_seqs, a.total_q, x.qb, qe);
    bounds(a.cu_k, lo, a.num_seqs, a.total_kv, x.kb, ke);
    x.nq = (int)(qe - x.qb);
    x.nk = (int)(ke - x.kb);
    x.q0 = (slot - (x.qb / kBlockQ + lo)) * kBlockQ;
    return x.q0 >= 0 && x.q0 < x.nq;
}

// Key tiles that query tile X of a place looks at.
__device__ __forceinline__ int tiles_of(const Place& x, int X) {
    const int64_t first = x.q0 + X * kM;
    if (first >= x.nq) return 0;
    const int64_t last = first + kM < x.nq ? first + kM : x.nq;    // behind its last query
    const int64_t seen = (int64_t)x.nk - x.nq + last;
    return seen > 0 ? (int)((seen + kN - 1) / kN) : 0;
}

// Joins a row of the P blocks of a cluster, each with O [32 chunks of 4 channels][128 rows] in fp32 at the start of its
// shared memory (a tile's behind the other's), the row's maximum and sum in `best`.  Block `rank` joins 32 / P of the
// chunks, a thread half of those; the parts in their order, eight loads in flight.
template <int P>
__device__ __forceinline__ void join_row(const LatentPrefillArgs& a, uint32_t o, uint32_t best, int rank, int half, float c2,
                                         int64_t row, bool live) {
    constexpr int kEach = 16 / P, kAhead = 8 / P;
    float w[P], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int r = 0; r < P; ++r) {
        w[r] = cluster_load(cluster_addr(best, r));
        m = fmaxf(m, w[r]);
    }
#pragma unroll
    for (int r = 0; r < P; ++r) {
        w[r] = w[r] == -INFINITY ? 0.f : exp2_fast((w[r] - m) * c2);
        if (w[r] > 0.f) l += w[r] * cluster_load(cluster_addr(best + 4 * kM, r));
    }
    if (!live) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int first = rank * 2 * kEach + half * kEach;
    uint2* out = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + row * kHead) + first;
#pragma unroll
    for (int c = 0; c < kEach; c += kAhead) {
        float4 x[kAhead][P];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
#pragma unroll
            for (int r = 0; r < P; ++r)       // a part without weight left nothing there
                x[k][r] = w[r] > 0.f ? cluster_load4(cluster_addr(o + (first + c + k) * 16 * kM, r)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int r = 0; r < P; ++r) {
                y.x += w[r] * x[k][r].x; y.y += w[r] * x[k][r].y; y.z += w[r] * x[k][r].z; y.w += w[r] * x[k][r].w;
            }
            out[c + k] = make_uint2(pack_bf16x2(y.x * inv, y.y * inv), pack_bf16x2(y.z * inv, y.w * inv));
        }
    }
    if (a.lse && rank == 0 && half == 0) a.lse[row] = l == 0.f ? -INFINITY : m * a.scale + logf(l);
}

template <int DK, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
latent_prefill_kernel(const __grid_constant__ Maps maps, const LatentPrefillArgs a, const int64_t slots, const int group,
                      const int parts) {
    using G = Cfg<DK>;
    extern __shared__ __align__(1024) uint8_t sm[];   // swizzled tiles start at multiples of 1024 bytes
    if (smem_u32(sm) & 1023u) {               // the declaration's alignment; without it there would be no room for slack
        if (threadIdx.x == 0) atomicOr(a.status, kStatusTimeout);
        return;
    }
    Small* sw = reinterpret_cast<Small*>(sm + G::kSmall);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int rank = SPLIT ? cluster_rank() : 0;
    Place x;
    if (!find_place(a, slots, group, SPLIT ? blockIdx.x / parts : blockIdx.x, x)) {     // a slot without queries
        if (SPLIT) { cluster_meet(); cluster_meet(); }
        return;
    }
    int tiles[2] = {tiles_of(x, 0), tiles_of(x, 1)}, most = tiles[0] > tiles[1] ? tiles[0] : tiles[1];
    if (SPLIT) {                              // this block's share of the key tiles, which then are tiles 0, 1, ..
        const int from = (int)((int64_t)most * rank / parts), share = (int)((int64_t)most * (rank + 1) / parts) - from;
        most = share;
#pragma unroll
        for (int X = 0; X < 2; ++X) {
            const int left = tiles[X] - from;
            tiles[X] = left < 0 ? 0 : (left < share ? left : share);
        }
        x.kb += (int64_t)from * kN;
        x.nk -= from * kN;
    }

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sw->q_full[i], 1);
            mbar_init(&sw->v_full[i], 1);
            mbar_init(&sw->v_empty[i], 1);
            mbar_init(&sw->s_full[i], 1);
            mbar_init(&sw->p_half[i], 8);
            mbar_init(&sw->p_full[i], 8);
            mbar_init(&sw->o_done[i], 1);
        }
        for (int i = 0; i < (int)G::kKSlots; ++i) { mbar_init(&sw->k_full[i], 1); mbar_init(&sw->k_empty[i], 1); }
        mbar_init(&sw->drain, 1);
        fence_mbar_init();
        sw->count[0] = tiles[0];
        sw->count[1] = tiles[1];
    }
    if (warp == 17) {
        tmem_alloc(&sw->tmem, 512);
        tmem_relinquish();
    }
    if (warp == 16 && lane < 4) tma_prefetch_desc(lane == 0 ? &maps.q : lane == 1 ? &maps.k : lane == 2 ? &maps.v : &maps.r);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = sw->tmem;             // columns: S_A, S_B, O_A, O_B
    bool ok = true;

    if (warp == 16) {                         // ------------------------------------------------ producer
        uint32_t k_loads = 0, v_loads = 0, q_loads = 0;
        if (elect_one()) {
            auto load_k = [&](int j) {
                for (uint32_t s = 0; ok && s < G::kSlices; ++s, ++k_loads) {
                    const uint32_t slot = k_loads % G::kKSlots, round = k_loads / G::kKSlots;
                    if (round > 0 && !(ok = wait(&sw->k_empty[slot], (round - 1) & 1))) return;
                    mbar_arrive_expect_tx(&sw->k_full[slot], 16384);
                    uint8_t* dst = sm + G::kK + slot * 16384;
                    const int t = (int)x.kb + j * kN;
                    if (s < 2)
                        tma_load_3d(dst, &maps.k, s * 64, x.h, t, &sw->k_full[slot]);
                    else
                        tma_load_2d(dst, &maps.r, 0, t, &sw->k_full[slot]);
                }
            };
            auto load_q = [&](int X) {
                if (!tiles[X]) return;
                mbar_arrive_expect_tx(&sw->q_full[X], G::kSlices * 16384);
                for (uint32_t s = 0; s < G::kSlices; ++s)
                    tma_load_3d(sm + G::kQ + (X * G::kSlices + s) * 16384, &maps.q, s * 64, x.h,
                                (int)(x.qb + x.q0) + X * kM, &sw->q_full[X]);
                q_loads |= 1u << X;
            };
            load_q(0);
            if (most > 0) load_k(0);
            load_q(1);
            // values before the next keys: their stage is free long before those keys' slices
            for (int j = 0; ok && j < most; ++j) {
                if ((j > 1 && !(ok = wait(&sw->v_empty[j & 1], ((j >> 1) - 1) & 1)))) break;
                mbar_arrive_expect_tx(&sw->v_full[j & 1], 32768);
                for (int s = 0; s < 2; ++s)
                    tma_load_3d(sm + G::kV + (j & 1) * 32768 + s * 16384, &maps.v, s * 64, x.h, (int)x.kb + j * kN,
                                &sw->v_full[j & 1]);
                ++v_loads;
                if (j + 1 < most) load_k(j + 1);
            }
            if (!ok) {                        // copies in flight land before the block ends
                for (uint32_t i = 0; i < G::kKSlots; ++i)
                    if (k_loads > i) mbar_wait_bounded(&sw->k_full[i], ((k_loads - 1 - i) / G::kKSlots) & 1, kWaitNs);
                for (uint32_t i = 0; i < 2; ++i) {
                    if (v_loads > i) mbar_wait_bounded(&sw->v_full[i], ((v_loads - 1 - i) / 2) & 1, kWaitNs);
                    if (q_loads >> i & 1) mbar_wait_bounded(&sw->q_full[i], 0, kWaitNs);
                }
                atomicOr(a.status, kStatusTimeout);
            }
        }
        __syncwarp();
    } else if (warp == 17) {                  // ------------------------------------------------ issuer
        constexpr uint32_t id_s = idesc_bf16_f32(kM, kN, false, false), id_o = idesc_bf16_f32(kM, kHead, false, true);
        const uint64_t dq = smem_desc(smem_u32(sm + G::kQ), 16, 1024, kSwizzle128B);
        const uint64_t dk = smem_desc(smem_u32(sm + G::kK), 16, 1024, kSwizzle128B);
        const uint64_t dv = smem_desc(smem_u32(sm + G::kV), 16384, 1024, kSwizzle128B);
        const uint32_t el = elect_one();
        const int ta = tiles[0], tc = tiles[1];
        // the ring of key slices, as each query tile walks it
        struct Ring {
            uint32_t slot, phase;
        };
        Ring ra{0, 0}, rb{0, 0};
        // S_X of key tile j
        auto scores = [&](auto which, Ring& ring, int j) {
            constexpr int X = decltype(which)::value;
            const bool first = X == 0 || j >= ta, last = X == 1 || j >= tc;
            if (j == 0 && !(ok = wait_warp(&sw->q_full[X], 0))) return;
#pragma unroll
            for (uint32_t s = 0; s < G::kSlices; ++s) {
                const uint32_t slot = ring.slot;
                if (first && !(ok = wait_warp(&sw->k_full[slot], ring.phase))) return;
                tc_fence_after();
                const uint64_t y = desc_at(dk, slot * 16384);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mma_ss_elected(tb + X * 128, desc_at(dq, (X * G::kSlices + s) * 16384 + i * 32), desc_at(y, i * 32), id_s,
                                   s > 0 || i > 0, el);
                if (last) mma_commit_elected(&sw->k_empty[slot], el);
                if (++ring.slot == G::kKSlots) { ring.slot = 0; ring.phase ^= 1u; }
            }
            mma_commit_elected(&sw->s_full[X], el);
        };
        // O_X += P_X V of key tile j
        auto values = [&](auto which, int j) {
            constexpr int X = decltype(which)::value;
            const bool first = X == 0 || j >= ta, last = X == 1 || j >= tc;
            const uint64_t y = desc_at(dv, (j & 1) * 32768);
            if (first && !(ok = wait_warp(&sw->v_full[j & 1], (j >> 1) & 1))) return;
            // keys 0-31 and 64-95 first, then the others
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                if (!(ok = wait_warp(part ? &sw->p_full[X] : &sw->p_half[X], j & 1))) return;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int i = 2 * part + (k & 1) + 4 * (k >> 1);
                    mma_ts_elected(tb + 256 + X * 128, tb + X * 128 + i * 8, desc_at(y, i * 2048), id_o, j > 0 || i > 0, el);
                }
            }
            if (last) mma_commit_elected(&sw->v_empty[j & 1], el);
            if (j + 1 == (X ? tc : ta)) mma_commit_elected(&sw->o_done[X], el);
        };
        constexpr std::integral_constant<int, 0> A{};
        constexpr std::integral_constant<int, 1> B{};
        if (ta) scores(A, ra, 0);
        if (ok && tc) scores(B, rb, 0);
        for (int j = 0; ok && j < most; ++j) {
            if (j < ta) {
                values(A, j);
                if (ok && j + 1 < ta) scores(A, ra, j + 1);
            }
            if (ok && j < tc) {
                values(B, j);
                if (ok && j + 1 < tc) scores(B, rb, j + 1);
            }
        }
        if (!ok) {                            // products in flight land before TMEM is freed
            mma_commit_elected(&sw->drain, el);
            wait_warp(&sw->drain, 0);
            if (lane == 0) atomicOr(a.status, kStatusTimeout);
        }
    } else {                                  // ------------------------------------------------ softmax of tile X
        // warps 0-3 of a tile take the first 64 keys of each query, warps 4-7 the others
        const int X = warp >> 3, half = (warp >> 2) & 1, w = warp & 3, t = tid & 127;
        const int64_t i = x.q0 + X * kM + t;  // the thread's query in its sequence
        const int64_t seen = (int64_t)x.nk - x.nq + i + 1;
        const float c2 = a.scale * 1.44269504088896340736f;
        const uint32_t ts = tmem_addr(tb, 32 * w, X * 128), to = tmem_addr(tb, 32 * w, 256 + X * 128 + 64 * half);
        float m = -INFINITY, l = 0.f;
        // one thread's count for all: these warps meet at barriers and must agree on it, whatever a caller does to
        // the tables meanwhile
        const int count = sw->count[X];
        for (int j = 0; j < count; ++j) {
            ok = ok && wait_warp(&sw->s_full[X], j & 1);
            tc_fence_after();
            uint32_t s[2][32];
            tmem_ld32(ts + 64 * half, s[0]);
            tmem_ld32(ts + 64 * half + 32, s[1]);
            tmem_wait_ld();
            const int64_t lim = seen - (int64_t)j * kN - 64 * half;  // of these columns, those that the query sees
            if (__any_sync(0xffffffffu, lim < 64)) {
                const int edge = lim < 0 ? 0 : (lim < 64 ? (int)lim : 64);
#pragma unroll
                for (int k = 0; k < 64; ++k)
                    if (k >= edge) s[k >> 5][k & 31] = 0xff800000u;  // -inf
            }
            float part[2];                    // two chains of three-way maxima
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                part[b] = max3(__uint_as_float(s[b][0]), __uint_as_float(s[b][1]), __uint_as_float(s[b][2]));
#pragma unroll
                for (int k = 3; k < 31; k += 2)
                    part[b] = max3(part[b], __uint_as_float(s[b][k]), __uint_as_float(s[b][k + 1]));
            }
            const float mine = fmaxf(max3(part[0], part[1], __uint_as_float(s[0][31])), __uint_as_float(s[1][31]));
            // The two threads of a query exchange their maxima.  Behind the barrier every score is in registers, so
            // the weights may go over them; the slots are written again behind s_full, which waits for this tile's
            // weights.  A wait that ran out ends all of the tile's warps here
            sw->best[X][half][t] = mine;
            if (tile_or(X, !ok)) { ok = false; break; }
            const float mx = fmaxf(mine, sw->best[X][half ^ 1][t]);
            float f = 1.f;
            if (mx > m && (mx - m) * c2 > kRaise) {                  // also the first finite maximum
                f = exp2_fast((m - mx) * c2);
                m = mx;
            }
            l *= f;
            if (j > 0 && __any_sync(0xffffffffu, f != 1.f)) {        // rescale the warp's half rows of O
#pragma unroll 1
                for (int b = 0; b < 4; ++b) {
                    uint32_t o[16];
                    tmem_ld16(to + 16 * b, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                    tmem_st16(to + 16 * b, o);
                }
            }
            if ((int64_t)(j + 1) * kN > x.nk) {                      // value rows behind the sequence's end become zeros
                ok = wait_warp(&sw->v_full[j & 1], (j >> 1) & 1);
                if (ok && j * kN + t >= x.nk)
                    for (int k = 0; k < 8; ++k)
                        *reinterpret_cast<uint4*>(sm + G::kV + (j & 1) * 32768 + half * 16384 + t * 128 + k * 16) =
                            make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
            }
            const float z = m == -INFINITY ? 0.f : -m * c2;
            const float2 c22 = make_float2(c2, c2), z2 = make_float2(z, z);
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t p[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    float2 y = fma2(make_float2(__uint_as_float(s[b][2 * k]), __uint_as_float(s[b][2 * k + 1])), c22, z2);
                    y.x = exp2_fast(y.x);
                    y.y = exp2_fast(y.y);
                    sum = add2(sum, y);
                    p[k] = pack_bf16x2(y.x, y.y);
                }
                tmem_st16(ts + 32 * half + 16 * b, p);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && ok) mbar_arrive(b ? &sw->p_full[X] : &sw->p_half[X]);   // the product of half can begin
            }
            l += sum.x + sum.y;
        }
        if (count) {
            ok = ok && wait_warp(&sw->o_done[X], 0);
            float* sums = reinterpret_cast<float*>(sm + G::kQ + X * G::kSlices * 16384);   // the queries are done with
            sums[half * kM + t] = l;
            ok = !tile_or(X, !ok);
            l = sums[t] + sums[kM + t];
        }
        const int64_t row = (x.qb + i) * a.H + x.h;
        if constexpr (SPLIT) {
            // Both tiles' products are done: queries, keys and values make room for O.  After a wait that ran out the
            // part has no weight.
            const bool any = ok && count > 0;
            if (!ok && lane == 0) atomicOr(a.status, kStatusTimeout);
            soft_meet();
            tc_fence_after();
            if (any) {
                float4* o = reinterpret_cast<float4*>(sm) + (X * 32 + 16 * half) * kM + t;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    uint32_t y[32];
                    tmem_ld32(to + 32 * b, y);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        o[(8 * b + k) * kM] = make_float4(__uint_as_float(y[4 * k]), __uint_as_float(y[4 * k + 1]),
                                                          __uint_as_float(y[4 * k + 2]), __uint_as_float(y[4 * k + 3]));
                }
            }
            if (half == 0) {
                sw->best[X][0][t] = any ? m : -INFINITY;
                sw->best[X][1][t] = l;
            }
            cluster_meet();
            const bool live = i < x.nq && KDA_INDEX_OK(row, a.total_q * a.H, a.status);
            const uint32_t o = smem_u32(sm) + (X * 32 * kM + t) * 16, best = smem_u32(&sw->best[X][0][t]);
            if (parts == 2) join_row<2>(a, o, best, rank, half, c2, row, live);
            else if (parts == 4) join_row<4>(a, o, best, rank, half, c2, row, live);
            else join_row<8>(a, o, best, rank, half, c2, row, live);
            cluster_meet();                   // no block ends while another reads its memory
        } else if (ok) {                      // a thread stores half of its query's row
            tc_fence_after();
            const bool live = i < x.nq && KDA_INDEX_OK(row, a.total_q * a.H, a.status);
            const float inv = l == 0.f ? 0.f : 1.f / l;
            uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + row * kHead + 64 * half);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t o[32];
                if (count) {
                    tmem_ld32(to + 32 * b, o);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = 0u;
                }
                if (live) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint4 y;
                        y.x = pack_bf16x2(__uint_as_float(o[8 * k]) * inv, __uint_as_float(o[8 * k + 1]) * inv);
                        y.y = pack_bf16x2(__uint_as_float(o[8 * k + 2]) * inv, __uint_as_float(o[8 * k + 3]) * inv);
                        y.z = pack_bf16x2(__uint_as_float(o[8 * k + 4]) * inv, __uint_as_float(o[8 * k + 5]) * inv);
                        y.w = pack_bf16x2(__uint_as_float(o[8 * k + 6]) * inv, __uint_as_float(o[8 * k + 7]) * inv);
                        out[4 * b + k] = y;
                    }
                }
            }
            if (live && a.lse && half == 0) a.lse[row] = l == 0.f ? -INFINITY : m * a.scale + logf(l);
        } else if (lane == 0) {
            atomicOr(a.status, kStatusTimeout);
        }
    }
    if (SPLIT && warp >= 16) { cluster_meet(); cluster_meet(); }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 17) tmem_dealloc(tb, 512);
}

PFN_cuTensorMapEncodeTiled_v12000 encode() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
        return nullptr;
    }();
    return fn;
}

// [tokens, heads] rows of `width` channels, `step` elements apart; boxes of 64 channels x 1 head x 128 tokens.
bool map_heads(CUtensorMap* m, const void* base, int64_t tokens, int heads, int width, int64_t step) {
    const auto fn = encode();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)tokens};
    cuuint64_t strides[2] = {(cuuint64_t)step * 2, (cuuint64_t)step * heads * 2};
    cuuint32_t box[3] = {64, 1, 128}, es[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool map_shared(CUtensorMap* m, const void* base, int64_t tokens) {
    const auto fn = encode();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)kRope, (cuuint64_t)tokens}, strides[1] = {(cuuint64_t)kRope * 2};
    cuuint32_t box[2] = {64, 128}, es[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kDevices = 64;

// The kernel's shared memory, set once a device.
template <int DK, bool SPLIT>
cudaError_t set_up(int dev) {
    static std::atomic<bool> ready[kDevices];
    if (ready[dev].load(std::memory_order_acquire)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(latent_prefill_kernel<DK, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)Cfg<DK>::kBytes);
    if (e == cudaSuccess) ready[dev].store(true, std::memory_order_release);
    return e;
}

// A launch of `blocks` clusters of `parts` blocks; `attr` is its attribute and has to live as long.
template <int DK>
cudaLaunchConfig_t config(int64_t blocks, int parts, cudaStream_t s, cudaLaunchAttribute* attr) {
    attr->id = cudaLaunchAttributeClusterDimension;
    attr->val.clusterDim.x = (unsigned)parts;
    attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks * parts));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Cfg<DK>::kBytes;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = parts > 1 ? 1 : 0;
    return cfg;
}

// Clusters of `parts` blocks that run at the same time: what the SMs of each cluster's neighbourhood hold, which differs
// from card to card.  (Here 144 of 152 SMs in clusters of four, fewer than 128 in clusters of eight.)
template <int DK>
int clusters_at_once(int dev, int parts) {
    static std::atomic<int> known[kDevices][9];           // one more than the number; 0: not asked yet
    int n = known[dev][parts].load(std::memory_order_relaxed) - 1;
    if (n >= 0) return n;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config<DK>(1, parts, nullptr, &attr);
    if (cudaOccupancyMaxActiveClusters(&n, latent_prefill_kernel<DK, true>, &cfg) != cudaSuccess) {
        cudaGetLastError();                   // not the launch's
        return 0;
    }
    known[dev][parts].store(n + 1, std::memory_order_relaxed);
    return n;
}

// How many blocks share the keys of a block of queries: a rule on average lengths (kda_latent_split.h).  Measured, dk =
// 192: 1 x 100 queries over 16384 keys, 32 heads, 52 us in fours and 167 alone; 1 x 128 over 8192, one head, 19 in eights,
// 29 in fours, 86 alone; 1 x 64 over 600, 8 heads, 10.5 in fours and 11.4 alone; 1 x 512 without prefix, 8 heads, 12.2 in
// fours, 14.2 in twos and 12.3 alone; 1 x 200 over 4096, 18 heads, more clusters of eight than run at once 34.0, in fours
// 22.2; 4 x 512 without prefix, 4 heads, whose slots are more clusters of four than run at once, 15.6, alone 12.6.
template <int DK>
int parts_of(const LatentPrefillArgs& a, int64_t slots, int dev) {
    const int64_t each_q = (a.total_q + a.num_seqs - 1) / a.num_seqs, tiles = a.total_kv / a.num_seqs / kN;
    const int64_t busy = (each_q + kBlockQ - 1) / kBlockQ * a.num_seqs * a.H;
    return split_of(tiles, busy, slots * a.H, [&](int parts) { return clusters_at_once<DK>(dev, parts); });
}

template <int DK>
cudaError_t launch(const LatentPrefillArgs& a, cudaStream_t s) {
    Maps maps;
    // without keys nothing is loaded; the maps are then those of the queries
    const bool keys = a.total_kv > 0;
    if (!map_heads(&maps.q, a.q, a.total_q, a.H, DK, DK) ||
        !(keys ? map_heads(&maps.k, a.k, a.total_kv, a.H, kHead, a.kv_stride) : map_heads(&maps.k, a.q, a.total_q, a.H, DK, DK)) ||
        !(keys ? map_heads(&maps.v, a.v, a.total_kv, a.H, kHead, a.kv_stride) : map_heads(&maps.v, a.q, a.total_q, a.H, DK, DK)) ||
        !(keys && DK > kHead ? map_shared(&maps.r, a.k_rope, a.total_kv) : map_heads(&maps.r, a.q, a.total_q, a.H, DK, DK)))
        return cudaErrorInvalidValue;
    const int64_t slots = (a.total_q + kBlockQ - 1) / kBlockQ + a.num_seqs - 1, blocks = slots * a.H;
    // Heads run together, longest rows first, as far as the keys and values of an average sequence fit into L2, in groups
    // of one size.  All heads together end evenly, but long keys would be read from memory over and over: 1 x 2048 tokens,
    // 32 heads 37 us in one group and 46 in four; 1 x 8192 377 us in four groups, 383 in two, 436 in unequal ones;
    // 1 x 32768 5.97 ms in groups of two heads, 6.05 in groups of eight.
    const int64_t head_bytes = (a.total_kv / a.num_seqs + 1) * 2 * kHead * 2;
    const int64_t fit = kKeysInL2 > head_bytes ? kKeysInL2 / head_bytes : 1, groups = (a.H + fit - 1) / fit;
    const int group = (int)((a.H + groups - 1) / groups);            // groups of one size
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
    cudaError_t e = set_up<DK, false>(dev);
    if (e == cudaSuccess) e = set_up<DK, true>(dev);
    if (e != cudaSuccess) return e;
    const int parts = parts_of<DK>(a, slots, dev);
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = config<DK>(blocks, parts, s, &attr);
    e = cudaLaunchKernelEx(&cfg, parts > 1 ? latent_prefill_kernel<DK, true> : latent_prefill_kernel<DK, false>, maps, a, slots,
                           group, parts);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_latent_prefill(const LatentPrefillArgs& a, cudaStream_t s) {
    return a.dk == 192 ? launch<192>(a, s) : launch<128>(a, s);
}

}  // namespace kda
