// kda_latent_line.cuh -- what the latent decodes share, whatever their cache holds: all sequences' tiles in one line, cut
// into equal runs, one for each block; the partial results that pieces of sequences leave in the workspace, and the kernel
// that joins them.  Internal to a translation unit.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "kda_internal.h"
#include "kda_latent_common.cuh"
#include "kda_latent_runs.h"
#include "sm103_primitives.cuh"

namespace kda {
namespace {

using namespace latent;
using namespace sm103;

constexpr int kSMs = 152;
constexpr uint64_t kWaitNs = 4000000000ull;   // bound of every wait

// Position in a ring of SLOTS slots; `phase` flips each time round.
template <uint32_t SLOTS>
struct Ring {
    uint32_t slot = 0, phase = 0;
    __device__ __forceinline__ void next() {
        if (++slot == SLOTS) { slot = 0; phase ^= 1u; }
    }
};

// A block's run, in shared memory.
struct Line {
    int seq0, off0, lead0, len0, runs;
    int64_t total, begin, end;
};

// Walks the sequences of this block's run; every role walks by itself.
template <int TILE, int START>
struct WalkOf : RunWalkOf<TILE, START> {
    __device__ WalkOf(const Line* sw) : RunWalkOf<TILE, START>{sw->seq0, sw->off0, sw->lead0, sw->len0, sw->end - sw->begin} {}
    __device__ __forceinline__ bool next(const LatentDecodeArgs& a, Piece& p) {
        return RunWalkOf<TILE, START>::next(a.num_seqs, [&](int seq) { return clamped_len(a.c, a.seq_lens, seq); }, p);
    }
};

// A converged warp waits, and agrees on whether all its lanes saw the phase end in time.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_parked(bar, parity, kWaitNs));
}
// Workspace: a header a block (the sequence whose first piece it holds), then per (block, 0 or 1) and row the
// maximum (in log2) and the sum, then O.
struct Head {
    int n, parts, first_slot, pad;            // n = -1: none
};
// Whether a block's shared memory does not start at a multiple of 1024 bytes, as its declaration says and swizzled tiles
// need.  Such a block computes nothing: it reports itself, and leaves the join, which reads every block's header, one that
// names no sequence.  (With -DKDA_TEST_MISALIGNED every block is taken for one, to test just that.)
__device__ __forceinline__ bool misaligned(const void* sm, const LatentDecodeArgs& a) {
#ifndef KDA_TEST_MISALIGNED
    if ((smem_u32(sm) & 1023u) == 0) return false;
#endif
    wait_before();                            // the call before may still read its headers there
    if (threadIdx.x == 0) {
        reinterpret_cast<Head*>(a.workspace)[blockIdx.x] = Head{-1, 0, 0, 0};
        atomicOr(a.status, kStatusTimeout);
    }
    return true;
}
template <int NR>
struct Work {
    static __host__ __device__ size_t ml_at(int grid) { return ((size_t)grid * sizeof(Head) + 255) / 256 * 256; }
    static __host__ __device__ size_t o_at(int grid) {
        return ml_at(grid) + ((size_t)grid * 2 * NR * sizeof(float2) + 255) / 256 * 256;
    }
    static __host__ __device__ size_t bytes(int grid) { return o_at(grid) + (size_t)grid * 2 * NR * kLatent * sizeof(float); }
};

// All threads: the run of this block and the sequence it starts in.  Rounds of a sequence a thread; with up to
// THREADS sequences the lengths are read once.  Sequences of at most SHORT tiles are not cut, if runs have two places or
// more: the cut goes to the nearer end.
template <int TILE, int START, int SHORT, int THREADS>
__device__ void find_run(const LatentDecodeArgs& a, int runs, int p, Line* sw, int64_t* scratch) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int len = 0;
    auto tiles_at = [&](int n) {
        if (n >= a.num_seqs) return 0;
        len = clamped_len(a.c, a.seq_lens, n);
        return START + tiles_of<TILE>(len);
    };
    // the round's places before this thread's sequence, and in all
    auto scan = [&](int mine, int64_t& round) {
        int part = mine;                      // a warp's sum stays below 2^31: 32 sequences of at most 2^25 + START places
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, part, o);
            if (lane >= o) part += y;
        }
        if (lane == 31) scratch[warp] = part;
        __syncthreads();
        int64_t x = part;
        round = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) {
            const int64_t other = scratch[w];
            if (w < warp) x += other;
            round += other;
        }
        if (a.num_seqs > THREADS) __syncthreads();                   // scratch is written again
        return x - mine;
    };
    int mine = tiles_at(tid);
    int64_t round, at = scan(mine, round);
    int mine_len = len;
    int64_t total = round;
    for (int n0 = THREADS; n0 < a.num_seqs; n0 += THREADS) {
        int64_t more;
        scan(tiles_at(n0 + tid), more);
        total += more;
    }
    // with fewer places than blocks the first blocks take one each: a sequence's runs are consecutive
    if (total < runs) runs = (int)total;
    const bool spare = total < 2 * (int64_t)runs;
    const int64_t begin = p < runs ? run_begin(total, runs, p) : 0, end = p < runs ? run_begin(total, runs, p + 1) : 0;
    if (tid == 0) {
        sw->runs = runs;
        sw->total = total;
        if (p >= runs) sw->begin = sw->end = 0;
        if (end == total) sw->end = total;
    }
    int64_t before = 0;                       // places of the rounds before
    for (int n0 = 0; p < runs;) {
        const int64_t first = before + at;
        // where a cut at place x of this thread's sequence goes
        auto cut = [&](int64_t x) {
            if (spare || mine > START + SHORT) return x;
            return x - first <= first + mine - x ? first : first + mine;
        };
        if (mine > 0 && first <= begin && begin < first + mine) {
            const int64_t x = cut(begin);
            const int into = (int)(x - first);
            const bool next = into == mine;   // the run starts with the next sequence
            sw->begin = x;
            sw->seq0 = n0 + tid + (next ? 1 : 0);
            sw->off0 = next || into < START ? 0 : into - START;
            sw->lead0 = next ? START : (into < START ? START - into : 0);
            sw->len0 = next ? -1 : mine_len;
        }
        if (mine > 0 && end < total && first <= end && end < first + mine) sw->end = cut(end);
        before += round;
        n0 += THREADS;
        if (before > end || n0 >= a.num_seqs) break;                 // uniform
        mine = tiles_at(n0 + tid);
        mine_len = len;
        at = scan(mine, round);
    }
}

// Joins the pieces of the sequences that several runs share: out = sum_i w_i O_i / sum_i w_i l_i with
// w_i = 2^{m_i - max m}, the pieces in order.  Where a sequence has up to 32 pieces, a warp takes a quarter row (a
// float4 a lane) with eight pieces' loads in flight; where it has more, a block takes an eighth (a float2 a lane), its
// warps every eighth piece, in one round of loads for a sequence over the whole card: the rounds' latency is all that
// such a join takes (9000 cycles in three rounds, 41.5 us of a call; 6400 in one).
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32, kFewParts = 32, kMostParts = 256, kMostGrid = kJoinThreads,
              kJoinBlocks = 2 * kSMs, kBatch = 20;
template <int NR>
__global__ void __launch_bounds__(kJoinThreads, 2) latent_join_kernel(const LatentDecodeArgs a, const int grid, const int groups) {
    __shared__ Head heads_s[kMostGrid];
    __shared__ int list_s[2][kMostGrid], count_s[2][kJoinWarps];
    __shared__ float w_s[kMostParts], total_s, max_s;
    __shared__ float2 acc_s[kJoinWarps][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint8_t* ws = static_cast<const uint8_t*>(a.workspace);
    const float2* ml = reinterpret_cast<const float2*>(ws + Work<NR>::ml_at(grid));
    const float4* po = reinterpret_cast<const float4*>(ws + Work<NR>::o_at(grid));
    const int R = a.tokens_per_seq * a.H;
    allow_next();
    wait_before();
    // the sequences to join, of few pieces and of many, each in the order of their blocks: every block of this
    // kernel makes the same lists
    const Head mine = tid < grid ? reinterpret_cast<const Head*>(ws)[tid] : Head{-1, 0, 0, 0};
    const bool few = mine.n >= 0 && mine.parts <= kFewParts, many = mine.n >= 0 && mine.parts > kFewParts;
    const uint32_t fm = __ballot_sync(0xffffffffu, few), mm = __ballot_sync(0xffffffffu, many);
    heads_s[tid] = mine;
    if (lane == 0) { count_s[0][warp] = __popc(fm); count_s[1][warp] = __popc(mm); }
    __syncthreads();
    int at[2] = {0, 0}, count[2] = {0, 0};
    for (int w = 0; w < kJoinWarps; ++w)
        for (int k = 0; k < 2; ++k) {
            if (w < warp) at[k] += count_s[k][w];
            count[k] += count_s[k][w];
        }
    const uint32_t below = (1u << lane) - 1;
    if (few) list_s[0][at[0] + __popc(fm & below)] = tid;
    if (many) list_s[1][at[1] + __popc(mm & below)] = tid;
    __syncthreads();
    // task t of a list: the sequence's first block, its row and the part of it
    struct Task {
        Head h;
        int block, r, side;
        int64_t row;
        bool live;
    };
    auto task = [&](int kind, int t) {
        const int sides = kind ? 8 : 4;
        Task x;
        x.block = list_s[kind][t / (sides * NR)];
        x.r = (t / sides) % NR;
        x.side = t % sides;
        x.h = heads_s[x.block];
        const int q = (x.block % groups) * NR + x.r;
        x.row = (int64_t)x.h.n * R + q;
        x.live = q < R;
        return x;
    };
    auto slot = [&](const Task& x, int i) { return ((int64_t)(x.block + i * groups) * 2 + (i == 0 ? x.h.first_slot : 0)) * NR + x.r; };
    auto part2 = [&](const Task& x, int i) {
        return reinterpret_cast<const float2*>(po)[slot(x, i) * (kLatent / 2) + x.side * 32 + lane];
    };
    auto store_lse = [&](const Task& x, float mx, float total) {
        if (a.lse && x.side == 0 && lane == 0)
            a.lse[x.row] = total == 0.f ? -INFINITY : (mx + log2f(total)) * 0.69314718055994530942f;
    };
    auto add = [](float4& acc, float w, float4 x) {
        acc.x += w * x.x; acc.y += w * x.y; acc.z += w * x.z; acc.w += w * x.w;
    };
    // The few pieces of a sequence's row: QUARTERS quarters of it, BATCH pieces' loads in flight; the same sums in the same
    // order for every split.
    auto join_few = [&](auto quarters_c, auto batch_c) {
        constexpr int QUARTERS = decltype(quarters_c)::value, BATCH = decltype(batch_c)::value;
        for (int t = warp * gridDim.x + blockIdx.x; t < count[0] * NR * 4 / QUARTERS; t += gridDim.x * kJoinWarps) {
            const Task x = task(0, t * QUARTERS);
            if (!x.live) continue;
            const float2 y = lane < x.h.parts ? ml[slot(x, lane)] : make_float2(-INFINITY, 0.f);
            float4 o[BATCH][QUARTERS], acc[QUARTERS];
            auto load = [&](int i) {
#pragma unroll
                for (int k = 0; k < BATCH; ++k)
#pragma unroll
                    for (int q = 0; q < QUARTERS; ++q)
                        if (i + k < x.h.parts) o[k][q] = po[slot(x, i + k) * (kLatent / 4) + (x.side + q) * 32 + lane];
            };
            load(0);                          // the first loads go out before the weights are known
            float mx = y.x;
            for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            const float w = y.x == -INFINITY ? 0.f : exp2_fast(y.x - mx);
            float total = w * y.y;
            for (int d = 16; d; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
#pragma unroll
            for (int q = 0; q < QUARTERS; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int i = 0; i < x.h.parts; i += BATCH) {
                if (i > 0) load(i);
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const float wk = __shfl_sync(0xffffffffu, w, (i + k) & 31);
#pragma unroll
                    for (int q = 0; q < QUARTERS; ++q)
                        if (i + k < x.h.parts) add(acc[q], wk, o[k][q]);
                }
            }
            if (KDA_INDEX_OK(x.row, (int64_t)a.num_seqs * R, a.status)) {
                const float f = total == 0.f ? 0.f : 1.f / total;
#pragma unroll
                for (int q = 0; q < QUARTERS; ++q) {
                    uint2 v;
                    v.x = pack_bf16x2(acc[q].x * f, acc[q].y * f);
                    v.y = pack_bf16x2(acc[q].z * f, acc[q].w * f);
                    reinterpret_cast<uint2*>(a.out)[x.row * (kLatent / 4) + (x.side + q) * 32 + lane] = v;
                }
                store_lse(x, mx, total);
            }
        }
    };
    using std::integral_constant;
    // Up to two rounds of the card's warps quarter rows, dealt to all blocks before a block gets a second one; above that
    // whole rows, in one round of loads for four pieces.  (bf16, n sequences of up to 8192, 64 heads: 10 take 33.8 us, 37.2
    // with whole rows; 16 44.8, 46.2; 20, the first above the edge, 49.2, 50.9 with quarters of a block's warps side by side;
    // 64 sequences, 32 heads, 69.3 us, 71.3 with quarters.)
    if (count[0] * NR * 4 <= 2 * (int)gridDim.x * kJoinWarps)
        join_few(integral_constant<int, 1>(), integral_constant<int, 8>());
    else
        join_few(integral_constant<int, 4>(), integral_constant<int, 4>());
    for (int t = blockIdx.x; t < count[1] * NR * 8; t += gridDim.x) {
        const Task x = task(1, t);
        if (!x.live) continue;                // uniform
        const int parts = x.h.parts < kMostParts ? x.h.parts : kMostParts;
        float2 o[kBatch], y[kMostParts / 32], acc = make_float2(0.f, 0.f);
        if (warp == 0) {
#pragma unroll
            for (int k = 0; k < kMostParts / 32; ++k)
                y[k] = lane + 32 * k < parts ? ml[slot(x, lane + 32 * k)] : make_float2(-INFINITY, 0.f);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (warp + k * kJoinWarps < parts) o[k] = part2(x, warp + k * kJoinWarps);
        if (warp == 0) {
            float mx = -INFINITY, sum = 0.f;
#pragma unroll
            for (int k = 0; k < kMostParts / 32; ++k) mx = fmaxf(mx, y[k].x);
            for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
#pragma unroll
            for (int k = 0; k < kMostParts / 32; ++k) {
                const float w = y[k].x == -INFINITY ? 0.f : exp2_fast(y[k].x - mx);
                w_s[lane + 32 * k] = w;
                sum += w * y[k].y;
            }
            for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            if (lane == 0) { total_s = sum; max_s = mx; }
        }
        __syncthreads();
        for (int i = warp; i < parts; i += kBatch * kJoinWarps) {
            if (i > warp) {
#pragma unroll
                for (int k = 0; k < kBatch; ++k)
                    if (i + k * kJoinWarps < parts) o[k] = part2(x, i + k * kJoinWarps);
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (i + k * kJoinWarps < parts) {
                    const float w = w_s[i + k * kJoinWarps];
                    acc.x += w * o[k].x;
                    acc.y += w * o[k].y;
                }
        }
        acc_s[warp][lane] = acc;
        __syncthreads();
        if (warp == 0 && KDA_INDEX_OK(x.row, (int64_t)a.num_seqs * R, a.status)) {
            for (int k = 1; k < kJoinWarps; ++k) {
                acc.x += acc_s[k][lane].x;
                acc.y += acc_s[k][lane].y;
            }
            const float f = total_s == 0.f ? 0.f : 1.f / total_s;
            reinterpret_cast<uint32_t*>(a.out)[x.row * (kLatent / 2) + x.side * 32 + lane] = pack_bf16x2(acc.x * f, acc.y * f);
            store_lse(x, max_s, total_s);
        }
        __syncthreads();
    }
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

// Query rows a block takes: the smallest of 16, 32, 64 that holds them all, else 64 in several groups.
int rows_a_block(int R) { return R <= 16 ? 16 : (R <= 32 ? 32 : 64); }
int groups_of(int R) { return (R + rows_a_block(R) - 1) / rows_a_block(R); }
int runs_of(int groups) { return groups < kSMs ? kSMs / groups : 1; }

inline size_t line_workspace_bytes(int tokens_per_seq, int H) {
    const int R = tokens_per_seq * H, groups = groups_of(R), grid = runs_of(groups) * groups;
    if (runs_of(groups) == 1) return Work<64>::ml_at(grid);         // one run: no piece goes to the workspace (settle)
    switch (rows_a_block(R)) {
        case 16: return Work<16>::bytes(grid);
        case 32: return Work<32>::bytes(grid);
        default: return Work<64>::bytes(grid);
    }
}

}  // namespace
}  // namespace kda
