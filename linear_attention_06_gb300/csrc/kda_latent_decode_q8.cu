// kda_latent_decode_q8.cu -- absorbed latent attention over the 8-bit paged cache (kda_latent_decode_q8).
//
// For one sequence, the R = T' H query rows x_r = [q_latent | q_rope] of its step and its cached rows y_j 2^{e_j}
// (kda_latent_q8.cuh), whose first 512 channels c_j are the values too:
//
//     s_rj = scale 2^{e_j} x_r . y_j,   o_r = sum_j p_rj 2^{e_j} c_j / sum_j p_rj,   p_rj = e^{s_rj}.
//
// The cache's bytes bound the call, half as many as in bf16, so the tile has to be multiplied as it lies in memory:
// widened to 16 bits it would move through shared memory three times more.  tcgen05 multiplies 8-bit operands; the other
// operand, where it is not 8-bit by nature, goes in as the sum of two 8-bit numbers:
//
// - A query row under a power of two, x = 2^k (x' + x''), both e4m3: eight significant bits, all of a bf16 channel, down
//   to 2^-10 of the row's largest.  x' and x'' are two rows of one operand, so that the tile is read once for both.
// - A weight w_rj = 2^{log2 p_rj + e_j - m_r} as e4m3 and, of what that leaves, 2^7 times in e4m3 with accumulators of its
//   own (up to 32 rows) or e5m2 in the same ones (64 rows, whose accumulators take all there is): 2^-9 or 2^-8 of the
//   weight (bf16: 2^-8), and steps of 2^-16 where it is faint.  The row's reference m_r is a whole number (scores near 0
//   keep their bits beside e_j, and moves are exact).  It is raised at once where a weight would pass 2^6 or 2^8.75.  It is
//   lowered where faint weights count: a token of 2^-12 is lost in silence, a thousand of them beside a few bright ones (a
//   first token that takes nearly all weight and a long flat tail behind it is what models really do) are not.  So each row
//   keeps an account of what its weights lost, |w - w' - w''|, less 2^-8.5 of the weights, and a row in debt puts the next
//   tile at kLowSet and starts anew.  A tile's losses are known two tiles later: they are summed behind its products, and
//   the accounts meet at the next vote.  A tile loses 2^-8 (2^-7 with e5m2) at most, if all 128 weights lie where the steps
//   are coarsest, beside a first tile of 2^kSet; what is lost in all is below 2^-7 of the sum, and 3.6e-3 of it at most in
//   8192 tokens with bright ones every 1 to 8 tiles and tails of 2^-8 .. 2^-20.  (With references held by the tiles'
//   largest weights alone, 2^-5 or more in one tile of three, the same tails lost up to 8%.)  Never lower than 2^-30 of the
//   highest reference before it: O and the sums then stay far inside fp32.
//
// The sums are those of w 2^-e, exact powers, while e is at most kPlainPower; rows of larger e beside rows of zeros would
// spread them over more than fp32 has, and then they are taken of p itself, under references of their own (`apart`).
//
// Products, per tile of 128 cached rows (NR = query rows of a block, 16, 32 or 64):
//   S [128 tokens x 2 NR]  = Y X^T            M = 128, N = 2 NR (x' and x'' of each row), K = 512 + rope
//   O^T [512 x 2 NR]      += C^T [W' W'']^T          four blocks of M = 128 channels, N = 2 NR, K = 128 tokens (64 rows:
//                                                     [512 x NR], N = NR, twice, each time reading the tile)
// The tokens lie on the lanes of tensor memory, so a softmax thread has one token of its rows: 2^{e_j} is one number a
// thread, weights of consecutive rows pack into words, and the tile's operands keep the full M = 128 (with the rows on the
// lanes a product of 64 rows takes as long, and the sum of the two terms crosses warps).  What that layout makes dear, a
// maximum over tokens, is not needed in every tile: references move only when a vote finds a weight too large or a row in
// debt; the sums stay in registers, a part a thread, until the piece ends.
//
// Work: as in the bf16 decode, one line of tiles in equal runs (kda_latent_line.cuh).  Block: a producer warp (TMA boxes
// of page rows), an issuing warp, a query loader, and two or four teams of four warps that quantise the queries and turn S
// into W.
//
// Measured (GB300, 6761 GB/s measured copy rate; ragged lengths of 1/4 to all of the stated context), one token: 64
// sequences of up to 8192, 32 heads, 47.2 us (0.58 of that rate; bf16 cache 69.9 us); 64 heads 64.0 us, 686 TFLOP/s (bf16
// 77.2 us); 256 of up to 8192, no rope, 135 us (0.74; bf16 210 us); one of 131072 26.8 us (0.42; bf16 36.7 us).  What is
// missing, at 32 heads: a fifth in the tiles (a tile's 3500 cycles are a chain: its load behind freed slots, 900 cycles of
// products for S, 1700 from S to W, 1000 of products for O; the slots hold two tiles and a half), and what is fixed: 1.6 us
// until a block knows its run, 3 us until its queries are quantised, 2 us from its last row to its stored result, 4 us of
// join.  At 64 heads the slots hold two tiles, the chain takes 4500 cycles, and the accounts are part of it (without them 58.6
// us).
#include <atomic>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "kda_internal.h"
#include "kda_latent_common.cuh"
#include "kda_latent_line.cuh"
#include "kda_latent_q8.cuh"
#include "sm103_primitives.cuh"

namespace kda {
namespace {

using namespace latent;
using namespace sm103;

constexpr int kRows = 128;                    // cached rows a tile
// Softmax warps work in teams of four (a warp for each quarter of a tile's tokens), the rows shared by the teams: sixteen a
// team (64 x 8192 cached tokens, 32 heads: 47.9 us, with four teams of eight 50.3; 256 x 8192, no rope, 138 and 147).
constexpr int teams_of(int nr) { return nr >= 64 ? 4 : 2; }
constexpr int soft_of(int nr) { return 128 * teams_of(nr); }
constexpr int threads_of(int nr) { return 128 + soft_of(nr); }       // before them: producer, issuer, queries, (TMEM)
constexpr int kBar = 1;                       // named barriers: all softmax warps; behind it one for each team
// The line (kda_latent_line.cuh): a piece's start and end take a block as long as three tiles (64 x 8192 cached tokens, 32
// heads: 47.8 us, 49.4 with one place; 32 x 4096, 4 tokens x 16 heads: 31.0, 32.9; with four places 47.8 and 30.9), and
// sequences of at most three tiles are not cut (before the accounts, 57 of up to 1084, 8 tokens x 12 heads: 35.5 us, 38.4
// with four; 182 of up to 285, 64 heads: 28.9, 30.3 with one).
constexpr int kPlaces = 3, kShort = 3;
constexpr float kDeep = 30.f;                 // log2 of how far a reference may lie below the highest before it
// The sums of p are those of the weights times 2^-e, in units of 2^m too, while all rows' e are at most this: a row's sum is
// then 2^-15 or more, and what a weight below 2^-126 would have added to it, 2^-62 at most, is nothing.
constexpr int kPlainPower = 15;

// Shared memory of a block with NR query rows: queries [slice][2 NR][128 bytes], their rope slice [2 NR][64], weights
// [buffers][128 tokens][2 NR] or, with 64 rows, [2 terms][128 tokens][NR], a tile's rope slice, then the latent slices (128 channels) of the tiles in flight.
// With 64 rows there is room for two whole tiles beside one buffer of weights.
template <int NR, bool ROPE>
struct Cfg {
    static constexpr uint32_t kQSlice = 2 * NR * 128, kQRope = ROPE ? 2 * NR * 64 : 0;
    // both terms of the weights side by side, with accumulators of their own (kO columns a block of channels): tensor
    // memory has room for that up to 32 rows
    static constexpr bool kWide = NR <= 32;
    static constexpr uint32_t kO = kWide ? 2 * NR : NR, kTiles = kWide ? 1 : 2;
    static constexpr uint32_t kPitch = NR == 16 ? 32 : 64, kPTile = kRows * kPitch;
    // log2 of a tile's largest weight: the largest that fits (64, whose rest times 2^7 is at most 256, and 448) and where a
    // larger one is put, where a piece's first tile is put, and where a tile is put whose row has lost too much
    static constexpr float kHigh = kWide ? 6.f : 8.75f, kHighSet = kWide ? 4.f : 6.f;
    static constexpr float kSet = kWide ? 1.f : 2.f, kLowSet = kWide ? 2.f : 3.f;
    // -2^-8.5, the share of its weights that a row may lose, in fp16 pairs; the rest of a wide weight is held times 2^7
    static constexpr uint32_t kShare = kWide ? 0xb5a8b5a8u : 0x99a899a8u;
    static constexpr uint32_t kQ = 0, kQR = 4 * kQSlice, kP = kQR + kQRope;
    static constexpr uint32_t kBuffers = NR == 64 ? 1 : 2;
    static constexpr uint32_t kRopeAt = kP + kBuffers * kTiles * kPTile, kSliceAt = kRopeAt + (ROPE ? 8192 : 0);
    static constexpr uint32_t kSmallBytes = 3 * 1024;
    static constexpr uint32_t kFit = (232448 - kSmallBytes - kSliceAt) / 16384, kSlices = kFit < 12 ? kFit : 12;
    static constexpr uint32_t kSmall = kSliceAt + kSlices * 16384;
    static constexpr uint32_t kBytes = kSmall + kSmallBytes;
    static constexpr uint32_t kCols = NR == 16 ? 256 : 512;   // TMEM: O^T 4 kO, S 2 x 2 NR
    static_assert(kBytes <= 232448 && kSlices >= 5, "shared memory");
    static_assert(kQR % 1024 == 0 && kP % 1024 == 0 && kSliceAt % 1024 == 0, "swizzled tiles");
};

struct Small : Line {
    uint64_t full[12], empty[12];             // latent slices
    uint64_t rope_full, rope_empty;
    uint64_t s_full[2], p_full[2], pv_done[2];
    uint64_t raw_full, q_full, q_empty;       // queries: bf16 landed, quantised, no longer needed
    uint64_t o_free, drain;
    uint32_t tmem;
    int piece[5], more;                       // the softmax warps' piece
    uint32_t vote[2][16];                     // a tile's votes, a warp each: any weight too large, any e above kPlainPower
    alignas(16) float ref[64], top[64];       // -m_r, and the highest m_r has been
    alignas(16) float move[64];               // by how much m_r moves; at a piece's end O's (second) factor
    alignas(16) float off[64];                // the sums' reference less m_r; at a piece's end O's first factor
    alignas(16) float unit[64];               // scale log2(e) 2^k of the query row
    alignas(16) int seen[64];                 // tokens that the row sees
    union {                                   // each team's part, whichever it is
        alignas(16) float red[4][4][16];      // a team's, a warp's: maxima, sums
        uint32_t loss[4][2][4][8];            // a team's, a tile's, a warp's: what its rows lost, in pairs
    };
};
static_assert(sizeof(Small) <= 3 * 1024, "small area");

using Walk = WalkOf<kRows, kPlaces>;

// OR and AND of a predicate over the softmax warps; also a barrier between them.
template <int SOFT>
__device__ __forceinline__ bool soft_or(bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "bar.red.or.pred p, %2, %3, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)pred), "n"(kBar), "n"(SOFT)
        : "memory");
    return r != 0;
}
template <int SOFT>
__device__ __forceinline__ bool soft_and(bool pred) { return !soft_or<SOFT>(!pred); }
template <int SOFT>
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync %0, %1;" ::"n"(kBar), "n"(SOFT) : "memory"); }
__device__ __forceinline__ void team_sync(int team) { asm volatile("bar.sync %0, 128;" ::"r"(kBar + 1 + team) : "memory"); }

// N consecutive 32-bit columns of the warp's lanes.
template <int N>
__device__ __forceinline__ void load_cols(uint32_t at, uint32_t (&r)[N]) {
    if constexpr (N == 8) tmem_ld8(at, r);
    if constexpr (N == 16) tmem_ld16(at, r);
}

// Reduces v[h] over the warp's lanes, for N values at once: each step halves the values a lane still holds, so N - 1 (and
// a few) exchanges and not 5 N.  The lane h * 32 / N is left with value h.
template <int N, typename Op>
__device__ __forceinline__ float reduce_rows(float (&v)[N], const Op& op) {
    const int lane = threadIdx.x & 31;
    int d = 16;
#pragma unroll
    for (int n = N / 2; n >= 1; n /= 2, d /= 2) {
        const bool upper = lane & d;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float mine = upper ? v[i + n] : v[i], other = upper ? v[i] : v[i + n];
            v[i] = op(mine, __shfl_xor_sync(0xffffffffu, other, d));
        }
    }
    for (; d >= 1; d /= 2) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], d));
    return v[0];
}
// The same sum of N pairs of fp16 numbers.
template <int N>
__device__ __forceinline__ uint32_t sum_pairs(uint32_t (&v)[N]) {
    const int lane = threadIdx.x & 31;
    int d = 16;
#pragma unroll
    for (int n = N / 2; n >= 1; n /= 2, d /= 2) {
        const bool upper = lane & d;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const uint32_t mine = upper ? v[i + n] : v[i], other = upper ? v[i] : v[i + n];
            v[i] = add_f16x2(mine, __shfl_xor_sync(0xffffffffu, other, d));
        }
    }
    for (; d >= 1; d /= 2) v[0] = add_f16x2(v[0], __shfl_xor_sync(0xffffffffu, v[0], d));
    return v[0];
}

__device__ __forceinline__ float2 pair(uint32_t x, uint32_t y) { return make_float2(__uint_as_float(x), __uint_as_float(y)); }
// The largest magnitude's bits among eight bf16 numbers, as fp32.
__device__ __forceinline__ uint32_t largest(const uint4& v) {
    constexpr uint32_t kAbs = 0x7fff7fffu;
    const uint32_t m = __vmaxu2(__vmaxu2(v.x & kAbs, v.y & kAbs), __vmaxu2(v.z & kAbs, v.w & kAbs));
    return max(m << 16, m & 0xffff0000u);
}
// Eight bf16 numbers times f as the sum of two e4m3 numbers each.
__device__ __forceinline__ void two_terms(const uint4& v, float f, uint2 (&y)[2]) {
    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
    uint32_t h[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = to_f16x2(__uint_as_float(x[i] << 16) * f, __uint_as_float(x[i] & 0xffff0000u) * f);
    y[0] = make_uint2(f16_to_e4m3x4(h[0], h[1]), f16_to_e4m3x4(h[2], h[3]));
    e4m3x4_to_f16(y[0].x, b[0], b[1]);
    e4m3x4_to_f16(y[0].y, b[2], b[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = sub_f16x2(h[i], b[i]);
    y[1] = make_uint2(f16_to_e4m3x4(b[0], b[1]), f16_to_e4m3x4(b[2], b[3]));
}

struct Maps {
    CUtensorMap q, c, r;                      // queries' latent slices, cached latent slices, cached rope slices
};

template <int NR, bool ROPE>
__global__ void __launch_bounds__(threads_of(NR), 1)
latent_decode_q8_kernel(const __grid_constant__ Maps maps, const LatentDecodeArgs a, const int groups, const int map_rows) {
    using G = Cfg<NR, ROPE>;
    constexpr int kTeams = teams_of(NR), kSoft = soft_of(NR), kThreads = threads_of(NR), kWarps = kSoft / 32;
    constexpr int NH = NR / kTeams;           // rows of a team
    extern __shared__ __align__(1024) uint8_t sm[];   // swizzled tiles start at multiples of 1024 bytes
    if (misaligned(sm, a)) return;
    Small* sw = reinterpret_cast<Small*>(sm + G::kSmall);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int runs = gridDim.x / groups, run = blockIdx.x / groups, group = blockIdx.x % groups;
    const int R = a.tokens_per_seq * a.H;
    const int rows = R - group * NR < NR ? R - group * NR : NR;      // live query rows
    const int shift = 31 - __clz(a.c.page_size);

    // as in the bf16 decode: this kernel sets itself up while the one before it ends, and the join while this one does
    allow_next();
    if (tid == 0) {
        for (uint32_t i = 0; i < G::kSlices; ++i) { mbar_init(&sw->full[i], 1); mbar_init(&sw->empty[i], 1); }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sw->s_full[i], 1);
            mbar_init(&sw->p_full[i], kWarps);
            mbar_init(&sw->pv_done[i], 1);
        }
        mbar_init(&sw->rope_full, 1);
        mbar_init(&sw->rope_empty, 1);
        mbar_init(&sw->raw_full, 1);
        mbar_init(&sw->q_full, kWarps);
        mbar_init(&sw->q_empty, 1);
        mbar_init(&sw->o_free, kWarps);
        mbar_init(&sw->drain, 1);
        fence_mbar_init();
        tma_prefetch_desc(&maps.q);
        tma_prefetch_desc(&maps.c);
        if (ROPE) tma_prefetch_desc(&maps.r);
    }
    if (warp == 3) {
        tmem_alloc(&sw->tmem, G::kCols);
        tmem_relinquish();
    }
    wait_before();
    find_run<kRows, kPlaces, kShort, kThreads>(a, runs, run, sw, reinterpret_cast<int64_t*>(sw->ref));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = sw->tmem;
    const uint32_t ts = tb + 4 * G::kO;       // S buffers
    bool ok = true;
    uint32_t loads = 0, rope_loads = 0;       // producer: latent and rope slices issued

    if (warp == 0) {                          // ------------------------------------------------ producer
        const int box = a.c.page_size < kRows ? a.c.page_size : kRows;
        constexpr int kWidth = kLatent + (ROPE ? kRope : 0);
        Walk walk(sw);
        Piece p;
        Ring<G::kSlices> ring;
        bool used = false;                    // the ring has gone round once
        while (ok && walk.next(a, p)) {
            const int64_t table = (int64_t)p.n * a.c.max_pages;
            // the first cache row of this lane's box in tile x; -1: none, map_rows: outside the cache, read as zeros
            auto row_of = [&](int x) -> int {
                if (lane * box >= kRows || lane * box >= p.len - x * kRows) return -1;
                const int pos = x * kRows + lane * box;
                if (!KDA_INDEX_OK(table + (pos >> shift), (int64_t)a.num_seqs * a.c.max_pages, a.status)) return map_rows;
                const int page = a.c.block_table[table + (pos >> shift)];
                return page < 0 || page >= a.c.num_pages ? map_rows : (page << shift) + (pos & (a.c.page_size - 1));
            };
            int row = row_of(p.off);
            for (int j = 0; ok && j < p.tiles; ++j) {
                const int next_row = j + 1 < p.tiles ? row_of(p.off + j + 1) : -1;
                const int live = p.len - (p.off + j) * kRows;
                const int valid = live < 0 ? 0 : (live < kRows ? live : kRows);
                const uint32_t boxes = (valid + box - 1) / box;
                for (int k = 0; k < 4; ++k) {
                    if (used && !(ok = wait_warp(&sw->empty[ring.slot], ring.phase ^ 1u))) break;
                    if (lane == 0) mbar_arrive_expect_tx(&sw->full[ring.slot], boxes * box * 128);
                    __syncwarp();
                    if (row >= 0)
                        tma_load_2d(sm + G::kSliceAt + ring.slot * 16384 + lane * box * 128, &maps.c, k * 128, row,
                                    &sw->full[ring.slot]);
                    ring.next();
                    ++loads;
                    if (ring.slot == 0) used = true;
                }
                if (!ok) break;
                if constexpr (ROPE) {
                    if (rope_loads > 0 && !(ok = wait_warp(&sw->rope_empty, (rope_loads - 1) & 1))) break;
                    if (lane == 0) mbar_arrive_expect_tx(&sw->rope_full, boxes * box * 64);
                    __syncwarp();
                    if (row >= 0) tma_load_2d(sm + G::kRopeAt + lane * box * 64, &maps.r, kLatent, row, &sw->rope_full);
                    ++rope_loads;
                }
                // The next tile into L2 behind this one's loads, where a request fetches 64 rows or more: its own loads
                // wait for ring slots and then find it near (64 x 8192 cached tokens, 32 heads: 47.8 us, 49.8 without;
                // pages of 16 gain nothing).
                const int next_live = live - kRows - lane * box;
                if (box >= 64 && next_row >= 0 && next_row < map_rows && next_live > 0)
                    bulk_prefetch_l2(static_cast<const uint8_t*>(a.c.cache) + (int64_t)next_row * kWidth,
                                     (uint32_t)(next_live < box ? next_live : box) * kWidth);
                row = next_row;
            }
        }
        if (!ok && lane == 0) {               // copies in flight land before the block ends
            for (uint32_t i = 0; i < G::kSlices; ++i)
                if (loads > i) mbar_wait_bounded(&sw->full[i], ((loads - 1 - i) / G::kSlices) & 1, kWaitNs);
            if (ROPE && rope_loads > 0) mbar_wait_bounded(&sw->rope_full, (rope_loads - 1) & 1, kWaitNs);
        }
    } else if (warp == 1) {                   // ------------------------------------------------ issuer
        constexpr uint32_t id_s = idesc_f8_f32(128, 2 * NR, false, false, false);
        constexpr uint32_t id_o[2] = {idesc_f8_f32(128, G::kO, false, true, true), idesc_f8_f32(128, NR, true, true, true)};
        constexpr uint32_t p_swizzle = G::kPitch == 64 ? kSwizzle64B : kSwizzle32B;
        // base descriptors: queries and cached rows as keys, the rope slices of both, weights, cached rows as values
        const uint64_t dq = smem_desc(smem_u32(sm + G::kQ), 16, 1024, kSwizzle128B);
        const uint64_t dqr = smem_desc(smem_u32(sm + G::kQR), 16, 512, kSwizzle64B);
        const uint64_t dk = smem_desc(smem_u32(sm + G::kSliceAt), 16, 1024, kSwizzle128B);
        const uint64_t dr = smem_desc(smem_u32(sm + G::kRopeAt), 16, 512, kSwizzle64B);
        const uint64_t dp = smem_desc(smem_u32(sm + G::kP), 16, 8 * G::kPitch, p_swizzle);
        const uint64_t dv = smem_desc(smem_u32(sm + G::kSliceAt), 16384, 1024, kSwizzle128B);
        const uint32_t el = elect_one();
        Walk walk(sw);
        Piece p;
        Ring<G::kSlices> in, out;             // next slice for S, next slice for O
        Ring<2> sb;                           // S buffers
        uint32_t scores = 0, products = 0;    // tiles that S, O have
        uint32_t seg = 0;
        while (ok && walk.next(a, p)) {
            if (!(ok = wait_warp(&sw->q_full, seg & 1))) break;
            tc_fence_after();
            // Slices of the next tile are multiplied as they land, between the value products of the tile before it: its
            // scores are ready soon after its last slice.
            int qk = 0, part = 0, pv = 0;     // tile and slice that S is at, tile that O is at
            bool freed = seg == 0;            // O of the piece before has been read
            uint64_t idle = 0;                // since when nothing could be issued
            constexpr int kParts = ROPE ? 5 : 4;
            while (pv < p.tiles) {
                bool landed = false, ready = false;
                if (qk < p.tiles && qk <= pv + 1)
                    landed = __all_sync(0xffffffffu, part < 4 ? mbar_test(&sw->full[in.slot], in.phase)
                                                              : mbar_test(&sw->rope_full, scores & 1));
                if (landed) {
                    tc_fence_after();
                    const uint32_t d = ts + sb.slot * 2 * NR;
                    if (part < 4) {
                        const uint64_t y = desc_at(dk, in.slot * 16384), x = desc_at(dq, part * G::kQSlice);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma_f8_ss_elected(d, desc_at(y, i * 32), desc_at(x, i * 32), id_s, part > 0 || i > 0, el);
                        in.next();
                    } else {
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            mma_f8_ss_elected(d, desc_at(dr, i * 32), desc_at(dqr, i * 32), id_s, 1, el);
                        mma_commit_elected(&sw->rope_empty, el);
                    }
                    if (++part == kParts) {
                        mma_commit_elected(&sw->s_full[sb.slot], el);
                        if (qk + 1 == p.tiles) mma_commit_elected(&sw->q_empty, el);
                        sb.next();
                        ++scores;
                        ++qk;
                        part = 0;
                    }
                } else if (pv < qk && !freed) {
                    ready = freed = __all_sync(0xffffffffu, mbar_test(&sw->o_free, (seg - 1) & 1));
                } else if (pv < qk) {
                    ready = __all_sync(0xffffffffu, mbar_test(&sw->p_full[products % G::kBuffers], products / G::kBuffers & 1));
                    if (ready) {
                        tc_fence_after();
                        const uint64_t x = desc_at(dp, products % G::kBuffers * G::kTiles * G::kPTile);
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            const uint64_t y = desc_at(dv, out.slot * 16384);
#pragma unroll
                            for (int term = 0; term < (int)G::kTiles; ++term)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    mma_f8_ss_elected(tb + b * G::kO, desc_at(y, i * 4096),
                                                      desc_at(x, term * G::kPTile + i * 32 * G::kPitch), id_o[term],
                                                      pv > 0 || term > 0 || i > 0, el);
                            mma_commit_elected(&sw->empty[out.slot], el);
                            out.next();
                        }
                        mma_commit_elected(&sw->pv_done[products % G::kBuffers], el);
                        ++products;
                        ++pv;
                    }
                }
                if (landed || ready) {
                    idle = 0;
                } else {
                    const uint64_t now = globaltimer_ns();
                    if (idle == 0) idle = now;
                    if (!(ok = __all_sync(0xffffffffu, now - idle < kWaitNs))) break;
                }
            }
            ++seg;
        }
        if (!ok) {                            // products in flight land before TMEM is freed
            mma_commit_elected(&sw->drain, el);
            wait_warp(&sw->drain, 0);
        }
    } else if (warp == 2) {                   // ------------------------------------------------ queries
        // A piece's queries, in bf16, to where they are quantised in place.  Behind the tiles that all blocks have asked
        // for they would come 3 to 5 us after their request: the next piece's are in L2 by then.
        Walk walk(sw);
        Piece p, next;
        uint32_t seg = 0;
        for (bool more = walk.next(a, p); more; p = next) {
            if (seg > 0 && !(ok = wait_warp(&sw->q_empty, (seg - 1) & 1))) break;
            if (lane == 0) mbar_arrive_expect_tx(&sw->raw_full, 8 * NR * 128);
            __syncwarp();
            if (lane < 8) tma_load_2d(sm + G::kQ + lane * NR * 128, &maps.q, lane * 64, p.n * R + group * NR, &sw->raw_full);
            ++seg;
            more = walk.next(a, next);
            const int64_t q = (int64_t)next.n * R + group * NR;
            if (more && lane == 0 && KDA_INDEX_OK(q + rows - 1, (int64_t)a.num_seqs * R, a.status)) {
                bulk_prefetch_l2(static_cast<const __nv_bfloat16*>(a.q_latent) + q * kLatent, rows * kLatent * 2);
                if (ROPE) bulk_prefetch_l2(static_cast<const __nv_bfloat16*>(a.q_rope) + q * kRope, rows * kRope * 2);
            }
        }
        if (seg > 0 && lane == 0) mbar_wait_bounded(&sw->raw_full, (seg - 1) & 1, kWaitNs);   // landed, whatever the others do
    } else if (warp >= 4) {                   // ------------------------------------------------ softmax
        const int w = (warp - 4) & 3, team = (warp - 4) >> 2, t = tid - (kThreads - kSoft);
        const int tok = 32 * w + lane;        // this thread's token of a tile; its rows are h0 .. h0 + NH - 1
        const int h0 = team * NH;
        const uint32_t lanes = tmem_addr(tb, 32 * w, h0);            // O^T: columns of this team
        const uint32_t s_lanes = tmem_addr(ts, 32 * w, h0);
        Walk walk(sw);
        Piece p{};
        Ring<G::kSlices> in;                  // the tile's first latent slice
        Ring<2> sb;                           // this tile's S buffer
        uint32_t tile = 0, pieces = 0;        // tiles before this one, of all pieces; pieces whose queries were taken
        // the value products of tile n are done
        auto have_products = [&](uint32_t n) { return wait_warp(&sw->pv_done[n % G::kBuffers], n / G::kBuffers & 1); };
        bool first_piece = true;
        Head head{-1, 0, 0, 0};
        int64_t at = sw->begin + sw->lead0;   // the piece's first tile in the line
        // the next piece, agreed on: one thread reads its sequence's length for all, since these warps meet at barriers and
        // must agree on the number of tiles, whatever a caller does to the lengths meanwhile
        auto announce = [&]() {
            if (t != 0) return;
            Piece x{};
            sw->more = walk.next(a, x);
            settle(x, runs);
            sw->piece[0] = x.n; sw->piece[1] = x.len; sw->piece[2] = x.off; sw->piece[3] = x.tiles; sw->piece[4] = x.all;
        };
        // A piece's queries in 8 bits, a warp a row.  The 128 bytes of channels 128 k .. 128 k + 63 of a row in bf16 lie
        // where the row's first terms of slice k go, those of the next 64 where its second terms go: in place.  The rope
        // part (a lane has a part of one of its warp's rows) goes through registers.  The loop is not unrolled: it runs once a piece, and
        // its instructions have to be fetched (unrolled, 3400 cycles of a block's start).
        auto take_queries = [&](const Piece& p) {
            constexpr int kMine = NR / kWarps;                       // rows of a warp
            static_assert(kMine <= 4, "a lane has one part of a row");
            const int rope_row = warp - 4 + kWarps * (lane >> 3);
            uint4 rope = make_uint4(0, 0, 0, 0);
            uint32_t rope_most = 0;
            int rope_power = 0;
            if constexpr (ROPE) {
                const int64_t q = (int64_t)p.n * R + group * NR + rope_row;
                if (rope_row < rows && KDA_INDEX_OK(q, (int64_t)a.num_seqs * R, a.status))
                    rope = __ldcg(static_cast<const uint4*>(a.q_rope) + q * (kRope / 8) + (lane & 7));
            }
            if (t < NR) sw->seen[t] = t < rows ? p.len - a.tokens_per_seq + 1 + (group * NR + t) / a.H : 0;
            ok = ok && wait_warp(&sw->raw_full, pieces & 1);
            if constexpr (ROPE) {
                rope_most = largest(rope);
                for (int d = 1; d < 8; d *= 2) rope_most = max(rope_most, __shfl_xor_sync(0xffffffffu, rope_most, d));
            }
#pragma unroll 1
            for (int i = 0; i < kMine; ++i) {
                const int r = warp - 4 + kWarps * i;
                uint4 x[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    x[c] = *reinterpret_cast<const uint4*>(sm + G::kQ + (4 * c + (lane >> 3)) * NR * 128 + sw128_offset(r, (lane & 7) * 16));
                    if (r >= rows) x[c] = make_uint4(0, 0, 0, 0);
                }
                uint32_t most = max(largest(x[0]), largest(x[1]));
                if constexpr (ROPE) most = max(most, __shfl_sync(0xffffffffu, rope_most, i * 8));
                most = __reduce_max_sync(0xffffffffu, most);         // also: all lanes have read the row
                const int k = power_for(most);
                if ((lane >> 3) == i) rope_power = k;
                __syncwarp();
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int slice = 4 * c + (lane >> 3);           // of 64 channels
                    uint2 y[2];
                    two_terms(x[c], two_to(-k), y);
#pragma unroll
                    for (int term = 0; term < 2; ++term)
                        *reinterpret_cast<uint2*>(sm + G::kQ + (slice >> 1) * G::kQSlice +
                                                  sw128_offset(term * NR + r, (slice & 1) * 64 + (lane & 7) * 8)) = y[term];
                }
                if (lane == 0) {
                    // (8-bit numbers end at 448: an infinite channel makes its row's scores NaN here)
                    sw->unit[r] = most < 0x7f800000u ? a.scale * 1.44269504088896340736f * two_to(k) : NAN;
                    sw->ref[r] = 0.f;
                    sw->top[r] = -INFINITY;
                }
            }
            if (ROPE && rope_row < NR) {
                uint2 y[2];
                two_terms(rope, two_to(-rope_power), y);
#pragma unroll
                for (int term = 0; term < 2; ++term)
                    *reinterpret_cast<uint2*>(sm + G::kQR + sw64_offset(term * NR + rope_row, (lane & 7) * 8)) = y[term];
            }
            ++pieces;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && ok) mbar_arrive(&sw->q_full);
        };
        announce();
        soft_sync<kSoft>();
        bool more = sw->more;
        if (more) {
            p = Piece{sw->piece[0], sw->piece[1], sw->piece[2], sw->piece[3], sw->piece[4]};
            take_queries(p);
            soft_sync<kSoft>();
        }
        while (more) {                        // (a warp whose wait ran out leaves at a barrier, with the others)
            announce();                       // all have read this piece's
            // this thread's cached row in tile x: its page, and its scale byte (0, the lowest, where there is none: such a
            // row reads as zeros and sets no reference)
            const int64_t entry = (int64_t)p.n * a.c.max_pages;
            const int len = p.len, off = p.off, tiles = p.tiles;
            auto page_of = [&](int x) -> int {
                const uint32_t pos = (uint32_t)x * kRows + tok;      // below 2^31 + 2^9
                if (pos >= (uint32_t)len) return -1;
                return KDA_INDEX_OK(entry + (pos >> shift), (int64_t)a.num_seqs * a.c.max_pages, a.status)
                           ? a.c.block_table[entry + (pos >> shift)] : -1;
            };
            auto byte_of = [&](int x, int page) -> uint8_t {
                if ((uint32_t)page >= (uint32_t)a.c.num_pages) return 0;
                const int64_t i = (uint32_t)(page << shift) + (((uint32_t)x * kRows + tok) & (uint32_t)(a.c.page_size - 1));
                return KDA_INDEX_OK(i, (int64_t)a.c.num_pages * a.c.page_size, a.status) ? __ldcg(a.c.scales + i) : 0;
            };
            const int page = page_of(off);
            int next_page = page_of(off + 1);
            const int least = p.len - a.tokens_per_seq + 1 + group * NR / a.H;      // tokens that the first row sees

            uint8_t byte = byte_of(off, page);
            // What a lane knows of two of its team's rows (as every warp of the team does): what they lost so far less their
            // share, by how much their references moved in this tile; its warp's losses in the tile before; and which rows
            // lost too much, the even and the odd ones.
            constexpr int kPairs = NH / 2;
            const int pair_row = h0 + 2 * (lane % kPairs);
            float2 lost = make_float2(0.f, 0.f), moved = make_float2(1.f, 1.f);
            uint32_t lost_here = 0, sick[2] = {0, 0};
            // The sums under references of their own, in the smallest code rather than the fastest (unrolled, it cost ordinary
            // calls 3%: 256 x 8192 cached tokens, no rope, 143 us and not 138): from then on l stands still.  The team's
            // thread of a row's number has the sum of the tiles since, and by how much the reference has risen since.
            bool apart = false;
            float sum_apart = 0.f, risen = 0.f;
            auto add_apart = [&](uint32_t s_at, float two_e, int unseen) {
#pragma unroll 1
                for (int round = 0; round < 2; ++round) {            // maxima, sums
                    team_sync(team);                                 // what was here has been read
#pragma unroll 1
                    for (int i = 0; i < NH; ++i) {
                        const float s = __uint_as_float(tmem_ld1(s_at + i)) + __uint_as_float(tmem_ld1(s_at + NR + i));
                        float u = fmaf(s * two_e, sw->unit[h0 + i], sw->ref[h0 + i] - sw->off[h0 + i]);
                        if (unseen >= sw->seen[h0 + i]) u = -INFINITY;
                        if (round) u = exp2_fast(u);
#pragma unroll 1
                        for (int d = 16; d; d >>= 1) {
                            const float other = __shfl_xor_sync(0xffffffffu, u, d);
                            u = round ? u + other : fmaxf(u, other);
                        }
                        if (lane == 0) sw->red[team][w][i] = u;
                    }
                    team_sync(team);
                    const int i = t & 127;
                    if (i < NH) {
                        const float* r = &sw->red[team][0][i];
                        if (round) {
                            sum_apart += (r[0] + r[16]) + (r[32] + r[48]);
                        } else {
                            const float up = fmaxf(rintf(fmaxf(fmaxf(r[0], r[16]), fmaxf(r[32], r[48]))), 0.f);
                            sw->off[h0 + i] += up;
                            sum_apart *= exp2_fast(-up);
                            risen += up;
                        }
                    }
                }
                team_sync(team);
            };
            float l[NH];
#pragma unroll
            for (int i = 0; i < NH; ++i) l[i] = 0.f;
            for (int j = 0; j < tiles; ++j) {
                const int base = (off + j) * kRows;
                const int e = power_of(byte);
                byte = byte_of(off + j + 1, next_page);              // a tile ahead, and its page two
                next_page = page_of(off + j + 2);
                // a wait that runs out is not left alone: the warps meet at barriers, and stop together
                ok = ok && wait_warp(&sw->s_full[sb.slot], sb.phase);
                tc_fence_after();
                const float2 two_e = make_float2(two_to(e), two_to(e)), fe = make_float2((float)e, (float)e);
                constexpr int N = NH;                                // rows a step
                const int unseen = least - base < kRows ? base + tok : INT_MIN;      // where some rows do not see some tokens
                const uint32_t s_at = s_lanes + sb.slot * 2 * NR;
                float x[NH];                  // the weights
                uint32_t y[2][NH / 4];        // in 8 bits, both terms
                uint32_t held[kPairs], rest[kPairs], theirs = 0;     // the weights in fp16, what the first term left
                bool move = j == 0 || sick[0] != 0 || sick[1] != 0;  // references have to move: a piece's first tile sets them
                bool voted = false, stop = false;
                for (;;) {
#pragma unroll
                    for (int c = 0; c < NH; c += N) {                // log2 of the weights
                        uint32_t s1[N], s2[N];
                        load_cols<N>(s_at + c, s1);
                        load_cols<N>(s_at + NR + c, s2);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < N; i += 4) {
                            const float4 u = *reinterpret_cast<const float4*>(sw->unit + h0 + c + i);
                            const float4 m = *reinterpret_cast<const float4*>(sw->ref + h0 + c + i);
                            const float2 v = fma2(mul2(add2(pair(s1[i], s1[i + 1]), pair(s2[i], s2[i + 1])), two_e),
                                                  make_float2(u.x, u.y), add2(fe, make_float2(m.x, m.y)));
                            const float2 w = fma2(mul2(add2(pair(s1[i + 2], s1[i + 3]), pair(s2[i + 2], s2[i + 3])), two_e),
                                                  make_float2(u.z, u.w), add2(fe, make_float2(m.z, m.w)));
                            x[c + i] = v.x; x[c + i + 1] = v.y; x[c + i + 2] = w.x; x[c + i + 3] = w.y;
                        }
                    }
                    if (unseen >= 0) {
#pragma unroll
                        for (int i = 0; i < NH; ++i)
                            if (unseen >= sw->seen[h0 + i]) x[i] = -INFINITY;
                    }
                    if (move) {               // the team agrees
                        float v[NH];
#pragma unroll
                        for (int i = 0; i < NH; ++i) v[i] = x[i];
                        const float mx = reduce_rows<NH>(v, [](float p, float q) { return fmaxf(p, q); });
                        team_sync(team);                             // the losses that were here have been read
                        if (lane % (32 / NH) == 0) sw->red[team][w][lane / (32 / NH)] = mx;
                        team_sync(team);
                        if (const int i = t & 127; i < NH) {
                            const float z = fmaxf(fmaxf(sw->red[team][0][i], sw->red[team][1][i]),
                                                  fmaxf(sw->red[team][2][i], sw->red[team][3][i]));
                            const float m = -sw->ref[h0 + i], top = sw->top[h0 + i];
                            const bool low = (i & 1 ? sick[1] : sick[0]) >> (i >> 1) & 1 && z < G::kLowSet - 0.5f;
                            float n = m;
                            if (z > -INFINITY && (j == 0 || z > G::kHigh || low)) {
                                n = fmaxf(m + rintf(z - (j == 0 ? G::kSet : z > G::kHigh ? G::kHighSet : G::kLowSet)), top - kDeep);
                                sw->ref[h0 + i] = -n;
                                sw->top[h0 + i] = fmaxf(top, n);
                            }
                            sw->move[h0 + i] = n - m;
                            if (j == 0 || apart) sw->off[h0 + i] = j == 0 ? 0.f : sw->off[h0 + i] - (n - m);
                        }
                        team_sync(team);
                        if (j > 0) ok = ok && have_products(tile - 1);
                        tc_fence_after();
#pragma unroll
                        for (int c = 0; c < NH; c += 8) {
                            float f[8];
                            bool still = true;                       // none of these rows moves
#pragma unroll
                            for (int n = 0; n < 8; ++n) {
                                const float d = sw->move[h0 + c + n];
                                still = still && d == 0.f;
                                x[c + n] -= d;
                                f[n] = exp2_fast(fminf(-d, 100.f));  // 0 where it is below 2^-126
                                if (!apart) l[c + n] *= f[n];
                            }
                            if (j > 0 && ok && !still) {             // O^T, column r by f_r
#pragma unroll 1
                                for (uint32_t at = 0; at < G::kO; at += NR) {
                                    uint32_t o[4][8];
#pragma unroll
                                    for (int b = 0; b < 4; ++b) tmem_ld8(lanes + b * G::kO + at + c, o[b]);
                                    tmem_wait_ld();
#pragma unroll
                                    for (int b = 0; b < 4; ++b) {
#pragma unroll
                                        for (int n = 0; n < 8; ++n) o[b][n] = __float_as_uint(__uint_as_float(o[b][n]) * f[n]);
                                        tmem_st8(lanes + b * G::kO + at + c, o[b]);
                                    }
                                }
                            }
                        }
                        tmem_wait_st();
                        // a row that was told to move starts a new account
                        const uint32_t bit = 1u << lane % kPairs;
                        const float2 f = make_float2(exp2_fast(fminf(-sw->move[pair_row], 100.f)),
                                                     exp2_fast(fminf(-sw->move[pair_row + 1], 100.f)));
                        lost = make_float2((sick[0] & bit ? fminf(lost.x, 0.f) : lost.x) * f.x,
                                           (sick[1] & bit ? fminf(lost.y, 0.f) : lost.y) * f.y);
                        moved = make_float2(moved.x * f.x, moved.y * f.y);
                        sick[0] = sick[1] = 0;
                    }
                    float most = x[0];
#pragma unroll
                    for (int i = 1; i < NH; ++i) most = fmaxf(most, x[i]);
#pragma unroll
                    for (int i = 0; i < NH; i += 4) {                // (fp16 holds 11 bits of a weight, differences are exact)
#pragma unroll
                        for (int n = 0; n < 4; ++n) x[i + n] = exp2_fast(x[i + n]);
                        y[0][i / 4] = to_e4m3x4(x[i], x[i + 1], x[i + 2], x[i + 3]);
                        uint32_t lo, hi;
                        e4m3x4_to_f16(y[0][i / 4], lo, hi);
                        held[i / 2] = to_f16x2(x[i], x[i + 1]);
                        held[i / 2 + 1] = to_f16x2(x[i + 2], x[i + 3]);
                        lo = sub_f16x2(held[i / 2], lo);
                        hi = sub_f16x2(held[i / 2 + 1], hi);
                        rest[i / 2] = G::kWide ? mul_f16x2(lo, k128) : lo;
                        rest[i / 2 + 1] = G::kWide ? mul_f16x2(hi, k128) : hi;
                        y[1][i / 4] = G::kWide ? f16_to_e4m3x4(rest[i / 2], rest[i / 2 + 1]) : f16_to_e5m2x4(rest[i / 2], rest[i / 2 + 1]);
                    }
                    if (voted) break;
                    // (a large e in a later tile: once more too, without a move)
                    uint32_t vote = __any_sync(0xffffffffu, most > G::kHigh || e > kPlainPower);
                    if (vote) vote |= __any_sync(0xffffffffu, e > kPlainPower) ? 2 : 0;
                    if (lane == 0) sw->vote[j & 1][warp - 4] = vote;
                    if (lane % (32 / kPairs) == 0) sw->loss[team][j & 1][w][lane / (32 / kPairs)] = lost_here;
                    // once a tile, by all teams, whatever their references do: the barrier is all softmax warps'
                    if (soft_or<kSoft>(!ok)) { stop = true; break; }
                    voted = true;
                    uint32_t votes = 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) votes |= sw->vote[j & 1][team * 4 + k];
                    apart = apart || (votes & 2) != 0;
                    theirs = sw->loss[team][j & 1][lane / kPairs & 3][lane % kPairs];
                    if ((votes & 1) == 0) break;
                    move = true;              // once more from the scores
                }
                if (stop) { ok = false; break; }
                if (__builtin_expect(apart, 0)) add_apart(s_at, two_to(e), unseen);
                if (len - base < kRows) {                  // the tile's rows behind the sequence's end become zeros
                    const int valid = len - base < 0 ? 0 : len - base;
                    Ring<G::kSlices> slice = in;
                    for (int k = 0; k < 4; ++k, slice.next())
                        for (int i = t; i < (kRows - valid) * 8; i += kSoft)
                            *reinterpret_cast<uint4*>(sm + G::kSliceAt + slice.slot * 16384 + (valid + (i >> 3)) * 128 + (i & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                }
                // the weights that were here have been read
                if (tile >= G::kBuffers) ok = ok && have_products(tile - G::kBuffers);
                if (ok) {
                    uint8_t* pt = sm + G::kP + tile % G::kBuffers * G::kTiles * G::kPTile;
#pragma unroll
                    for (int term = 0; term < 2; ++term) {
                        const uint32_t* v = y[term];
                        const int col = h0 + (G::kWide ? term * NR : 0);
                        const uint32_t off = (G::kWide ? 0 : term * G::kPTile) +
                                             (G::kPitch == 64 ? sw64_offset(tok, col) : sw32_offset(tok, col));
                        if constexpr (NH == 16)
                            *reinterpret_cast<uint4*>(pt + off) = make_uint4(v[0], v[1], v[2], v[3]);
                        else
                            *reinterpret_cast<uint2*>(pt + off) = make_uint2(v[0], v[1]);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && ok) mbar_arrive(&sw->p_full[tile % G::kBuffers]);
                const float2 back = apart ? make_float2(0.f, 0.f) : make_float2(two_to(-e), two_to(-e));
#pragma unroll
                for (int i = 0; i < NH; i += 2) {
                    const float2 v = fma2(make_float2(x[i], x[i + 1]), back, make_float2(l[i], l[i + 1]));
                    l[i] = v.x;
                    l[i + 1] = v.y;
                }
                // what the tile before lost joins the accounts; this one's loss is summed over the warp for the next vote
                float2 loss = f16x2_to_floats(theirs);
#pragma unroll
                for (int d = kPairs; d <= 2 * kPairs; d *= 2) {
                    loss.x += __shfl_xor_sync(0xffffffffu, loss.x, d);
                    loss.y += __shfl_xor_sync(0xffffffffu, loss.y, d);
                }
                lost = make_float2(fmaf(loss.x, moved.x, lost.x), fmaf(loss.y, moved.y, lost.y));
                moved = make_float2(1.f, 1.f);
                constexpr uint32_t kRowPairs = (1u << kPairs) - 1;
                sick[0] = __ballot_sync(0xffffffffu, lost.x > 0.f) & kRowPairs;
                sick[1] = __ballot_sync(0xffffffffu, lost.y > 0.f) & kRowPairs;
#pragma unroll
                for (int i = 0; i < NH; i += 4) {
                    uint32_t lo, hi;
                    if constexpr (G::kWide)
                        e4m3x4_to_f16(y[1][i / 4], lo, hi);
                    else
                        e5m2x4_to_f16(y[1][i / 4], lo, hi);
                    rest[i / 2] = fma_f16x2(held[i / 2], G::kShare, sub_f16x2(rest[i / 2], lo) & 0x7fff7fffu);
                    rest[i / 2 + 1] = fma_f16x2(held[i / 2 + 1], G::kShare, sub_f16x2(rest[i / 2 + 1], hi) & 0x7fff7fffu);
                }
                lost_here = sum_pairs<kPairs>(rest);
                ++tile;
                sb.next();
                in.next(); in.next(); in.next(); in.next();
            }
            if (!soft_and<kSoft>(ok)) { ok = false; break; }
            // ---- the piece is done: its rows' sums, then O^T out of tensor memory
            const bool whole = is_whole(p);
            const int slot = blockIdx.x * 2 + (first_piece ? 0 : 1);
            if (p.off == 0 && !whole) {
                head.n = p.n;
                head.first_slot = first_piece ? 0 : 1;
                // never past the last run, whatever happens to the lengths while the call runs: the join reads by it
                const int last = run_of(sw->total, sw->runs, at + p.all - 1);
                head.parts = (last >= run && last < runs ? last : runs - 1) - run + 1;
            }
            uint8_t* ws = static_cast<uint8_t*>(a.workspace);
            float2* ml = reinterpret_cast<float2*>(ws + Work<NR>::ml_at(gridDim.x));
            float* po = reinterpret_cast<float*>(ws + Work<NR>::o_at(gridDim.x));
            const float sum = reduce_rows<NH>(l, [](float p, float q) { return p + q; });
            if (lane % (32 / NH) == 0) sw->red[team][w][lane / (32 / NH)] = sum;
            if (const int i = t & 127; i < NH) {                     // (a row's unit is not needed any more)
                sw->move[h0 + i] = sum_apart;
                sw->unit[h0 + i] = exp2_fast(-risen);
            }
            soft_sync<kSoft>();
            if (t < NR) {
                const float* part = &sw->red[t / NH][0][t % NH];
                const float total = fmaf((part[0] + part[16]) + (part[32] + part[48]), sw->unit[t], sw->move[t]);
                // total 2^(m + off) = f 2^k: no large m against a large logarithm, here and in the join.  f is in [1, 2), and
                // in [2^-10, 2^-9) where the join adds up to 152 pieces' f times their mean: values end above 2^127
                const float off = sw->off[t];
                const int power = (int)(__float_as_uint(total) >> 23) - 127 + (whole ? 0 : 10);
                const float f = total == 0.f ? 0.f : total * two_to(-power), k = total == 0.f ? -INFINITY : (float)power + (off - sw->ref[t]);
                if (whole) {
                    const int64_t row = (int64_t)p.n * R + group * NR + t;
                    if (a.lse && t < rows && KDA_INDEX_OK(row, (int64_t)a.num_seqs * R, a.status))
                        a.lse[row] = total == 0.f ? -INFINITY : k * 0.69314718055994530942f + logf(f);
                } else if (KDA_INDEX_OK((int64_t)slot * NR + t, (int64_t)gridDim.x * 2 * NR, a.status)) {
                    ml[(int64_t)slot * NR + t] = make_float2(k, f);
                }
                // O is in units of 2^m: times 2^-off in two steps, since O / total may be far from O 2^-off / total
                const int half = -(int)off >> 1;
                sw->move[t] = total == 0.f ? 0.f : (whole ? 1.f / total : two_to(-power)) * two_to(-(int)off - half);
                sw->off[t] = two_to(half);
            }
            soft_sync<kSoft>();
            // the next piece's queries while this one's last products run (those with the queries are done: their S has
            // been read); its first scores are then computed while this piece's result is written
            more = sw->more;
            const Piece next{sw->piece[0], sw->piece[1], sw->piece[2], sw->piece[3], sw->piece[4]};
            if (more) take_queries(next);
            ok = soft_and<kSoft>(ok && have_products(tile - 1));
            if (!ok) break;
            tc_fence_after();
            // column r of block b: row r, channels 128 b ..; a lane stores its channel of 8 rows at a time, so a
            // warp's store is 64 bytes of a row in bf16, 128 in fp32
            const int64_t row = whole ? (int64_t)p.n * R + group * NR : (int64_t)slot * NR;
            const bool inside = whole ? KDA_INDEX_OK(row + rows - 1, (int64_t)a.num_seqs * R, a.status)
                                      : KDA_INDEX_OK(row + NR - 1, (int64_t)gridDim.x * 2 * NR, a.status);
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + (row + h0) * kLatent + tok;
            float* part = po + (row + h0) * kLatent + tok;
#pragma unroll
            for (int c = 0; c < NH; c += 8) {
                uint32_t o[4][8], rest[4][8];
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    tmem_ld8(lanes + b * G::kO + c, o[b]);
                    if (G::kWide) tmem_ld8(lanes + b * G::kO + NR + c, rest[b]);
                }
                tmem_wait_ld();
                if constexpr (G::kWide) {
#pragma unroll
                    for (int b = 0; b < 4; ++b)
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            o[b][i] = __float_as_uint(fmaf(__uint_as_float(rest[b][i]), 0x1p-7f, __uint_as_float(o[b][i])));
                }
                if (__builtin_expect(apart, 0)) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float g = sw->off[h0 + c + i];
#pragma unroll
                        for (int b = 0; b < 4; ++b) o[b][i] = __float_as_uint(__uint_as_float(o[b][i]) * g);
                    }
                }
                const int live = inside ? rows - h0 - c : 0;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < live) {
                        const float f = sw->move[h0 + c + i];
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            if (whole)
                                out[(c + i) * kLatent + b * 128] = __float2bfloat16_rn(__uint_as_float(o[b][i]) * f);
                            else
                                part[(c + i) * kLatent + b * 128] = __uint_as_float(o[b][i]) * f;
                        }
                    }
            }
            tc_fence_before();
            // everyone has read the sums before the next piece writes them
            soft_sync<kSoft>();
            if (lane == 0) mbar_arrive(&sw->o_free);
            at += p.tiles + kPlaces;
            p = next;
            first_piece = false;
        }
        if (t == 0) reinterpret_cast<Head*>(a.workspace)[blockIdx.x] = head;
    }
    if (!ok && lane == 0) atomicOr(a.status, kStatusTimeout);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 3) tmem_dealloc(tb, G::kCols);
}

// [rows, width] elements of 2 or 1 bytes, boxes of `channels` x box_rows, swizzled over the box's row.
bool map_rows_2d(CUtensorMap* m, const void* base, int bytes, int64_t rows, int width, int channels, int box_rows) {
    const auto fn = encode();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)width * bytes};
    cuuint32_t box[2] = {(cuuint32_t)channels, (cuuint32_t)box_rows}, es[2] = {1, 1};
    return fn(m, bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims,
              strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              channels * bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NR, bool ROPE>
cudaError_t launch(const LatentDecodeArgs& a, cudaStream_t s) {
    using G = Cfg<NR, ROPE>;
    const int R = a.tokens_per_seq * a.H, groups = groups_of(R), grid = runs_of(groups) * groups;
    const int box = a.c.page_size < kRows ? a.c.page_size : kRows, width = kLatent + (ROPE ? kRope : 0);
    // a cache without pages: any readable row; every box then starts behind the map's last row
    const int64_t c_rows = a.c.num_pages > 0 ? (int64_t)a.c.num_pages * a.c.page_size : 1;
    const void* c_base = a.c.num_pages > 0 ? a.c.cache : a.workspace;
    Maps maps;
    if (!map_rows_2d(&maps.q, a.q_latent, 2, (int64_t)a.num_seqs * R, kLatent, 64, NR) ||
        !map_rows_2d(&maps.c, c_base, 1, c_rows, width, 128, box) || !map_rows_2d(&maps.r, c_base, 1, c_rows, width, kRope, box))
        return cudaErrorInvalidValue;
    static std::atomic<bool> ready[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(latent_decode_q8_kernel<NR, ROPE>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, (int)G::kBytes);
        if (e != cudaSuccess) return e;
        ready[dev].store(true, std::memory_order_release);
    }
    const cudaError_t e = launch_overlapped(latent_decode_q8_kernel<NR, ROPE>, grid, threads_of(NR), G::kBytes, s, maps, a, groups,
                                            (int)c_rows);
    return e != cudaSuccess ? e : launch_overlapped(latent_join_kernel<NR>, kJoinBlocks, kJoinThreads, 0, s, a, grid, groups);
}

template <int NR>
cudaError_t launch_rope(const LatentDecodeArgs& a, cudaStream_t s) {
    return a.c.rope_dim ? launch<NR, true>(a, s) : launch<NR, false>(a, s);
}

}  // namespace

size_t latent_decode_q8_workspace_bytes(int tokens_per_seq, int H) { return line_workspace_bytes(tokens_per_seq, H); }

cudaError_t launch_latent_decode_q8(const LatentDecodeArgs& a, cudaStream_t s) {
    switch (rows_a_block(a.tokens_per_seq * a.H)) {
        case 16: return launch_rope<16>(a, s);
        case 32: return launch_rope<32>(a, s);
        default: return launch_rope<64>(a, s);
    }
}

}  // namespace kda
