// kda_latent_decode.cu -- absorbed latent attention over the paged cache (kda_latent_decode).
//
// For one sequence, the R = T' H query rows x_r = [q_latent | q_rope] of its step and its cached rows
// y_j = [c_j | r_j]:
//
//     s_rj = scale x_r . y_j,   p_rj = e^{s_rj - m_r},   o_r = sum_j p_rj c_j / sum_j p_rj.
//
// All rows read the same y_j, so a cached row is read once for up to 64 query rows: it is key (576 channels)
// and value (its first 512) in one.  With 32 rows that is 60 flop a byte, far below the card's 280, and the
// cache's bytes bound the call; with 128 rows (242 flop a byte) memory and tensor cores meet.
//
// Products, per tile of 64 cached rows (NR = query rows of a block, 16, 32 or 64), on tcgen05:
//   S [64 x 64 tokens]    = X Y^T       M = 64 (rows beyond NR are not looked at), K = 512 + rope
//   O^T [512 x NR]       += C^T P^T     four products of M = 128 channels, N = NR, K = 64 tokens
// The second is transposed so that the 512 wide output lies on the 128 lanes of tensor memory in four blocks of
// NR columns (a row-major O would need M = 128 rows for R = 32 and all of tensor memory), and so that the tile is
// read in place, as it lies in the cache, by both products.
//
// Work: the tiles of all sequences form one line, cut into equal runs, one for each block of a grid of one
// block an SM (divided by the row groups, which take the same run at the same time and so share the tile in
// L2).  The lengths are on the device, so every block finds its own run.  A run that covers a sequence whole
// writes its output; other pieces leave (O, m, l) in the workspace, and a second kernel joins them in their
// order, whatever order the blocks ran in.
//
// Block: a producer warp (TMA boxes of page rows), an issuing warp, a query loader, and four warps that turn S
// into P.  The running maximum m is only raised when a score exceeds it by more than 2^8: P then stays below 2^8
// in bf16, whose precision does not depend on the exponent, sums are fp32, and the rescaling of O in tensor
// memory is rare.  P is rounded to bf16 for the tensor cores; its sum is taken before that rounding.
//
// Measured (GB300, 6688 GB/s measured copy rate), 32 heads, one token: 608 x 4096 cached tokens 417 us, 1.03 of that
// rate; 64 x 8192 105.3 us (0.86); 1 x 131072 36.5 us (0.62).  What is missing there is fixed: 3 us until a block's
// first load (lengths, then page entries), 3 us from its last row to its result, 3-5 us of join; and the SMs' unequal
// shares of the bandwidth (their ends are spread over 5%).  128 heads, 64 x 8192: 211.8 us, 689 TFLOP/s: two groups of
// 64 rows, each with room for two tiles only, so that a tile's load waits for the one before the last.
#include <atomic>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <math.h>
#include <stdint.h>

#include "kda_internal.h"
#include "kda_latent_common.cuh"
#include "kda_latent_runs.h"
#include "sm103_primitives.cuh"

namespace kda {
namespace {

using namespace latent;
using namespace sm103;

constexpr int kThreads = 256;                 // warps 0-3: producer, issuer, queries, (TMEM); warps 4-7: softmax
constexpr int kSoft = 128;
constexpr int kBar = 1;                       // named barrier of the softmax warps
constexpr int kSMs = 152;
constexpr float kRaise = 8.f;                 // log2 of how far a score may exceed the running maximum
constexpr uint64_t kWaitNs = 4000000000ull;   // bound of every wait

// Shared memory of a block with NR query rows: queries [slice][NR][64], P [2][NR][64], the rope slices of the
// tiles in flight, then their latent slices in pairs (128 channels, one M = 128 operand).
template <int NR, bool ROPE>
struct Cfg {
    static constexpr uint32_t kSlice = NR * 128, kSlices = ROPE ? 9 : 8;
    static constexpr uint32_t kQ = 0, kP = kSlice * kSlices;
    static constexpr uint32_t kRopeSlots = ROPE ? (NR == 64 ? 1 : 2) : 0;
    static constexpr uint32_t kRopeAt = kP + 2 * kSlice, kPairAt = kRopeAt + kRopeSlots * 8192;
    static constexpr uint32_t kPairs = (225 * 1024 - kPairAt) / 16384;
    static constexpr uint32_t kSmall = kPairAt + kPairs * 16384;
    static constexpr uint32_t kBytes = kSmall + 1024;
    static constexpr uint32_t kCols = NR == 64 ? 512 : 256;       // TMEM: O^T 4 NR, S 2 x 64
    static_assert(kBytes <= 232448, "shared memory");
    static_assert(64 * 128 <= kSmall - (kSlices - 1) * kSlice, "the M = 64 operand stays inside the block's memory");
};

struct Small {
    uint64_t full[12], empty[12];             // latent pairs
    uint64_t rope_full[2], rope_empty[2];
    uint64_t q_full, q_empty;
    uint64_t s_full[2], p_full[2], pv_done[2];
    uint64_t o_free, drain;
    uint32_t tmem;
    int seq0, off0, lead0, len0, runs;
    int piece[5], more;                       // the softmax warps' piece
    int64_t total, begin, end;
    alignas(16) float fac[64];                // rescaling factors
    alignas(16) float inv[64];                // 1 / l at a piece's end
};
static_assert(sizeof(Small) <= 1024, "small area");

// Position in a ring of SLOTS slots; `phase` flips each time round.
template <uint32_t SLOTS>
struct Ring {
    uint32_t slot = 0, phase = 0;
    __device__ __forceinline__ void next() {
        if (++slot == SLOTS) { slot = 0; phase ^= 1u; }
    }
};

// Sequences of at most so many tiles are not cut, if runs have two places or more: the cut goes to the nearer end.  The
// partial results of two pieces cost more than the unevenness: 182 sequences of up to 285 tokens, 64 heads, 26.4 us
// against 34.7 when cut (28.9 with a limit of 4 tiles); 100 of up to 400, 32 heads, 16.8 against 19.7; with a limit of
// 8 tiles unevenness wins (57 of up to 1084, 8 tokens x 12 heads: 45 us, 39 with 6, 37 when cut).
constexpr int kShort = 6;

// Walks the sequences of this block's run; every role walks by itself.
struct Walk : RunWalk {
    __device__ Walk(const Small* sw) : RunWalk{sw->seq0, sw->off0, sw->lead0, sw->len0, sw->end - sw->begin} {}
    __device__ __forceinline__ bool next(const LatentDecodeArgs& a, Piece& p) {
        return RunWalk::next(a.num_seqs, [&](int seq) { return clamped_len(a.c, a.seq_lens, seq); }, p);
    }
};

// A converged warp waits, and agrees on whether all its lanes saw the phase end in time.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_parked(bar, parity, kWaitNs));
}
// OR and AND of a predicate over the softmax warps; also a barrier between them.
__device__ __forceinline__ bool soft_or(bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "bar.red.or.pred p, %2, %3, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)pred), "n"(kBar), "n"(kSoft)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ bool soft_and(bool pred) { return !soft_or(!pred); }
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync %0, %1;" ::"n"(kBar), "n"(kSoft) : "memory"); }

// Workspace: a header a block (the sequence whose first piece it holds), then per (block, 0 or 1) and row the
// maximum (in log2) and the sum, then O.
struct Head {
    int n, parts, first_slot, pad;            // n = -1: none
};
template <int NR>
struct Work {
    static __host__ __device__ size_t ml_at(int grid) { return ((size_t)grid * sizeof(Head) + 255) / 256 * 256; }
    static __host__ __device__ size_t o_at(int grid) {
        return ml_at(grid) + ((size_t)grid * 2 * NR * sizeof(float2) + 255) / 256 * 256;
    }
    static __host__ __device__ size_t bytes(int grid) { return o_at(grid) + (size_t)grid * 2 * NR * kLatent * sizeof(float); }
};

struct Maps {
    CUtensorMap q, qr, c;
};

// All threads: the run of this block and the sequence it starts in.  Rounds of a sequence a thread; with up to
// kThreads sequences the lengths are read once.
__device__ void find_run(const LatentDecodeArgs& a, int runs, int p, Small* sw, int64_t* scratch) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int len = 0;
    auto tiles_at = [&](int n) {
        if (n >= a.num_seqs) return 0;
        len = clamped_len(a.c, a.seq_lens, n);
        return kStart + tiles_of(len);
    };
    // the round's places before this thread's sequence, and in all
    auto scan = [&](int mine, int64_t& round) {
        int64_t x = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) scratch[warp] = x;
        __syncthreads();
        round = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) x += scratch[w];
            round += scratch[w];
        }
        __syncthreads();
        return x - mine;
    };
    int mine = tiles_at(tid);
    int64_t round, at = scan(mine, round);
    int mine_len = len;
    int64_t total = round;
    for (int n0 = kThreads; n0 < a.num_seqs; n0 += kThreads) {
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
            if (spare || mine > kStart + kShort) return x;
            return x - first <= first + mine - x ? first : first + mine;
        };
        if (mine > 0 && first <= begin && begin < first + mine) {
            const int64_t x = cut(begin);
            const int into = (int)(x - first);
            const bool next = into == mine;   // the run starts with the next sequence
            sw->begin = x;
            sw->seq0 = n0 + tid + (next ? 1 : 0);
            sw->off0 = next || into < kStart ? 0 : into - kStart;
            sw->lead0 = next ? kStart : (into < kStart ? kStart - into : 0);
            sw->len0 = next ? -1 : mine_len;
        }
        if (mine > 0 && end < total && first <= end && end < first + mine) sw->end = cut(end);
        before += round;
        n0 += kThreads;
        if (before > end || n0 >= a.num_seqs) break;                 // uniform
        mine = tiles_at(n0 + tid);
        mine_len = len;
        at = scan(mine, round);
    }
}

template <int NR, bool ROPE>
__global__ void __launch_bounds__(kThreads, 1)
latent_decode_kernel(const __grid_constant__ Maps maps, const LatentDecodeArgs a, const int groups, const int map_rows) {
    using G = Cfg<NR, ROPE>;
    extern __shared__ __align__(1024) uint8_t sm[];   // swizzled tiles start at multiples of 1024 bytes
    if (smem_u32(sm) & 1023u) {               // the declaration's alignment
        if (threadIdx.x == 0) atomicOr(a.status, kStatusTimeout);
        return;
    }
    Small* sw = reinterpret_cast<Small*>(sm + G::kSmall);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int runs = gridDim.x / groups, run = blockIdx.x / groups, group = blockIdx.x % groups;
    const int R = a.tokens_per_seq * a.H;
    const int rows = R - group * NR < NR ? R - group * NR : NR;      // live query rows

    // this kernel may start while the one before it in the stream ends, and the join while this one does: each
    // sets itself up and then waits for everything before it
    allow_next();
    if (tid == 0) {
        for (uint32_t i = 0; i < G::kPairs; ++i) { mbar_init(&sw->full[i], 1); mbar_init(&sw->empty[i], 1); }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sw->rope_full[i], 1);
            mbar_init(&sw->rope_empty[i], 1);
            mbar_init(&sw->s_full[i], 1);
            mbar_init(&sw->p_full[i], 4);
            mbar_init(&sw->pv_done[i], 1);
        }
        mbar_init(&sw->q_full, 1);
        mbar_init(&sw->q_empty, 1);
        mbar_init(&sw->o_free, 4);
        mbar_init(&sw->drain, 1);
        fence_mbar_init();
        tma_prefetch_desc(&maps.q);
        if (ROPE) tma_prefetch_desc(&maps.qr);
        tma_prefetch_desc(&maps.c);
    }
    if (warp == 3) {
        tmem_alloc(&sw->tmem, G::kCols);
        tmem_relinquish();
    }
    wait_before();
    find_run(a, runs, run, sw, reinterpret_cast<int64_t*>(sw->fac));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = sw->tmem;
    const uint32_t ts = tb + 4 * NR;          // S buffers
    bool ok = true;
    uint32_t loads = 0, rope_loads = 0;       // producer: latent pairs and rope slices issued

    if (warp == 0) {                          // ------------------------------------------------ producer
        const int box = a.c.page_size < kTile ? a.c.page_size : kTile;
        const int shift = 31 - __clz(a.c.page_size);
        constexpr int width = kLatent + (ROPE ? kRope : 0);
        const int half = lane & 1, piece = lane >> 1;               // a lane issues one box of a pair
        Walk walk(sw);
        Piece p;
        Ring<G::kPairs> ring;
        Ring<ROPE ? G::kRopeSlots : 1> rope;
        bool used = false, rope_used = false; // the ring has gone round once
        while (ok && walk.next(a, p)) {
            const int64_t table = (int64_t)p.n * a.c.max_pages;
            // the page of this lane's box in tile x (a box outside the cache reads zeros)
            auto row_of = [&](int x) -> int {
                if (piece * box >= kTile || piece * box >= p.len - x * kTile) return -1;
                const int pos = x * kTile + piece * box;
                if (!KDA_INDEX_OK(table + (pos >> shift), (int64_t)a.num_seqs * a.c.max_pages, a.status)) return map_rows;
                const int page = a.c.block_table[table + (pos >> shift)];
                return page < 0 || page >= a.c.num_pages ? map_rows : (page << shift) + (pos & (a.c.page_size - 1));
            };
            // Where a tile lies on one page, the next tile is prefetched into L2 behind this one's loads, in one
            // request: its own loads wait for ring slots and then find it near.  Further ahead is slower (64 x 8192
            // cached tokens, 32 heads: 104.6 us one tile ahead, 106.7 two, 112.5 three, 136 five, 106.9 without):
            // the rows wait in both halves of L2.  So are prefetches of several small pages a tile (pages of 16:
            // 118.7 us with, 112.3 without).
            auto prefetch = [&](int r, int x) {
                const int left = p.len - x * kTile;
                if (box == kTile && half == 0 && r >= 0 && r < map_rows)
                    bulk_prefetch_l2(static_cast<const uint8_t*>(a.c.cache) + (int64_t)r * width * 2,
                                     (uint32_t)(left < kTile ? left : kTile) * width * 2);
            };
            int row = row_of(p.off);
            for (int j = 0; ok && j < p.tiles; ++j) {
                const int next_row = j + 1 < p.tiles ? row_of(p.off + j + 1) : -1;
                const int live = p.len - (p.off + j) * kTile;
                const int valid = live < 0 ? 0 : (live < kTile ? live : kTile);
                const uint32_t boxes = (valid + box - 1) / box;
                for (int k = 0; k < 4; ++k) {
                    if (used && !(ok = wait_warp(&sw->empty[ring.slot], ring.phase ^ 1u))) break;
                    if (lane == 0) mbar_arrive_expect_tx(&sw->full[ring.slot], boxes * box * 256);
                    __syncwarp();
                    if (row >= 0)
                        tma_load_2d(sm + G::kPairAt + ring.slot * 16384 + half * 8192 + piece * box * 128, &maps.c,
                                    (2 * k + half) * 64, row, &sw->full[ring.slot]);
                    ring.next();
                    ++loads;
                    if (ring.slot == 0) used = true;
                }
                if (!ok) break;
                if constexpr (ROPE) {
                    if (rope_used && !(ok = wait_warp(&sw->rope_empty[rope.slot], rope.phase ^ 1u))) break;
                    if (lane == 0) mbar_arrive_expect_tx(&sw->rope_full[rope.slot], boxes * box * 128);
                    __syncwarp();
                    if (row >= 0 && half == 0)
                        tma_load_2d(sm + G::kRopeAt + rope.slot * 8192 + piece * box * 128, &maps.c, kLatent, row,
                                    &sw->rope_full[rope.slot]);
                    rope.next();
                    ++rope_loads;
                    if (rope.slot == 0) rope_used = true;
                }
                prefetch(next_row, p.off + j + 1);
                row = next_row;
            }
        }
        if (!ok && lane == 0) {               // copies in flight land before the block ends
            for (uint32_t i = 0; i < G::kPairs; ++i)
                if (loads > i) mbar_wait_bounded(&sw->full[i], ((loads - 1 - i) / G::kPairs) & 1, kWaitNs);
            if constexpr (ROPE)
                for (uint32_t i = 0; i < G::kRopeSlots; ++i)
                    if (rope_loads > i)
                        mbar_wait_bounded(&sw->rope_full[i], ((rope_loads - 1 - i) / G::kRopeSlots) & 1, kWaitNs);
        }
    } else if (warp == 1) {                   // ------------------------------------------------ issuer
        constexpr uint32_t id_s = idesc_bf16_f32(64, 64, false, false);
        constexpr uint32_t id_o = idesc_bf16_f32(128, NR, true, false);
        // base descriptors: queries and cached rows as keys, rope slices, P, cached rows as values
        const uint64_t dq = smem_desc(smem_u32(sm + G::kQ), 16, 1024, kSwizzle128B);
        const uint64_t dk = smem_desc(smem_u32(sm + G::kPairAt), 16, 1024, kSwizzle128B);
        const uint64_t dr = smem_desc(smem_u32(sm + G::kRopeAt), 16, 1024, kSwizzle128B);
        const uint64_t dp = smem_desc(smem_u32(sm + G::kP), 16, 1024, kSwizzle128B);
        const uint64_t dv = smem_desc(smem_u32(sm + G::kPairAt), 8192, 1024, kSwizzle128B);
        const uint32_t el = elect_one();
        Walk walk(sw);
        Piece p;
        Ring<G::kPairs> in, out;              // next pair for S, next pair for O
        Ring<ROPE ? G::kRopeSlots : 1> rope;
        Ring<2> sb, pb;                       // S / P buffers
        uint32_t seg = 0;
        while (ok && walk.next(a, p)) {
            if (!(ok = wait_warp(&sw->q_full, seg & 1))) break;
            int qk = 0, pv = 0;
            while (pv < p.tiles) {
                bool go = qk == pv;
                if (!go && qk < p.tiles && qk == pv + 1) {           // ahead only when the tile has landed
                    Ring<G::kPairs> last = in;
                    last.next(); last.next(); last.next();
                    bool landed = mbar_test(&sw->full[last.slot], last.phase);
                    if (ROPE) landed = landed && mbar_test(&sw->rope_full[rope.slot], rope.phase);
                    go = __all_sync(0xffffffffu, landed);
                }
                if (go) {
                    const uint32_t d = ts + sb.slot * 64;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (!(ok = wait_warp(&sw->full[in.slot], in.phase))) break;
                        tc_fence_after();
                        const uint64_t y = desc_at(dk, in.slot * 16384);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            mma_ss_elected(d, desc_at(dq, (2 * k + (i >> 2)) * G::kSlice + (i & 3) * 32),
                                           desc_at(y, (i >> 2) * 8192 + (i & 3) * 32), id_s, k > 0 || i > 0, el);
                        in.next();
                    }
                    if (!ok) break;
                    if constexpr (ROPE) {
                        if (!(ok = wait_warp(&sw->rope_full[rope.slot], rope.phase))) break;
                        tc_fence_after();
                        const uint64_t y = desc_at(dr, rope.slot * 8192);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma_ss_elected(d, desc_at(dq, 8 * G::kSlice + i * 32), desc_at(y, i * 32), id_s, 1, el);
                        mma_commit_elected(&sw->rope_empty[rope.slot], el);
                        rope.next();
                    }
                    mma_commit_elected(&sw->s_full[sb.slot], el);
                    if (qk + 1 == p.tiles) mma_commit_elected(&sw->q_empty, el);
                    sb.next();
                    ++qk;
                } else {
                    if (!(ok = wait_warp(&sw->p_full[pb.slot], pb.phase))) break;
                    if (pv == 0 && seg > 0 && !(ok = wait_warp(&sw->o_free, (seg - 1) & 1))) break;
                    tc_fence_after();
                    const uint64_t x = desc_at(dp, pb.slot * G::kSlice);
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const uint64_t y = desc_at(dv, out.slot * 16384);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma_ss_elected(tb + b * NR, desc_at(y, i * 2048), desc_at(x, i * 32), id_o, pv > 0 || i > 0, el);
                        mma_commit_elected(&sw->empty[out.slot], el);
                        out.next();
                    }
                    mma_commit_elected(&sw->pv_done[pb.slot], el);
                    pb.next();
                    ++pv;
                }
            }
            ++seg;
        }
        if (!ok) {                            // products in flight land before TMEM is freed
            mma_commit_elected(&sw->drain, el);
            wait_warp(&sw->drain, 0);
        }
    } else if (warp == 2) {                   // ------------------------------------------------ queries
        Walk walk(sw);
        Piece p;
        uint32_t seg = 0;
        while (walk.next(a, p)) {
            if (seg > 0 && !(ok = wait_warp(&sw->q_empty, (seg - 1) & 1))) break;
            if (lane == 0) mbar_arrive_expect_tx(&sw->q_full, G::kSlice * G::kSlices);
            __syncwarp();
            const int row = p.n * R + group * NR;
            if (lane < 8)
                tma_load_2d(sm + G::kQ + lane * G::kSlice, &maps.q, lane * 64, row, &sw->q_full);
            else if (ROPE && lane == 8)
                tma_load_2d(sm + G::kQ + 8 * G::kSlice, &maps.qr, 0, row, &sw->q_full);
            ++seg;
        }
        if (!ok && seg > 0 && lane == 0) mbar_wait_bounded(&sw->q_full, (seg - 1) & 1, kWaitNs);
    } else if (warp >= 4) {                   // ------------------------------------------------ softmax
        const int w = warp - 4, t = tid - kSoft;
        const bool active = 16 * w < NR;
        const int r0 = 16 * w + lane / 4;     // this thread's rows: r0 and r0 + 8
        const float c2 = a.scale * 1.44269504088896340736f;
        const uint32_t lanes = tmem_addr(tb, 32 * w, 0);
        const uint32_t s_lanes = tmem_addr(ts, 32 * w, 0);
        Walk walk(sw);
        Piece p{};
        Ring<G::kPairs> in;                   // the tile's first latent pair
        Ring<2> sb, prev;                     // this tile's buffers; the previous tile's
        bool first_piece = true, used0 = false, used1 = false;
        Head head{-1, 0, 0, 0};
        int64_t at = sw->begin + sw->lead0;   // the piece's first tile in the line
        while (ok) {
            // one thread reads the next sequence's length for all: these warps meet at barriers and must agree on the
            // number of tiles, whatever a caller does to the lengths meanwhile
            if (t == 0) {
                sw->more = walk.next(a, p);
                settle(p, runs);              // here, once: the same test behind the tiles takes 2% of 128 heads' time
                sw->piece[0] = p.n; sw->piece[1] = p.len; sw->piece[2] = p.off; sw->piece[3] = p.tiles; sw->piece[4] = p.all;
            }
            soft_sync();
            if (!sw->more) break;
            p = Piece{sw->piece[0], sw->piece[1], sw->piece[2], sw->piece[3], sw->piece[4]};
            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
            int seen[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = r0 + 8 * e;
                seen[e] = r < rows ? p.len - a.tokens_per_seq + 1 + (group * NR + r) / a.H : 0;
            }
            for (int j = 0; j < p.tiles; ++j) {
                const int base = (p.off + j) * kTile;
                // a wait that runs out is not left alone: the four warps meet at barriers, and stop together
                ok = ok && wait_warp(&sw->s_full[sb.slot], sb.phase);
                tc_fence_after();
                uint32_t s[32];
                float f[2] = {1.f, 1.f};
                bool raise = false;
                if (active) {
                    tmem_ld_16x64(s_lanes + sb.slot * 64, s);
                    tmem_wait_ld();
                    const int lim[2] = {seen[0] - base, seen[1] - base};             // columns that the rows see
                    if (__any_sync(0xffffffffu, lim[0] < kTile || lim[1] < kTile)) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (8 * (i >> 2) + 2 * (lane & 3) + (i & 1) >= lim[(i >> 1) & 1]) s[i] = 0xff800000u;   // -inf
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = __uint_as_float(s[2 * e]);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            x = fmaxf(x, __uint_as_float(s[4 * i + 2 * e]));
                            x = fmaxf(x, __uint_as_float(s[4 * i + 2 * e + 1]));
                        }
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                        if (x > m[e] && (x - m[e]) * c2 > kRaise) {                  // also the first finite maximum
                            f[e] = exp2_fast((m[e] - x) * c2);
                            m[e] = x;
                            raise = true;
                        }
                        l[e] *= f[e];
                    }
                }
                if (p.len - base < kTile) {   // the tile's rows behind the sequence's end become zeros
                    const int valid = p.len - base < 0 ? 0 : p.len - base;
                    Ring<G::kPairs> pair = in;
                    for (int k = 0; k < 4; ++k, pair.next())
                        for (int i = t; i < (kTile - valid) * 16; i += kSoft)
                            *reinterpret_cast<uint4*>(sm + G::kPairAt + pair.slot * 16384 + ((i >> 3) & 1) * 8192 +
                                                      (valid + (i >> 4)) * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
                }
                if (soft_or((raise && j > 0) || !ok)) {              // rescale O^T, column r by f_r
                    if (!soft_and(ok)) { ok = false; break; }
                    if (active && (lane & 3) == 0) {
                        sw->fac[r0] = f[0];
                        sw->fac[r0 + 8] = f[1];
                    }
                    soft_sync();
                    ok = wait_warp(&sw->pv_done[prev.slot], prev.phase);
                    tc_fence_after();
#pragma unroll 1
                    for (int k = 0; k < NR / 16; ++k) {
                        float g[16];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            *reinterpret_cast<float4*>(g + 4 * i) = *reinterpret_cast<const float4*>(sw->fac + 16 * k + 4 * i);
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            uint32_t o[16];
                            tmem_ld16(lanes + b * NR + k * 16, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * g[i]);
                            tmem_st16(lanes + b * NR + k * 16, o);
                        }
                    }
                    tmem_wait_st();
                }
                // this P buffer was read by the products of two tiles ago
                if (sb.slot ? used1 : used0) ok = ok && wait_warp(&sw->pv_done[sb.slot], sb.phase ^ 1u);
                if (active && ok) {
                    uint8_t* pt = sm + G::kP + sb.slot * G::kSlice;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float z = m[e] == -INFINITY ? 0.f : -m[e] * c2;
                        float sum = 0.f;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float x = exp2_fast(fmaf(__uint_as_float(s[4 * i + 2 * e]), c2, z));
                            const float y = exp2_fast(fmaf(__uint_as_float(s[4 * i + 2 * e + 1]), c2, z));
                            sum += x + y;
                            *reinterpret_cast<uint32_t*>(pt + sw128_offset(r0 + 8 * e, 16 * i + 4 * (lane & 3))) =
                                pack_bf16x2(x, y);
                        }
                        l[e] += sum;
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && ok) mbar_arrive(&sw->p_full[sb.slot]);
                if (sb.slot) used1 = true; else used0 = true;
                prev = sb;
                sb.next();
                in.next(); in.next(); in.next(); in.next();
            }
            if (!soft_and(ok)) { ok = false; break; }
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
            if (active) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
                    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
                    const int r = r0 + 8 * e;
                    if ((lane & 3) == 0) {
                        sw->inv[r] = l[e] == 0.f ? 0.f : 1.f / l[e];
                        if (whole) {
                            const int64_t row = (int64_t)p.n * R + group * NR + r;
                            if (a.lse && r < rows && KDA_INDEX_OK(row, (int64_t)a.num_seqs * R, a.status))
                                a.lse[row] = l[e] == 0.f ? -INFINITY : m[e] * a.scale + logf(l[e]);
                        } else if (KDA_INDEX_OK((int64_t)slot * NR + r, (int64_t)gridDim.x * 2 * NR, a.status)) {
                            ml[(int64_t)slot * NR + r] = make_float2(m[e] == -INFINITY ? m[e] : m[e] * c2, l[e]);
                        }
                    }
                }
            }
            ok = soft_and(wait_warp(&sw->pv_done[prev.slot], prev.phase));   // also: inv is written
            if (!ok) break;
            tc_fence_after();
            // column r of block b: row r, channels 128 b ..; a lane stores its channel of 16 rows at a time, so a
            // warp's store is 64 bytes of a row in bf16, 128 in fp32
            const int64_t row = whole ? (int64_t)p.n * R + group * NR : (int64_t)slot * NR;
            const bool inside = whole ? KDA_INDEX_OK(row + rows - 1, (int64_t)a.num_seqs * R, a.status)
                                      : KDA_INDEX_OK(row + NR - 1, (int64_t)gridDim.x * 2 * NR, a.status);
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + row * kLatent + 32 * w + lane;
            float* part = po + row * kLatent + 32 * w + lane;
#pragma unroll
            for (int k = 0; k < NR / 16; ++k) {
                uint32_t o[4][16];
#pragma unroll
                for (int b = 0; b < 4; ++b) tmem_ld16(lanes + b * NR + k * 16, o[b]);
                tmem_wait_ld();
                const int live = inside ? rows - 16 * k : 0;
                if (whole) {
                    float f[16];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<float4*>(f + 4 * i) = *reinterpret_cast<const float4*>(sw->inv + 16 * k + 4 * i);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (i < live) {
#pragma unroll
                            for (int b = 0; b < 4; ++b)
                                out[i * kLatent + b * 128] = __float2bfloat16_rn(__uint_as_float(o[b][i]) * f[i]);
                        }
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (i < live) {
#pragma unroll
                            for (int b = 0; b < 4; ++b) part[i * kLatent + b * 128] = __uint_as_float(o[b][i]);
                        }
                }
                out += 16 * kLatent;
                part += 16 * kLatent;
            }
            tc_fence_before();
            // everyone has read inv before the next piece writes it
            soft_sync();
            if (lane == 0) mbar_arrive(&sw->o_free);
            at += p.tiles + kStart;
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

// Joins the pieces of the sequences that several runs share: out = sum_i w_i O_i / sum_i w_i l_i with
// w_i = 2^{m_i - max m}, the pieces in order.  Where a sequence has up to 32 pieces, a warp takes a quarter row (a
// float4 a lane) with eight pieces' loads in flight; where it has more, a block takes an eighth (a float2 a lane), its
// warps every eighth piece, in one round of loads for a sequence over the whole card: the rounds' latency is all that
// such a join takes (9000 cycles in three rounds, 41.5 us of a call; 6400 in one).
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32, kFewParts = 32, kMostParts = 256, kMostGrid = kJoinThreads,
              kJoinBlocks = 5 * kSMs, kBatch = 20;
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
    auto part = [&](const Task& x, int i) { return po[slot(x, i) * (kLatent / 4) + x.side * 32 + lane]; };
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
    for (int t = blockIdx.x * kJoinWarps + warp; t < count[0] * NR * 4; t += gridDim.x * kJoinWarps) {
        const Task x = task(0, t);
        if (!x.live) continue;
        const float2 y = lane < x.h.parts ? ml[slot(x, lane)] : make_float2(-INFINITY, 0.f);
        float4 o[8];                          // the first loads go out before the weights are known
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < x.h.parts) o[k] = part(x, k);
        float mx = y.x;
        for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        const float w = y.x == -INFINITY ? 0.f : exp2_fast(y.x - mx);
        float total = w * y.y;
        for (int d = 16; d; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = 0; i < x.h.parts; i += 8) {
            if (i > 0) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (i + k < x.h.parts) o[k] = part(x, i + k);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float wk = __shfl_sync(0xffffffffu, w, (i + k) & 31);
                if (i + k < x.h.parts) add(acc, wk, o[k]);
            }
        }
        if (KDA_INDEX_OK(x.row, (int64_t)a.num_seqs * R, a.status)) {
            const float f = total == 0.f ? 0.f : 1.f / total;
            uint2 v;
            v.x = pack_bf16x2(acc.x * f, acc.y * f);
            v.y = pack_bf16x2(acc.z * f, acc.w * f);
            reinterpret_cast<uint2*>(a.out)[x.row * (kLatent / 4) + x.side * 32 + lane] = v;
            store_lse(x, mx, total);
        }
    }
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

// [rows, width] bf16, boxes of 64 channels x box_rows, 128-byte swizzle.
bool map_rows_2d(CUtensorMap* m, const void* base, int64_t rows, int width, int box_rows) {
    const auto fn = encode();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)width * 2};
    cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, es[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Query rows a block takes: the smallest of 16, 32, 64 that holds them all, else 64 in several groups.
int rows_a_block(int R) { return R <= 16 ? 16 : (R <= 32 ? 32 : 64); }
int groups_of(int R) { return (R + rows_a_block(R) - 1) / rows_a_block(R); }
int runs_of(int groups) { return groups < kSMs ? kSMs / groups : 1; }

template <int NR, bool ROPE>
cudaError_t launch(const LatentDecodeArgs& a, cudaStream_t s) {
    using G = Cfg<NR, ROPE>;
    const int R = a.tokens_per_seq * a.H, groups = groups_of(R), grid = runs_of(groups) * groups;
    const int64_t q_rows = (int64_t)a.num_seqs * R;
    const int box = a.c.page_size < kTile ? a.c.page_size : kTile;
    // a cache without pages: any readable row; every box then starts behind the map's last row
    const int64_t c_rows = a.c.num_pages > 0 ? (int64_t)a.c.num_pages * a.c.page_size : 1;
    const void* c_base = a.c.num_pages > 0 ? a.c.cache : a.workspace;
    Maps maps;
    if (!map_rows_2d(&maps.q, a.q_latent, q_rows, kLatent, NR) ||
        !map_rows_2d(&maps.qr, ROPE ? a.q_rope : a.q_latent, q_rows, ROPE ? kRope : kLatent, NR) ||
        !map_rows_2d(&maps.c, c_base, c_rows, kLatent + (ROPE ? kRope : 0), box))
        return cudaErrorInvalidValue;
    static std::atomic<bool> ready[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(latent_decode_kernel<NR, ROPE>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, (int)G::kBytes);
        if (e != cudaSuccess) return e;
        ready[dev].store(true, std::memory_order_release);
    }
    const cudaError_t e = launch_overlapped(latent_decode_kernel<NR, ROPE>, grid, kThreads, G::kBytes, s, maps, a, groups,
                                            (int)c_rows);
    return e != cudaSuccess ? e : launch_overlapped(latent_join_kernel<NR>, kJoinBlocks, kJoinThreads, 0, s, a, grid, groups);
}

template <int NR>
cudaError_t launch_rope(const LatentDecodeArgs& a, cudaStream_t s) {
    return a.c.rope_dim ? launch<NR, true>(a, s) : launch<NR, false>(a, s);
}

}  // namespace

size_t latent_decode_workspace_bytes(int tokens_per_seq, int H) {
    const int R = tokens_per_seq * H, groups = groups_of(R), grid = runs_of(groups) * groups;
    if (runs_of(groups) == 1) return Work<64>::ml_at(grid);         // one run: no piece goes to the workspace (settle)
    switch (rows_a_block(R)) {
        case 16: return Work<16>::bytes(grid);
        case 32: return Work<32>::bytes(grid);
        default: return Work<64>::bytes(grid);
    }
}

cudaError_t launch_latent_decode(const LatentDecodeArgs& a, cudaStream_t s) {
    switch (rows_a_block(a.tokens_per_seq * a.H)) {
        case 16: return launch_rope<16>(a, s);
        case 32: return launch_rope<32>(a, s);
        default: return launch_rope<64>(a, s);
    }
}

}  // namespace kda
