// kda_latent_runs.h -- how a run of the latent decode's line of tiles is walked.  Integer arithmetic only, compiled for
// the device and, by the tests, for the host.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define KDA_RUNS_FN __host__ __device__ __forceinline__
#else
#define KDA_RUNS_FN inline
#endif

namespace kda {
namespace latent {

constexpr int kTile = 64;                     // cached rows a tile of the bf16 decode
// A sequence's places in the line: its tiles, behind START places that stand for what starting a piece costs a
// block (queries in, O out), so that runs with many pieces get fewer tiles.
constexpr int kStart = 1;                     // of the bf16 decode

struct Piece {                                // a run's share of one sequence
    int n, len, off, tiles, all;              // sequence, its length, first tile, tiles here, tiles in all
};

template <int TILE = kTile>
KDA_RUNS_FN int tiles_of(int len) { return len > TILE ? (len - 1) / TILE + 1 : 1; }

// The first tile of run p of `runs` over `total` tiles (a 32-bit division where it fits, a fifth of the time), and
// the run that holds tile x.
KDA_RUNS_FN int64_t run_begin(int64_t total, int runs, int p) {
    return total < (1 << 23) ? (int64_t)((uint32_t)total * (uint32_t)p / (uint32_t)runs) : total * p / runs;
}
KDA_RUNS_FN int run_of(int64_t total, int runs, int64_t x) { return (int)(((x + 1) * runs - 1) / total); }

// Walks the sequences of a run of tiles of TILE rows; length(n) is sequence n's length.
template <int TILE, int START>
struct RunWalkOf {
    int n, off, lead, len;                    // next sequence, its first tile here, start places before it, its length or -1
    int64_t left;                             // places of the run that are left
    template <typename Length>
    KDA_RUNS_FN bool next(int num_seqs, const Length& length, Piece& p) {
        if (left <= 0 || n >= num_seqs) return false;
        p.n = n;
        p.len = len >= 0 ? len : length(n);
        len = -1;
        p.all = tiles_of<TILE>(p.len);
        p.off = off;
        const int64_t behind = left - lead;   // places of the run behind the sequence's start places
        p.tiles = behind < p.all - off ? (behind > 0 ? (int)behind : 0) : p.all - off;
        left = behind - p.tiles;
        lead = START;
        off = 0;
        ++n;
        return p.tiles > 0;                   // a run may end inside the start places
    }
};
using RunWalk = RunWalkOf<kTile, kStart>;

// Whether a piece's result is its sequence's, and goes to the output.  Other pieces go to the workspace, which a line in
// one run does not have: there every piece is the only one of its sequence (settle), also where a length that grew since
// the line was measured makes it look cut.
KDA_RUNS_FN void settle(Piece& p, int runs) {
    if (runs == 1) p.all = p.off + p.tiles;
}
KDA_RUNS_FN bool is_whole(const Piece& p) { return p.off == 0 && p.tiles == p.all; }

}  // namespace latent
}  // namespace kda
