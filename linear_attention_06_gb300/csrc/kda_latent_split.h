// kda_latent_split.h -- how many blocks of the latent prefill share the keys of a block of queries.  Integer arithmetic
// on sizes that the host knows; the tests call it as it stands.
#pragma once

#include <stdint.h>

namespace kda {
namespace latent {

// A share of an average sequence's key tiles, the join, which takes about as long as three tiles (3 us), and the
// clusters that do not start with the first: those of slots without queries end at once, but a cluster's place takes a
// sixteenth of a tile a block to be given away again.  All in key tiles of 1.4 us; measured, dk = 192, in fours with 36
// clusters at once, an average sequence of 4 tiles: 12.3 us in 36 clusters, 15.6 in 44, 18.5 in 56, 25.0 in 68.
constexpr int kJoinTiles = 3;
inline int64_t split_cost(int64_t tiles, int64_t clusters, int64_t at_once, int parts) {
    if (parts == 1) return tiles;
    const int64_t late = clusters > at_once ? clusters - at_once : 0;
    return (tiles + parts - 1) / parts + kJoinTiles + (late * parts + 15) / 16;
}

// The cheapest of 1, 2, 4 and 8, each part with a tile of an average sequence and all clusters with queries (`busy`
// of `clusters`) at work at the same time; at_once(parts) is how many the device runs.
template <typename AtOnce>
int split_of(int64_t tiles, int64_t busy, int64_t clusters, const AtOnce& at_once) {
    int best = 1;
    int64_t least = tiles;
    for (int parts = 2; parts <= 8 && parts <= tiles; parts *= 2) {
        if (tiles - (tiles + parts - 1) / parts < kJoinTiles) continue;
        const int64_t room = at_once(parts), cost = split_cost(tiles, clusters, room, parts);
        if (busy > room || cost > least) continue;
        best = parts;
        least = cost;
    }
    return best;
}

}  // namespace latent
}  // namespace kda
