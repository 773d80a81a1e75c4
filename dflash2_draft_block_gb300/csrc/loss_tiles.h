// How the unary loss's products are cut into tiles, for host and device.
#pragma once

#include <stdint.h>

namespace df2 {

constexpr int kLossStats = 64;    // columns that share a maximum
constexpr int kLossGroup = 16;    // M units that share a pass over W (8: 3% slower; 32: 2%)

// Tiles of clusters: `across` by `shared`.  A quad (a cluster of two CTA pairs) takes two tiles
// that are neighbours along `shared` and so have an operand in common; where `shared` is odd, the
// last of it with two of the other index, which have nothing in common.
__host__ __device__ inline int loss_cluster_tiles(int across, int shared, bool quad) {
    return quad ? across * (shared / 2) + (shared & 1) * ((across + 1) / 2) : across * shared;
}

struct LossTile {
    int mu, nt;     // M unit and N tile, of 256 each; either may be one past the end in a quad
    int part;       // -1: the whole sum; else the place of this part of it among the parts
    int k0, k1;     // K steps
    bool alone;     // the pairs of a cluster share nothing
};

// The clusters' work: `whole` tiles, then `rest` tiles in `ways` parts each (1: whole, too).
struct LossSplit {
    int whole, rest, ways;
    __host__ __device__ int items() const { return whole + rest * ways; }
};

// The K steps of item i of them: all that the issuer of the products has to know of it.
__host__ __device__ inline void loss_steps(int i, const LossSplit& work, int k_total, int* k0, int* k1) {
    const bool split = work.ways > 1 && i >= work.whole;
    const int kind = split ? (i - work.whole) / work.rest : 0;
    *k0 = split ? int(int64_t(k_total) * kind / work.ways) : 0;
    *k1 = split ? int(int64_t(k_total) * (kind + 1) / work.ways) : k_total;
}

// Item i of them, for pair `which` of the cluster.  LOGITS (h W^T): M fastest in groups, so that W
// streams past while a group's rows of h stay in L2; quads take two M units.  The gradients: N
// fastest, so that the clusters of a moment share g's rows; quads take two N tiles.
template <bool LOGITS, bool QUAD>
__host__ __device__ inline LossTile loss_tile(int i, int n_mu, int n_nt, const LossSplit& work, int k_total, int which) {
    constexpr int kPairs = QUAD ? 2 : 1;
    LossTile t;
    const bool split = work.ways > 1 && i >= work.whole;
    t.part = split ? i - work.whole : -1;  // the parts of a kind together, of all tiles
    const int kind = split ? t.part / work.rest : 0;
    const int j = split ? i - kind * work.rest : i;
    t.alone = false;
    if (LOGITS) {
        constexpr int kRun = kLossGroup / kPairs;
        const int n_m = n_mu / kPairs, odd = j - n_m * n_nt;
        if (odd < 0) {
            const int first = j / (kRun * n_nt) * kRun, left = n_m - first;
            const int wide = kRun < left ? kRun : left, rest = j - first * n_nt;
            t.mu = (first + rest % wide) * kPairs + which;
            t.nt = rest / wide;
        } else {
            t.mu = n_mu - 1;
            t.nt = odd * 2 + which;
            t.alone = true;
        }
    } else {
        const int n_n = n_nt / kPairs, odd = j - n_mu * n_n;
        if (odd < 0) {
            t.nt = j % n_n * kPairs + which;
            t.mu = j / n_n;
        } else {
            t.nt = n_nt - 1;
            t.mu = odd * 2 + which;
            t.alone = true;
        }
    }
    loss_steps(i, work, k_total, &t.k0, &t.k1);
    return t;
}

// dh's product has few tiles and long sums (of V): its tiles go to the clusters whole as long as
// that fills rounds of all of them, and what is left over is cut along V.  Into how many parts:
// the busiest cluster's steps (of 64) at 0.3 us, and the parts' way out and back at 4 TB/s, in
// ns.  The live rows decide, so it is worked out on the device, by each kernel that needs it;
// in whole numbers, so that all find the same.
constexpr int kLossWays = 64;        // parts of a tile at most
constexpr int kLossPartTiles = 8;    // parts a cluster at most, on average
__host__ __device__ inline int loss_way_limit(int64_t steps) {
    const int64_t s = (steps + 3) / 4;
    return int(s < kLossWays ? s : kLossWays);
}
// `ways` ways, as a key whose least is the best: the time, and of equal ones the fewer ways.
__host__ __device__ inline int64_t loss_way_key(int ways, int64_t rest, int64_t steps, int64_t units, bool quad) {
    if (ways > 1 && ways * rest > kLossPartTiles * units) return INT64_MAX;
    int64_t ns = (rest * ways + units - 1) / units * ((steps + ways - 1) / ways) * 300;
    if (ways > 1) ns += 3000 + ways * rest * (quad ? 262 : 131);
    return ns * 128 + ways;
}

}  // namespace df2
