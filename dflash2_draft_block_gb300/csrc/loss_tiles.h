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
    int split;
    int k0, k1;     // K steps
    bool alone;     // the pairs of a cluster share nothing
};

// Tile i of the clusters' tiles * splits, for pair `which` of the cluster.  LOGITS (h W^T): M fastest
// in groups, so that W streams past while a group's rows of h stay in L2; quads take two M units.
// The gradients: N fastest, so that the clusters of a moment share g's rows; quads take two N
// tiles.
template <bool LOGITS, bool QUAD>
__host__ __device__ inline LossTile loss_tile(int i, int n_mu, int n_nt, int splits, int k_total, int which) {
    constexpr int kPairs = QUAD ? 2 : 1;
    const int tiles = LOGITS ? loss_cluster_tiles(n_nt, n_mu, QUAD) : loss_cluster_tiles(n_mu, n_nt, QUAD);
    LossTile t;
    t.split = i / tiles;
    const int j = i - t.split * tiles;
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
    t.k0 = int(int64_t(k_total) * t.split / splits);
    t.k1 = int(int64_t(k_total) * (t.split + 1) / splits);
    return t;
}

// How many ways dh's product is split along V, for `tiles` tiles of `steps` steps (of 64) on
// `units` clusters: the busiest cluster's steps at 0.3 us, and the partial sums' way out and
// back at 4 TB/s, in ns.  The live rows decide, so it is worked out on the device, by each
// kernel that needs it; in whole numbers, so that all find the same.
constexpr int kLossSplits = 64;
constexpr int64_t kLossPartial = int64_t(1) << 27;  // fp32 sums held at most
__host__ __device__ inline int loss_split_limit(int64_t steps) {
    const int64_t s = (steps + 3) / 4;
    return int(s < kLossSplits ? s : kLossSplits);
}
// s ways, as a key whose least is the best: the time, and of equal ones the fewer ways.
__host__ __device__ inline int64_t loss_split_key(int s, int64_t tiles, int64_t steps, int64_t units, int64_t rows,
                                                  int64_t D) {
    if (s > 1 && s * rows * D > kLossPartial) return INT64_MAX;
    int64_t ns = (tiles * s + units - 1) / units * ((steps + s - 1) / s) * 300;
    if (s > 1) ns += 3000 + s * rows * D * 2 / 1000;
    return ns * 128 + s;
}

}  // namespace df2
