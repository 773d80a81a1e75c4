"""The unary loss's tiles, compiled on the CPU from the header that host and device share, and
swept over shapes: every 256 x 256 tile and every K step of it is computed once, the clusters of
a launch stay inside the tiles, neighbours that share an operand have the same one, and the split
of dh's product fits its space and is one that no other beats."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dflash2_draft_block_gb300", "csrc")

CODE = r"""
#include <cstdint>
#include <cstring>
#define __host__
#define __device__
#include "loss_tiles.h"
using namespace df2;
// 0: every tile and K step once, and the parts of a tile where their sum looks for them; counts:
// [n_mu][n_nt][k_total] bytes of scratch
template <bool L, bool Q>
static int sweep(int n_mu, int n_nt, int rest, int ways, int k_total, uint8_t* counts) {
    const int pairs = Q ? 2 : 1;
    const int tiles = L ? loss_cluster_tiles(n_nt, n_mu, Q) : loss_cluster_tiles(n_mu, n_nt, Q);
    if (rest > tiles) rest = tiles;
    const LossSplit work{tiles - rest, rest, ways};
    std::memset(counts, 0, size_t(n_mu) * n_nt * k_total);
    if (work.items() != tiles - rest + rest * ways) return 8;
    for (int i = 0; i < work.items(); ++i) {
        LossTile t[2];
        for (int q = 0; q < pairs; ++q) {
            t[q] = loss_tile<L, Q>(i, n_mu, n_nt, work, k_total, q);
            if (t[q].mu < 0 || t[q].nt < 0 || t[q].mu > n_mu || t[q].nt > n_nt) return 1;
            if (t[q].k0 < 0 || t[q].k1 > k_total || t[q].k0 > t[q].k1) return 2;
            const bool split = ways > 1 && i >= work.whole;
            if (!split && (t[q].part != -1 || t[q].k0 != 0 || t[q].k1 != k_total)) return 9;
            if (split) {
                const int tile = t[q].part % rest;  // the part's tile, and the whole one that its sum is
                const LossTile w = loss_tile<L, Q>(work.whole + tile, n_mu, n_nt, work, k_total, q);
                if (t[q].part < 0 || t[q].part >= rest * ways || w.mu != t[q].mu || w.nt != t[q].nt) return 10;
                if (t[q].k0 == t[q].k1) return 11;
            }
            if (t[q].mu >= n_mu || t[q].nt >= n_nt) {
                if (!Q || q != 1 || !t[q].alone) return 3;
                continue;
            }
            for (int k = t[q].k0; k < t[q].k1; ++k) ++counts[(size_t(t[q].mu) * n_nt + t[q].nt) * k_total + k];
        }
        if (Q) {  // one list of K steps, and the shared operand where there is one
            if (t[0].alone != t[1].alone || t[0].k0 != t[1].k0 || t[0].k1 != t[1].k1 || t[0].part != t[1].part) return 4;
            if (!t[0].alone && (L ? t[0].nt != t[1].nt : t[0].mu != t[1].mu)) return 5;
        } else if (t[0].alone) {
            return 6;
        }
    }
    for (size_t i = 0; i < size_t(n_mu) * n_nt * k_total; ++i)
        if (counts[i] != 1) return 7;
    return 0;
}
extern "C" int sweep_tiles(int logits, int quad, int n_mu, int n_nt, int rest, int ways, int k_total, uint8_t* counts) {
    if (logits) return quad ? sweep<true, true>(n_mu, n_nt, rest, ways, k_total, counts) : sweep<true, false>(n_mu, n_nt, rest, ways, k_total, counts);
    return quad ? sweep<false, true>(n_mu, n_nt, rest, ways, k_total, counts) : sweep<false, false>(n_mu, n_nt, rest, ways, k_total, counts);
}
extern "C" int64_t way_key(int ways, int64_t rest, int64_t steps, int64_t units, int quad) {
    return loss_way_key(ways, rest, steps, units, quad != 0);
}
extern "C" int way_limit(int64_t steps) { return loss_way_limit(steps); }
extern "C" int part_tiles() { return kLossPartTiles; }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("tiles")
    (d / "t.cpp").write_text(CODE)
    subprocess.run([gxx, "-std=c++17", "-O2", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, str(d / "t.cpp"), "-o",
                    str(d / "t.so")], check=True)
    lib = ctypes.CDLL(str(d / "t.so"))
    lib.way_key.restype = ctypes.c_int64
    lib.way_key.argtypes = [ctypes.c_int] + [ctypes.c_int64] * 3 + [ctypes.c_int]
    lib.way_limit.argtypes = [ctypes.c_int64]
    return lib


def test_every_tile_once(lib):
    rng = random.Random(1)
    shapes = [(m, n) for m in range(1, 8) for n in range(1, 8)]
    shapes += [(rng.randint(1, 60), rng.randint(1, 60)) for _ in range(60)] + [(16, 97), (33, 16), (32, 17), (17, 1), (1, 50)]
    counts = (ctypes.c_uint8 * (70 * 100 * 64))()
    for m, n in shapes:
        for quad in (0, 1):
            assert lib.sweep_tiles(1, quad, m, n, 0, 1, 3, counts) == 0, (m, n, quad)
            for rest, ways, steps in ((0, 1, 1), (9, 1, 5), (1, 3, 7), (7, 5, 5), (35, 8, 50), (9999, 4, 16)):
                if m * n * steps < 70 * 100 * 64:
                    assert lib.sweep_tiles(0, quad, m, n, rest, ways, steps, counts) == 0, (m, n, quad, rest, ways, steps)


def test_ways(lib):
    """The parts fit their space, none is empty, and with one part to a cluster and round nothing is cut."""
    rng = random.Random(2)
    none = (1 << 63) - 1
    for _ in range(3000):
        units, quad = rng.choice([(36, 1), (76, 0)])
        steps, rest = rng.randint(1, 5000), rng.randint(0, units - 1)
        limit = lib.way_limit(steps)
        assert 1 <= limit <= min(64, max(1, (steps + 3) // 4))
        keys = {s: lib.way_key(s, rest, steps, units, quad) for s in range(1, limit + 1)}
        best = min(keys.values())
        s = best & 127
        assert best != none and keys[s] == best and 1 <= s <= limit <= steps + 3
        assert s == 1 or s * rest <= lib.part_tiles() * units
        assert s <= steps
        assert rest or s == 1
