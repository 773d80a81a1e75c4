"""How dh's product is cut, against its cost counted another way: every item is dealt to its cluster with
the K steps that it really has, and the slowest cluster's steps are added up.

The rule's own time takes every part as long as the longest; dealt out, a cluster may hold shorter
ones, each by one step.  So no choice that the rule passed over is better, counted this way, than the one
it took by more than a step (0.3 us) for each round of parts."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dflash2_draft_block_gb300", "csrc")

CODE = r"""
#include <cstdint>
#define __host__
#define __device__
#include "loss_tiles.h"
using namespace df2;
extern "C" int64_t way_key(int ways, int64_t rest, int64_t steps, int64_t units, int quad) {
    return loss_way_key(ways, rest, steps, units, quad != 0);
}
extern "C" int way_limit(int64_t steps) { return loss_way_limit(steps); }
// The steps of the slowest of `units` clusters, and those of all together.
extern "C" int64_t slowest(int tiles, int ways, int units, int steps, int64_t* all) {
    const int rest = tiles % units;
    const LossSplit work{tiles - rest, rest, ways};
    int64_t worst = 0;
    *all = 0;
    for (int u = 0; u < units; ++u) {
        int64_t mine = 0;
        for (int i = u; i < work.items(); i += units) {
            int k0, k1;
            loss_steps(i, work, steps, &k0, &k1);
            mine += k1 - k0;
        }
        worst = mine > worst ? mine : worst;
        *all += mine;
    }
    return worst;
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("split")
    (d / "t.cpp").write_text(CODE)
    subprocess.run([gxx, "-std=c++17", "-O2", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, str(d / "t.cpp"), "-o",
                    str(d / "t.so")], check=True)
    lib = ctypes.CDLL(str(d / "t.so"))
    lib.way_key.restype = lib.slowest.restype = ctypes.c_int64
    lib.way_key.argtypes = [ctypes.c_int] + [ctypes.c_int64] * 3 + [ctypes.c_int]
    lib.way_limit.argtypes = [ctypes.c_int64]
    lib.slowest.argtypes = [ctypes.c_int] * 4 + [ctypes.POINTER(ctypes.c_int64)]
    return lib


def test_no_other_split_is_faster(lib):
    rng = random.Random(3)
    cut = 0
    for _ in range(400):
        units, quad = rng.choice([(36, 1), (38, 1), (76, 0)])
        tiles, steps = rng.randint(1, 200), rng.choice([rng.randint(1, 100), rng.randint(1, 4000)])
        rest, limit = tiles % units, lib.way_limit(steps)
        chosen = min(lib.way_key(s, rest, steps, units, quad) for s in range(1, limit + 1)) & 127

        def cost(ways):
            total = ctypes.c_int64()
            busy = lib.slowest(tiles, ways, units, steps, ctypes.byref(total))
            assert total.value == tiles * steps  # every step once
            # a part goes out and comes back: 256 x 256 sums of 4 bytes a pair, twice, at 4 TB/s
            moved = ways * rest * (2 if quad else 1) * 2 * 256 * 256 * 4 / 4e3 if ways > 1 else 0.0
            return 300.0 * busy + moved + (3000 if ways > 1 else 0)

        took = cost(chosen)
        cut += chosen > 1
        for ways in range(1, limit + 1):
            if ways == 1 or ways * rest <= 8 * units:
                rounds = -(-rest * ways // units)
                # (131 and 262 ns a part, in whole numbers: 0.1 a part)
                assert took <= cost(ways) + 300.0 * rounds + 0.2 * rest * (ways + chosen), (units, tiles, steps, chosen, ways)
    assert cut > 100
