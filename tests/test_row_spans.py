"""Whether two matrices share bytes, compiled on the CPU from the header the calls use, against the sets of
their bytes: exact where their rows are equally far apart, never a miss where they are not."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dflash2_draft_block_gb300", "csrc")

CODE = r"""
#include "row_spans.h"
extern "C" int share(uint64_t a, int64_t a_row, int64_t a_ld, uint64_t b, int64_t b_row, int64_t b_ld, int64_t N) {
    return df2::rows_share_bytes(df2::RowSpan{uintptr_t(a), a_row, a_ld}, df2::RowSpan{uintptr_t(b), b_row, b_ld}, N);
}
"""


@pytest.fixture(scope="module")
def share(tmp_path_factory):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("spans")
    (d / "t.cpp").write_text(CODE)
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, str(d / "t.cpp"), "-o",
                    str(d / "t.so")], check=True)
    f = ctypes.CDLL(str(d / "t.so")).share
    f.argtypes = [ctypes.c_uint64, ctypes.c_int64, ctypes.c_int64, ctypes.c_uint64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64]
    return f


def bytes_of(at, row, ld, N):
    return {at + n * ld + i for n in range(N) for i in range(row)}


def test_against_sets_of_bytes(share):
    rng = random.Random(1)
    seen = set()
    for _ in range(20000):
        N, a_row, b_row = rng.randint(1, 5), rng.randint(1, 9), rng.randint(1, 9)
        a_ld = rng.randint(a_row, 20)
        b_ld = max(b_row, a_ld) if rng.random() < 0.8 else rng.randint(b_row, 20)
        a, b = rng.randint(100, 220), rng.randint(100, 220)
        want = bool(bytes_of(a, a_row, a_ld, N) & bytes_of(b, b_row, b_ld, N))
        got = bool(share(a, a_row, a_ld, b, b_row, b_ld, N))
        assert got == want if a_ld == b_ld or N == 1 else got or not want, (a, a_row, a_ld, b, b_row, b_ld, N)
        seen.add((got, want, a_ld == b_ld))
    assert {(True, True, True), (False, False, True), (True, True, False), (False, False, False)} <= seen


def test_halves_of_a_wide_matrix(share):
    base, D, ld = 1 << 40, 1000 * 4, 2000 * 4
    assert not share(base, D, ld, base + D, D, ld, 1 << 30)
    assert not share(base + D, D, ld, base, D, ld, 1 << 30)
    assert share(base, D, ld, base + D - 4, D, ld, 2) and share(base, D + 4, ld, base + D, D, ld, 2)
    assert not share(base, D, ld, base + ld, D, ld, 1) and share(base, D, ld, base + ld, D, ld, 2)
    assert not share(base, ld, 2 * ld, base + ld, ld, 2 * ld, 1 << 20)  # every other row
