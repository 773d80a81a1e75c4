"""Dropout without a GPU: the random words against published values, the binding's checks
against a stand-in for the library, and the library's own refusals, which return before they
touch a device."""
import ctypes as ct

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import dflash2_draft_block_gb300 as df2  # noqa: E402
from dflash2_draft_block_gb300 import _abi, build  # noqa: E402
from dropout_words import dropped, philox, threshold, words  # noqa: E402

BF, F32, I64 = torch.bfloat16, torch.float32, torch.int64
VP = ct.c_void_p


def test_words_against_published_values():
    """The known answers that the generator's authors publish with it."""
    ones = 0xFFFFFFFF
    for counter, key, want in [
            ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            ((ones,) * 4, (ones,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
             (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))]:
        assert tuple(int(w) for w in philox(counter, key)) == want


def test_words_order():
    first = [int(w) for w in philox((0, 0, 0, 0), (0, 0))]
    assert [int(w) for w in words(range(8), 0, 0)] == [v for w in first for v in (w & 0xFFFF, w >> 16)]
    assert threshold(0.1) == 6554 and threshold(1.0) == 65536 and threshold(0.0) == 0


def test_the_rate_is_kept():
    """2^20 words: the share dropped is within 5 standard deviations of the rate."""
    n = 1 << 20
    for rate in (0.1, 0.5, 0.9):
        _, keep = dropped(np.ones(n), rate, 1234567890123, 42)
        assert abs((1 - keep.mean()) - rate) < 5 * (rate * (1 - rate) / n) ** 0.5 + 2.0 ** -16


class FakeLib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def fake(monkeypatch):
    lib = FakeLib()
    monkeypatch.setattr(df2, "lib", lambda: lib)
    monkeypatch.setattr(df2, "_on_device", lambda t: True)
    monkeypatch.setattr(df2, "_stream", lambda stream, device: ct.c_void_p(0))
    return lib


def t(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def test_valid_calls_reach_the_library(fake):
    assert df2.dropout(t(6, 24), 0.1, 7).dtype == BF
    x = t(6, 40)[:, :24]
    out = df2.dropout(x, 0.1, 7, 3, residual=t(6, 24, dtype=F32))
    assert out.dtype == F32 and out.shape == (6, 24)
    name, a = fake.calls[-1]
    assert name == "dflash2_dropout" and a[1:8] == (0, 6, 24, 40, 0.1, 7, 3) and a[8] == 0
    assert df2.dropout(t(2, 3, 8), 0.5, (1 << 64) - 1).shape == (2, 3, 8)
    assert fake.calls[-1][1][2:5] == (1, 48, 48)
    assert df2.dropout(t(5), 0.5, 0).shape == (5,)
    draw = torch.zeros(1, dtype=I64)
    df2.dropout(t(5, 8), 0.5, 0, draw)
    assert fake.calls[-1][1][8] == draw.data_ptr()
    acc = t(5, 8, dtype=F32)
    assert df2.dropout_grad(t(5, 8), 0.5, 0, accumulate=True, out=acc) is acc
    a = fake.calls[-1][1]
    assert a[9] == a[11] == acc.data_ptr()
    assert df2.dropout_grad(t(5, 8), 0.5, 0, dtype=F32).dtype == F32
    before = len(fake.calls)
    assert df2.dropout(t(0, 8), 0.5, 0).shape == (0, 8) and len(fake.calls) == before


@pytest.mark.parametrize("call, error", [
    (lambda: df2.dropout(t(4, 8), 1.5, 0), ValueError),
    (lambda: df2.dropout(t(4, 8), float("nan"), 0), ValueError),
    (lambda: df2.dropout(t(4, 8), 0.1, -1), ValueError),
    (lambda: df2.dropout(t(4, 8), 0.1, 1 << 64), ValueError),
    (lambda: df2.dropout(t(4, 8), 0.1, 0.5), TypeError),
    (lambda: df2.dropout(t(4, 8), 0.1, 0, -1), ValueError),
    (lambda: df2.dropout(t(4, 8), 0.1, 0, 1.5), TypeError),
    (lambda: df2.dropout(t(4, 8), 0.1, 0, t(1)), TypeError),
    (lambda: df2.dropout(t(4, 8), 0.1, 0, t(2, dtype=I64)), ValueError),
    (lambda: df2.dropout(t(4, 8, dtype=torch.float16), 0.1, 0), TypeError),
    (lambda: df2.dropout(t(8, 4).t(), 0.1, 0), ValueError),
    (lambda: df2.dropout(t(2, 4, 8)[:, :, ::2], 0.1, 0), ValueError),
    (lambda: df2.dropout([1.0], 0.1, 0), TypeError),
    (lambda: df2.dropout(t(4, 8), 0.1, 0, residual=t(4, 9)), ValueError),
    (lambda: df2.dropout(t(4, 8), 0.1, 0, residual=t(4, 8), dtype=F32), TypeError),
    (lambda: df2.dropout(t(4, 8), 0.1, 0, residual=t(4, 8, dtype=F32), out=t(4, 8)), TypeError),
    (lambda: df2.dropout(t(4, 8), 0.1, 0, dtype=torch.float16), TypeError),
    (lambda: df2.dropout(t(4, 8), 0.1, 0, dtype=F32, out=t(4, 8)), TypeError),
    (lambda: df2.dropout(t(4, 8), 0.1, 0, out=t(8, 4)), ValueError),
    (lambda: df2.dropout_grad(t(4, 8), 0.1, 0, accumulate=True), ValueError),
])
def test_refusals(fake, call, error):
    with pytest.raises(error):
        call()
    assert not fake.calls


def test_library_refusals():
    build.build()
    f = _abi.load().dflash2_dropout
    x = 1 << 20

    def call(x=x, xd=0, N=4, D=8, xl=8, rate=0.5, at=0, res=0, rl=0, out=1 << 24, od=0, ol=8):
        return f(x, xd, N, D, xl, rate, 1, 2, at, res, rl, out, od, ol, None)

    assert call(N=0) == 0
    for bad in (dict(xd=2), dict(od=-1), dict(rate=-0.1), dict(rate=1.01), dict(rate=float("nan")), dict(N=-1),
                dict(D=0), dict(xl=7), dict(ol=7), dict(res=x, rl=7), dict(x=0), dict(out=0)):
        assert call(**bad) == 1, bad
    for bad in (dict(N=1 << 38), dict(D=1 << 41, xl=1 << 41, ol=1 << 41), dict(x=x + 1), dict(out=(1 << 24) + 1),
                dict(od=1, out=(1 << 24) + 2), dict(at=x + 4), dict(res=(1 << 22) + 1, rl=8)):
        assert call(**bad) == 2, bad
    # overlaps other than in place: shifted, another dtype, other rows
    for bad in (dict(out=x + 2), dict(out=x, od=1), dict(out=x, ol=16), dict(out=x - 2),
                dict(res=(1 << 24) + 2, rl=8), dict(res=1 << 24, rl=16)):
        assert call(**bad) == 1, bad
