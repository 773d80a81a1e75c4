"""The unary loss without a GPU: its definition's gradients against differences, the binding's
checks against a stand-in for the library, and the library's own refusals, which return before
they touch a device."""
import ctypes as ct

import pytest

torch = pytest.importorskip("torch")

import dflash2_draft_block_gb300 as df2  # noqa: E402
from dflash2_draft_block_gb300 import _abi, build  # noqa: E402
from unary_loss_ref import reference  # noqa: E402

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
P, V, D = 12, 50, 24


@pytest.mark.parametrize("mul, cap", [(1.0, 0.0), (0.7, 0.0), (1.3, 4.0)])
def test_the_definition_against_differences(mul, cap):
    """Central differences of step s in 64 bits: third order s^2 (logits move by a few s) and
    2^-52 / s of losses near 5."""
    g = torch.Generator().manual_seed(3)
    h, W = torch.randn(P, D, generator=g).double(), torch.randn(V, D, generator=g).double() / 2
    t = torch.randint(0, V, (P,), generator=g)
    t[4] = -1
    w = torch.rand(P, generator=g).double()
    live = t >= 0

    def total(h, W):
        return float((reference(h, W, t, w, mul, cap)[0][0][live] * w[live]).sum())

    _, _, dh, dW = reference(h, W, t, w, mul, cap)[0]
    s = 2.0 ** -16
    for d, x, grad in ((torch.randn(P, D, generator=g).double(), "h", dh), (torch.randn(V, D, generator=g).double(), "W", dW)):
        up = total(h + s * d, W) if x == "h" else total(h, W + s * d)
        down = total(h - s * d, W) if x == "h" else total(h, W - s * d)
        size = float((grad.abs() * d.abs()).sum())
        assert abs((up - down) / (2 * s) - float((grad * d).sum())) < 1e-5 * size + 1e-9


class FakeLib:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith("_workspace_size"):
            return lambda *a: 256

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


def z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def args(**more):
    return dict(h=z(P, D), W_lm=z(V, D), targets=z(P, dtype=I32), **more)


def test_valid_calls_reach_the_library(fake):
    loss, lse = df2.unary_ce(**args())
    assert loss.shape == lse.shape == (P,)
    name, a = fake.calls[-1]
    assert name == "dflash2_unary_ce" and a[1:3] == (P, D) and a[4:7] == (V, 1.0, 0.0)
    mine = (z(P, dtype=F32), None)
    assert df2.unary_ce(**args(), out=mine)[0] is mine[0] and fake.calls[-1][1][9] == 0
    got = df2.unary_loss_grad(**args())
    assert got[2].dtype == BF and got[2].shape == (P, D) and got[3] is None
    got = df2.unary_loss_grad(**args(), dW=True, dtype=F32, row_weights=z(P, dtype=F32))
    assert got[2].dtype == got[3].dtype == F32 and got[3].shape == (V, D)
    dW = z(V, D, dtype=F32)
    got = df2.unary_loss_grad(**args(), dW=dW, accumulate=True, output_multiplier=0.5, final_logit_softcapping=30.0)
    name, a = fake.calls[-1]
    assert name == "dflash2_unary_loss_grad" and got[3] is dW and a[5:7] == (0.5, 30.0) and a[9] is True
    assert a[13] == 0 and a[15] == 1
    got = df2.unary_loss_grad(**args(), dh=None)
    assert got[2] is None and fake.calls[-1][1][12] == 0
    df2.unary_ce(z(P, D), z(V, D), z(3, 4, dtype=I32))  # targets of any shape


@pytest.mark.parametrize("change, error", [
    (dict(h=z(P, D, dtype=F32)), TypeError),
    (dict(h=z(D)), ValueError),
    (dict(h=z(P, 2 * D)[:, :D]), ValueError),
    (dict(W_lm=z(V, D + 8)), ValueError),
    (dict(W_lm=z(V, D, dtype=torch.float16)), TypeError),
    (dict(targets=z(P, dtype=torch.int64)), TypeError),
    (dict(targets=z(P + 1, dtype=I32)), ValueError),
    (dict(row_weights=z(P)), TypeError),
    (dict(row_weights=z(P + 1, dtype=F32)), ValueError),
    (dict(dh=z(P, D + 1)), ValueError),
    (dict(dh=z(P, D, dtype=torch.float16)), TypeError),
    (dict(dh="yes"), TypeError),
    (dict(dW=z(V, 2 * D)[:, :D]), ValueError),
    (dict(accumulate=True), ValueError),
    (dict(accumulate=True, dW=True), ValueError),
    (dict(dtype=torch.float16), TypeError),
    (dict(out=(z(P), z(P, dtype=F32))), TypeError),
    (dict(out=(z(P - 1, dtype=F32), None)), ValueError),
    (dict(workspace=z(8)), ValueError),
    (dict(dev_status=z(1)), TypeError),
])
def test_refusals(fake, change, error):
    with pytest.raises(error):
        df2.unary_loss_grad(**{**args(), **change})
    assert not fake.calls


def test_library_refusals():
    build.build()
    lib = _abi.load()
    base = 1 << 24

    def call(P=P, D=D, V=V, mul=1.0, cap=0.0, h=base, W=2 * base, t=3 * base, w=0, acc=0, loss=4 * base, lse=5 * base,
             dh=6 * base, dhd=0, dW=7 * base, dWd=0, ws=8 * base, n=1 << 40):
        return lib.dflash2_unary_loss_grad(h, P, D, W, V, mul, cap, t, w, acc, loss, lse, dh, dhd, dW, dWd, ws, n, 0, None)

    inf, nan = float("inf"), float("nan")
    for bad in (dict(P=-1), dict(D=0), dict(V=0), dict(mul=0.0), dict(mul=-1.0), dict(mul=nan), dict(mul=inf), dict(cap=-1.0),
                dict(cap=nan), dict(cap=inf), dict(h=0), dict(W=0), dict(t=0), dict(loss=0), dict(dhd=2), dict(dWd=-1),
                dict(dh=base), dict(dh=2 * base), dict(dW=2 * base + 16), dict(dW=6 * base), dict(loss=5 * base + 4),
                dict(lse=4 * base), dict(loss=3 * base), dict(loss=6 * base + 8)):
        assert call(**bad) == 1, bad
    for bad in (dict(D=20), dict(P=(1 << 20) + 1), dict(D=(1 << 20) + 8), dict(V=(1 << 24) + 1), dict(h=base + 8), dict(W=2 * base + 2),
                dict(dh=6 * base + 8), dict(dW=7 * base + 4), dict(t=3 * base + 2), dict(loss=4 * base + 1),
                dict(lse=5 * base + 2), dict(w=9 * base + 1), dict(cap=1e-40), dict(cap=1e-20, mul=1e20)):
        assert call(**bad) == 2, bad
    assert call(P=0, acc=1) == 0 and call(P=0, dW=0) == 0


def test_workspace_sizes():
    """They grow with the rows up to the size of a piece, and hold less without gradients."""
    build.build()
    lib = _abi.load()
    ce, both = lib.dflash2_unary_ce_workspace_size, lib.dflash2_unary_loss_grad_workspace_size
    assert ce(0, 64, 100) == 0 and ce(8, 60, 100) == 0 and both(8, 64, 0, 1, 1) == 0
    P, D, V = 4096, 4096, 151936
    assert ce(P, D, V) < both(P, D, V, 0, 1) < both(P, D, V, 1, 1)
    copy = lambda n: n * (2 * D + 16)  # noqa: E731  (the copy of h, and a few words a row)
    assert both(4 * P, D, V, 1, 0) < (5 << 30) + copy(4 * P)
    assert both(64 * P, D, V, 1, 0) < (5 << 30) + copy(64 * P)
    assert both(64 * P, D, V, 1, 1) - both(64 * P, D, V, 1, 0) == V * D * 4
    assert ce(64 * P, D, V) < (1 << 30) + (1 << 20) + copy(64 * P)
