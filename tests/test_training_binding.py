"""The training calls' refusals, on the CPU: the binding against a stand-in for the library
(CPU tensors standing in for device tensors), and the library's own argument checks, which
return before they touch a device."""
import ctypes as ct
import math

import pytest

torch = pytest.importorskip("torch")

import dflash2_draft_block_gb300 as df2  # noqa: E402
from dflash2_draft_block_gb300 import _abi, build, optim  # noqa: E402

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
VP = ct.c_void_p


class FakeLib:
    """Records each call; status 0; workspace queries answer 256 bytes."""

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


def bf(*s):
    return torch.zeros(s, dtype=BF)


def f32(*s):
    return torch.zeros(s, dtype=F32)


def i32(*s):
    return torch.zeros(s, dtype=I32)


P, K, r, V, D, N = 12, 4, 16, 50, 24, 10


def sel():
    return dict(pred=i32(P), targets=i32(P), topk_ids=i32(P, K), topk_vals=f32(P, K), G=f32(P, r), A=bf(V, r), Bc=bf(V, r))


# ---------------------------------------------------------------- binding --

def test_valid_calls_reach_the_library(fake):
    assert df2.embedding(bf(V, D), i32(2, 5)).shape == (2, 5, D)
    assert df2.embedding(bf(V, D), i32(N), dtype=F32).dtype == F32
    out = f32(N, D + 8)[:, 3:3 + D]
    assert df2.embedding(bf(V, 2 * D)[:, :D], i32(N), out=out) is out
    name, args = fake.calls[-1]
    assert name == "dflash2_embedding" and args[2:5] == (V, D, 2 * D) and args[10] == D + 8
    assert df2.embedding_grad(bf(N, D), i32(N), V).shape == (V, D)
    assert df2.embedding_grad(f32(2, 5, D), i32(2, 5), V, dtype=BF).dtype == BF
    got = df2.selector_loss_grad(**sel(), row_weights=f32(P))
    assert [tuple(t.shape) for t in got] == [(P,), (P,), (P, K), (P, r), (V, r), (V, r)]
    got = df2.selector_loss_grad(**sel(), dA=None, dBc=bf(V, r), accumulate=True)
    assert got[4] is None and got[5].dtype == BF
    opt = df2.AdamW([f32(5, 3), bf(7)], [f32(5, 3), bf(7)], state_bits=8, master_weights=True)
    opt.step(grad_scale=f32(1))
    name, args = fake.calls[-1]
    assert name == "dflash2_adamw" and args[1:3] == (2, 8) and args[6] == 1 and opt.step_count == 1
    assert [e.n for e in args[0]] == [15, 7] and [e.param_dtype for e in args[0]] == [1, 0]
    assert args[0][0].master == opt.master_weights[0].data_ptr()
    assert opt.state["exp_avg_scale"][0].shape == (1,) and opt.state["exp_avg"][0].dtype == torch.float8_e4m3fn


@pytest.mark.parametrize("call, err", [
    (lambda: df2.embedding(i32(V, D), i32(N)), TypeError),                      # table of integers
    (lambda: df2.embedding(bf(V, D), f32(N)), TypeError),                       # ids of floats
    (lambda: df2.embedding(bf(V, D).t(), i32(N)), ValueError),                  # rows not dense
    (lambda: df2.embedding(bf(V, D), i32(N), out=bf(N, D + 1)), ValueError),
    (lambda: df2.embedding(bf(V, D), i32(N), out=bf(N - 1, D)), ValueError),
    (lambda: df2.embedding(bf(V, D), i32(N), out=bf(N, D), dtype=F32), TypeError),
    (lambda: df2.embedding(bf(V, D), i32(N), dtype=torch.float16), TypeError),
    (lambda: df2.embedding(bf(V, D), i32(N), dev_status=f32(1)), TypeError),
    (lambda: df2.embedding(bf(V, D), torch.zeros(N, dtype=I32, device="meta")), ValueError),
    (lambda: df2.embedding_grad(bf(N + 1, D), i32(N), V), ValueError),           # a row too many
    (lambda: df2.embedding_grad(bf(D, N).t(), i32(N), V), ValueError),
    (lambda: df2.embedding_grad(bf(N, D), i32(N), V, out=f32(V + 1, D)), ValueError),
    (lambda: df2.embedding_grad(bf(N, D), i32(N), V, accumulate=True), ValueError),  # added to nothing
    (lambda: df2.embedding_grad(bf(N, D), i32(N), V, dtype=torch.float64), TypeError),
    (lambda: df2.embedding_grad(bf(N, D), i32(N), V, workspace=torch.zeros(255, dtype=torch.uint8)), ValueError),
    (lambda: df2.selector_loss_grad(**{**sel(), "targets": i32(P - 1)}), ValueError),
    (lambda: df2.selector_loss_grad(**{**sel(), "topk_vals": f32(P, K + 1)}), ValueError),
    (lambda: df2.selector_loss_grad(**{**sel(), "Bc": bf(V, r + 8)}), ValueError),
    (lambda: df2.selector_loss_grad(**{**sel(), "G": bf(P, r)}), TypeError),
    (lambda: df2.selector_loss_grad(**sel(), row_weights=f32(P + 1)), ValueError),
    (lambda: df2.selector_loss_grad(**sel(), accumulate=True), ValueError),
    (lambda: df2.selector_loss_grad(**sel(), dA=f32(V, r), dBc=bf(V, r)), TypeError),   # two types
    (lambda: df2.selector_loss_grad(**sel(), dA=f32(V, r + 1)), ValueError),
    (lambda: df2.selector_loss_grad(**sel(), dtype=torch.float16), TypeError),
    (lambda: df2.selector_loss_grad(**sel(), out=(f32(P), i32(P), f32(P, K), f32(P - 1, r))), ValueError),
    (lambda: df2.AdamW([f32(4)], state_bits=16), ValueError),
    (lambda: df2.AdamW([i32(4)]), TypeError),
    (lambda: df2.AdamW([f32(4, 4).t()[:, :2]]), ValueError),
    (lambda: df2.AdamW([f32(4)], lr=[1.0, 2.0]), ValueError),
    (lambda: df2.AdamW([f32(4)], master_weights=[f32(5)]), ValueError),
    (lambda: df2.AdamW([f32(4)], master_weights=[bf(4)]), TypeError),
    (lambda: df2.AdamW([f32(4)], state={"exp_avg": [f32(4)], "exp_avg_sq": [f32(3)]}), ValueError),
    (lambda: df2.AdamW([f32(4)], [f32(5)]).step(), ValueError),
    (lambda: df2.AdamW([f32(4)], [f32(4), f32(4)]).step(), ValueError),
    (lambda: df2.AdamW([f32(4)], [torch.zeros(4, dtype=torch.float16)]).step(), TypeError),
    (lambda: df2.AdamW([f32(4)], [f32(4)]).step(grad_scale=f32(2)), ValueError),
    (lambda: df2.AdamW([f32(4)], [f32(4)]).step(lr=[1.0, 2.0]), ValueError),
])
def test_refusals_come_before_the_library(fake, call, err):
    with pytest.raises(err):
        call()
    assert not fake.calls


def test_adamw_sees_tensors_that_change(fake):
    p, g = [f32(8), f32(8)], [f32(8), f32(8)]
    opt = df2.AdamW(p, g)
    opt.step()
    table = fake.calls[-1][1][0]
    opt.step()
    assert fake.calls[-1][1][0] is table and opt.step_count == 2     # the same descriptors
    other = [bf(8), None]
    opt.step(other)
    table = fake.calls[-1][1][0]
    assert table[0].grad == other[0].data_ptr() and table[0].grad_dtype == 0 and table[1].n == 0
    opt.step(lr=0.5)
    assert [e.lr for e in fake.calls[-1][1][0]] == [0.5, 0.5]
    with pytest.raises(ValueError):
        opt.step([f32(8), f32(9)])
    assert opt.step_count == 4
    opt.step()                                                        # after a refused step: bound anew
    assert fake.calls[-1][1][0][1].grad == g[1].data_ptr()


def test_host_tensors_are_refused():
    with pytest.raises(TypeError):
        df2.embedding(bf(V, D), i32(N))
    with pytest.raises(TypeError):
        df2.embedding_grad(bf(N, D), i32(N), V)
    with pytest.raises(TypeError):
        df2.selector_loss_grad(**sel())
    with pytest.raises(TypeError):
        df2.AdamW([f32(4)])


def test_the_descriptor_is_the_header_s():
    """ctypes lays dflash2_adamw_tensor out as the header declares it."""
    S = _abi.AdamWTensor
    assert [n for n, _ in S._fields_] == ["param", "master", "grad", "exp_avg", "exp_avg_2", "exp_avg_scale",
                                          "exp_avg_2_scale", "n", "param_dtype", "grad_dtype", "lr", "weight_decay"]
    assert ct.sizeof(S) == 7 * 8 + 8 + 4 + 4 + 8 + 8
    assert optim.ADAMW_BLOCK == 256


# ------------------------------------------------------------ the library --

@pytest.fixture(scope="module")
def lib():
    build.build()
    return _abi.load()


FAKE, FAKE2, ODD = VP(0x1000), VP(0x2000), VP(0x1001)


def test_embedding_validation(lib):
    f = lib.dflash2_embedding
    args = dict(t=FAKE, tdt=0, V=10, D=8, ld=8, ids=FAKE, N=4, s=1.0, out=FAKE2, odt=1, old=8)
    call = lambda **k: f(*{**args, **k}.values(), None, None)
    assert call(V=0) == 1 and call(D=0) == 1 and call(N=-1) == 1 and call(tdt=2) == 1 and call(odt=-1) == 1
    assert call(ld=7) == 1 and call(old=7) == 1 and call(s=math.inf) == 1 and call(s=math.nan) == 1
    assert call(t=None) == 1 and call(ids=None) == 1 and call(out=None) == 1
    assert call(V=(1 << 30) + 1) == 2 and call(N=1 << 31) == 2 and call(D=(1 << 24) + 1, ld=1 << 25, old=1 << 25) == 2
    assert call(N=1 << 20, D=(1 << 20) + 1, ld=1 << 21, old=1 << 21) == 2        # N * D over 2^40
    assert call(t=ODD) == 2 and call(out=VP(0x2002)) == 2 and call(ids=VP(0x1002)) == 2
    assert call(N=0, t=None, ids=None, out=None) == 0


def test_embedding_grad_validation(lib):
    f, size = lib.dflash2_embedding_grad, lib.dflash2_embedding_grad_workspace_size
    args = dict(d=FAKE, ddt=0, dld=8, ids=FAKE, N=4, V=10, D=8, s=1.0, acc=0, t=FAKE2, tdt=1, tld=8, ws=FAKE, wb=1 << 30)
    call = lambda **k: f(*{**args, **k}.values(), None, None)
    assert call(V=0) == 1 and call(D=0) == 1 and call(N=-1) == 1 and call(ddt=3) == 1 and call(tdt=7) == 1
    assert call(dld=7) == 1 and call(tld=7) == 1 and call(s=math.nan) == 1 and call(d=None) == 1 and call(t=None) == 1
    assert call(N=1 << 31) == 2 and call(ws=VP(0x1008)) == 2 and call(d=ODD) == 2
    assert call(wb=16) == 4 and call(ws=None) == 4
    assert call(N=0, acc=1, d=None, ids=None, t=None, ws=None, wb=0) == 0         # nothing to add
    assert size(0, 10, 8) == 0 and size(-1, 10, 8) == 0 and size(100, 10, 8) > 0
    for N in (1, 511, 513, 100_000, 1 << 20):
        for D_ in (1, 8, 100, 5120):
            # two copies of the (id, position) pairs at least, in pieces of 256 bytes
            assert size(N, 1000, D_) >= 16 * N and size(N, 1000, D_) % 256 == 0


def test_selector_loss_grad_validation(lib):
    f, size = lib.dflash2_selector_loss_grad, lib.dflash2_selector_loss_grad_workspace_size
    args = dict(pred=FAKE, tg=FAKE, P=4, ids=FAKE, vals=FAKE, G=FAKE, A=FAKE, B=FAKE, V=100, K=4, r=16, w=None, acc=0,
                loss=FAKE, lab=FAKE, ds=FAKE, dG=FAKE, dA=FAKE, dB=FAKE2, dt=1, ws=FAKE, wb=1 << 30)
    call = lambda **k: f(*{**args, **k}.values(), None, None)
    assert call(P=-1) == 1 and call(V=0) == 1 and call(K=0) == 1 and call(K=101) == 1 and call(r=0) == 1 and call(dt=5) == 1
    assert call(dA=FAKE2) == 1                                                  # one table for two
    assert call(r=12) == 2 and call(r=4104) == 2 and call(K=1025, V=5000) == 2 and call(V=(1 << 30) + 1) == 2
    assert call(P=1 << 29, K=4) == 2                                            # P * K over 2^31
    assert call(G=VP(0x1004)) == 2 and call(dB=VP(0x2008)) == 2 and call(vals=VP(0x1002)) == 2
    for name in ("pred", "tg", "ids", "vals", "G", "A", "B", "loss", "lab", "ds", "dG"):
        assert call(**{name: None}) == 1, name
    assert call(wb=64) == 4 and call(ws=None) == 4
    assert call(P=0, dA=None, dB=None, ws=None, wb=0) == 0
    assert size(0, 100, 4, 16) == 0 and size(5, 100, 101, 16) == 0 and size(5, 100, 4, 16) > 2 * 5 * 16 * 4


def test_adamw_validation(lib):
    f = lib.dflash2_adamw

    def call(bits=32, b1=0.9, b2=0.99, eps=1e-8, step=1, count=1, scale=None, **k):
        e = dict(param=0x1000, master=None, grad=0x2000, exp_avg=0x3000, exp_avg_2=0x4000, exp_avg_scale=0x5000,
                 exp_avg_2_scale=0x6000, n=0, param_dtype=1, grad_dtype=1, lr=1e-3, weight_decay=0.0)
        e.update(k)
        t = (_abi.AdamWTensor * 1)(_abi.AdamWTensor(**e))
        return f(t, count, bits, b1, b2, eps, step, scale, None)

    assert call() == 0 and call(count=0) == 0                                   # nothing to do
    assert call(bits=16) == 1 and call(b1=1.0) == 1 and call(b2=-0.1) == 1 and call(eps=-1.0) == 1 and call(step=0) == 1
    assert call(b1=math.nan) == 1 and call(eps=math.inf) == 1 and call(count=-1) == 1
    assert call(n=-1) == 1 and call(lr=math.nan) == 1 and call(weight_decay=-1.0) == 1 and call(param_dtype=2) == 1
    for name in ("param", "grad", "exp_avg", "exp_avg_2"):
        assert call(n=5, **{name: None}) == 1, name
    assert call(n=5, bits=8, exp_avg_scale=None) == 1
    assert call(n=5, param=0x1002) == 2 and call(n=5, exp_avg=0x3001) == 2 and call(n=5, master=0x7002) == 2
    assert call(scale=VP(0x1002)) == 2
    assert f(None, 1, 32, 0.9, 0.99, 1e-8, 1, None, None) == 1
