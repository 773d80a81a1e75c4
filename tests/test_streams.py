"""Calls on another stream than the current one, on the CPU against stand-ins
for the library and the streams: where the memory comes from that a call makes.

An allocator hands out again what was freed on a stream as soon as that stream's work is
queued.  Memory of the current stream may then still be written by it when a call's kernels
on another stream begin, so a call takes its memory from the stream it runs on."""
import contextlib
import ctypes as ct

import pytest

torch = pytest.importorskip("torch")

import dflash2_draft_block_gb300 as df2  # noqa: E402

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
P, K, r, V, D, N = 12, 4, 16, 50, 24, 10


class FakeLib:
    def __getattr__(self, name):
        if name.endswith("_workspace_size"):
            return lambda *a: 4096
        return lambda *a: 0


@pytest.fixture
def made(monkeypatch):
    """Every torch.empty (its address, and the stream it was made under) and record_stream."""
    current, log = ["current"], {"made": {}, "kept": {}}
    empty, hold = torch.empty, []

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    def traced(*a, **k):
        t = empty(*a, **k)
        hold.append(t)
        log["made"][t.data_ptr()] = current[-1]
        return t

    lib = FakeLib()
    monkeypatch.setattr(df2, "lib", lambda: lib)
    monkeypatch.setattr(df2, "_on_device", lambda t: True)
    monkeypatch.setattr(df2, "_stream", lambda stream, device: ct.c_void_p(0))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[-1])
    monkeypatch.setattr(torch, "empty", traced)
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: log["kept"].setdefault(t.data_ptr(), []).append(s), raising=False)
    return log


def z(*s, dtype=F32):
    return torch.zeros(s, dtype=dtype)


R, B, C, TAPS, GROUP = 3, 4, 32, 2, 4
H, W_LM, W_H = z(P, D, dtype=BF), z(V, D, dtype=BF), z(r, D, dtype=BF)
IDS, VALS, G, A, BC = z(P, K, dtype=I32), z(P, K), z(P, r), z(V, r, dtype=BF), z(V, r, dtype=BF)
X, W_PROJ, BASE = z(P, C, dtype=BF), z(2 * TAPS * C // GROUP, C, dtype=BF), z(2, TAPS, C)
DYN = z(P, TAPS, C // GROUP)

CALLS = {
    "unary_topk": lambda **k: df2.unary_topk(H, W_LM, K, W_H, **k),
    "unary_topk_noalloc": lambda **k: df2.unary_topk_noalloc(H, W_LM, K, W_H, **k),
    "selector_walk": lambda **k: df2.selector_walk(z(R, dtype=I32), IDS, VALS, G, A, BC, B, **k),
    "selector_ce": lambda **k: df2.selector_ce(VALS, IDS, z(P, dtype=I32), V, **k),
    "selector_pair_scores": lambda **k: [df2.selector_pair_scores(z(P, dtype=I32), IDS, VALS, G, A, BC, **k)],
    "draft_head": lambda **k: df2.draft_head(H, W_LM, K, W_H, A, BC, z(R, dtype=I32), B, z(P, dtype=I32), **k),
    "selector_lattice": lambda **k: [df2.selector_lattice(z(R, dtype=I32), IDS, VALS, G, A, BC, B, **k)],
    "lattice_walk": lambda **k: df2.lattice_walk(z(R, B - 1, K, K), IDS, B, V, **k),
    "conv_prepare": lambda **k: df2.conv_prepare(X, B, TAPS, GROUP, W_PROJ, BASE, **k),
    "conv_finish": lambda **k: [df2.conv_finish(X, B, TAPS, GROUP, DYN, BASE, **k)],
    "conv_finish_prepare": lambda **k: df2.conv_finish_prepare(X, B, TAPS, GROUP, DYN, BASE, W_PROJ, BASE, **k),
    "embedding": lambda **k: [df2.embedding(z(V, D, dtype=BF), z(N, dtype=I32), **k)],
    "embedding_grad": lambda **k: [df2.embedding_grad(z(N, D), z(N, dtype=I32), V, **k)],
    "selector_loss_grad": lambda **k: df2.selector_loss_grad(z(P, dtype=I32), z(P, dtype=I32), IDS, VALS, G, A, BC, **k),
}
SCRATCH = {"unary_topk", "draft_head", "conv_prepare", "conv_finish_prepare", "embedding_grad", "selector_loss_grad"}


@pytest.mark.parametrize("name", CALLS)
def test_memory_comes_from_the_call_s_stream(made, name):
    outs = CALLS[name](stream="side")
    scratch = 1 if name in SCRATCH else 0
    assert len(made["made"]) == len(outs) + scratch and set(made["made"].values()) == {"side"}
    for t in outs:
        # the caller goes on with the outputs on the current stream, which keeps them as well
        assert made["made"][t.data_ptr()] == "side" and made["kept"][t.data_ptr()] == ["current"]


@pytest.mark.parametrize("name", CALLS)
def test_no_stream_is_named_for_the_current_one(made, name):
    CALLS[name]()
    assert set(made["made"].values()) == {"current"} and not made["kept"]
