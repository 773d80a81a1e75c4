"""What the AdamW handle gives the library, on the CPU against a stand-in for it: the tensors
and rates as they are at the step, every step checked, each parameter at its own step."""
import copy
import ctypes as ct
import gc
import weakref

import pytest

torch = pytest.importorskip("torch")

import dflash2_draft_block_gb300 as df2  # noqa: E402
from dflash2_draft_block_gb300 import _abi  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


class FakeLib:
    """Records the descriptors (copied) and the step of every dflash2_adamw call."""

    def __init__(self):
        self.calls, self.refuse = [], 0

    def dflash2_status_string(self, code):
        return b"refused"

    def dflash2_adamw(self, table, count, bits, beta1, beta2, eps, step, scale, stream):
        held = (_abi.AdamWTensor * count)()
        ct.memmove(held, table, ct.sizeof(held))
        if not self.refuse:
            self.calls.append((held, step))
        return self.refuse


@pytest.fixture
def fake(monkeypatch):
    lib = FakeLib()
    monkeypatch.setattr(df2, "lib", lambda: lib)
    monkeypatch.setattr(df2, "_on_device", lambda t: True)
    monkeypatch.setattr(df2, "_stream", lambda stream, device: ct.c_void_p(0))
    return lib


def zeros(n, dtype=F32):
    return torch.zeros(n, dtype=dtype)


def handle(bits, master=True, n=3):
    params = [zeros(300 + i, BF) for i in range(n)]
    grads = [zeros(300 + i) for i in range(n)]
    return df2.AdamW(params, grads, state_bits=bits, master_weights=master)


def agree(opt, table):
    """The descriptors hold the tensors' present addresses."""
    fields = {"exp_avg": "exp_avg", "exp_avg_sq": "exp_avg_2", "exp_avg_rms": "exp_avg_2",
              "exp_avg_scale": "exp_avg_scale", "exp_avg_rms_scale": "exp_avg_2_scale"}
    for i, e in enumerate(table):
        assert e.param == opt.params[i].data_ptr() and e.grad == opt.grads[i].data_ptr()
        assert e.n == opt.params[i].numel()
        assert (e.master or 0) == (opt.master_weights[i].data_ptr() if opt.master_weights else 0)
        for name, ts in opt.state.items():
            assert getattr(e, fields[name]) == ts[i].data_ptr(), name


@pytest.mark.parametrize("bits", [32, 8])
def test_moved_tensors_are_seen(fake, bits):
    opt = handle(bits)
    opt.step()
    opt.step()
    lists = [opt.params, opt.grads, opt.master_weights, *opt.state.values()]
    for ts in lists:
        for t in ts:
            t.data = t.data.clone()
        opt.step()
        agree(opt, fake.calls[-1][0])
    for ts in lists:
        ts[1] = ts[1].clone()
        opt.step()
        agree(opt, fake.calls[-1][0])
    opt.state = {k: [t.clone() for t in ts] for k, ts in opt.state.items()}
    opt.step()
    agree(opt, fake.calls[-1][0])
    opt.state["exp_avg"] = [t.clone() for t in opt.state["exp_avg"]]
    opt.master_weights = [t.clone() for t in opt.master_weights]
    opt.step()
    agree(opt, fake.calls[-1][0])
    opt.master_weights = None
    opt.step()
    agree(opt, fake.calls[-1][0])


def test_another_type_at_the_same_address(fake):
    opt = handle(32)
    opt.step()
    opt.grads[1].data = opt.grads[1].data.view(BF)[:301]
    opt.step()
    agree(opt, fake.calls[-1][0])
    assert [e.grad_dtype for e in fake.calls[-1][0]] == [1, 0, 1]


@pytest.mark.parametrize("change, err", [
    (lambda o: o.state["exp_avg"].__setitem__(0, zeros(299)), ValueError),
    (lambda o: o.state["exp_avg_sq"].__setitem__(0, zeros(299)), ValueError),
    (lambda o: o.state["exp_avg_sq"].__setitem__(0, zeros(300, BF)), TypeError),
    (lambda o: o.state["exp_avg_sq"].pop(), ValueError),
    (lambda o: o.master_weights.__setitem__(2, zeros(302, BF)), TypeError),
    (lambda o: o.master_weights.__setitem__(2, zeros(604)[::2]), ValueError),
    (lambda o: setattr(o.master_weights[2], "data", zeros(301)), ValueError),
    (lambda o: setattr(o.state["exp_avg"][1], "data", zeros(7)), ValueError),
    (lambda o: setattr(o.params[1], "data", zeros(299, BF)), ValueError),
    (lambda o: setattr(o.params[1], "data", torch.zeros(301, dtype=torch.float16)), TypeError),
    (lambda o: setattr(o.state["exp_avg"][1], "data", o.state["exp_avg"][1].data[:7]), ValueError),   # where it was
    (lambda o: setattr(o.master_weights[0], "data", o.master_weights[0].data[:7]), ValueError),
    (lambda o: setattr(o.params[0], "data", o.params[0].data[:7]), ValueError),
    (lambda o: setattr(o.grads[0], "data", o.grads[0].data[:7]), ValueError),
    (lambda o: setattr(o.grads[0], "data", o.grads[0].data.view(torch.int32)), TypeError),
    (lambda o: o.grads.__setitem__(0, zeros(299)), ValueError),
    (lambda o: setattr(o.grads[0], "data", zeros(299)), ValueError),
    (lambda o: setattr(o.grads[0], "data", zeros(300, torch.float16)), TypeError),
    (lambda o: setattr(o.grads[0], "data", zeros(600)[::2]), ValueError),
    (lambda o: o.grads.pop(), ValueError),
    (lambda o: o.params.pop(), ValueError),
    (lambda o: o.params.__setitem__(0, "w"), TypeError),
    (lambda o: o.grads.__setitem__(0, 1.0), TypeError),
])
def test_what_no_longer_fits_is_refused(fake, change, err):
    """After two steps as well as before the first."""
    for steps in (0, 2):
        opt = handle(32)
        for _ in range(steps):
            opt.step()
        done = len(fake.calls)
        change(opt)
        with pytest.raises(err):
            opt.step()
        assert len(fake.calls) == done and opt.step_count == steps


def test_rates_set_on_the_handle_take_effect(fake):
    opt = handle(32)
    rates = lambda: [(e.lr, e.weight_decay) for e in fake.calls[-1][0]]
    opt.step()
    opt.lr = 0.5
    opt.step()
    assert rates() == [(0.5, 0.01)] * 3
    opt.lr = [0.1, 0.2, 0.3]
    opt.weight_decay = 0.25
    opt.step()
    assert rates() == [(0.1, 0.25), (0.2, 0.25), (0.3, 0.25)]
    opt.lr[1] = 7.0
    opt.weight_decay[2] = 0.0
    opt.step()
    assert rates() == [(0.1, 0.25), (7.0, 0.25), (0.3, 0.0)]
    opt.step(lr=1.0)
    assert rates() == [(1.0, 0.25), (1.0, 0.25), (1.0, 0.0)] and opt.lr == [1.0] * 3
    opt.lr = [1.0, 2.0]
    with pytest.raises(ValueError):
        opt.step()


def test_gradients_and_replaced_states_are_let_go(fake):
    """Between steps the handle keeps no gradient alive, nor a state that was replaced."""
    opt = df2.AdamW([zeros(10), zeros(20)])
    grads = [zeros(10), zeros(20)]
    refs = [weakref.ref(g) for g in grads]
    opt.step(grads)
    del grads
    gc.collect()
    assert all(r() is None for r in refs)
    opt.params[0].grad = zeros(10)
    ref = weakref.ref(opt.params[0].grad)
    opt.step()
    opt.params[0].grad = None
    gc.collect()
    assert ref() is None
    ref = weakref.ref(opt.state["exp_avg"][0])
    opt.state["exp_avg"][0] = zeros(10)
    gc.collect()
    assert ref() is None


def test_every_step_asks_for_the_current_device(fake, monkeypatch):
    """With another device made current between two steps, nothing is launched there."""
    opt = handle(32)
    opt.step()
    opt.step()
    done = len(fake.calls)

    def other(first, **others):
        raise ValueError(f"the tensors are on {first.device} but the current CUDA device is another")
    with monkeypatch.context() as m:
        m.setattr(df2, "_device", other)
        with pytest.raises(ValueError):
            opt.step()
    assert len(fake.calls) == done and opt.step_count == 2
    opt.step()
    assert len(fake.calls) == done + 1


def test_a_refused_step_does_not_count(fake, monkeypatch):
    """Under graph capture (where the library refuses) with the reason; otherwise by its status."""
    opt = handle(32)
    opt.step()
    fake.refuse = 2
    with pytest.raises(df2.DFlash2Error):
        opt.step()
    monkeypatch.setattr(df2, "_capturing", lambda stream, device: True)
    with pytest.raises(RuntimeError, match="captur"):
        opt.step()
    fake.refuse = 0
    assert len(fake.calls) == 1 and opt.step_count == 1
    opt.step()
    assert fake.calls[-1][1] == 2


def took(call):
    table, step = call
    return step, [i for i, e in enumerate(table) if e.n]


def test_a_parameter_counts_its_own_steps(fake):
    opt = df2.AdamW([zeros(5), zeros(6), zeros(7)])
    g = [zeros(5), zeros(6), zeros(7)]
    for have, want in (([1, 0, 1], [(1, [0, 2])]), ([1, 0, 1], [(2, [0, 2])]), ([1, 1, 0], [(3, [0]), (1, [1])]),
                       ([0, 1, 0], [(2, [1])]), ([0, 0, 0], []), ([1, 1, 1], [(4, [0]), (3, [1, 2])])):
        done = len(fake.calls)
        opt.step([x if on else None for x, on in zip(g, have)])
        got = fake.calls[done:]
        assert sorted(map(took, got)) == sorted(want)
        for table, _ in got:
            for e, x in zip(table, g):
                assert e.n in (0, x.numel()) and (e.n == 0 or e.grad == x.data_ptr())
    assert opt.step_count == 6
    saved = opt.state_dict()
    assert saved["step"] == [4, 3, 3]
    again = df2.AdamW(opt.params, **saved)
    again.step(g)
    assert sorted(map(took, fake.calls[-2:])) == [(4, [1, 2]), (5, [0])]
    assert df2.AdamW(opt.params, step=7).state_dict()["step"] == 7
    assert df2.AdamW(opt.params, step=[7, 7, 7]).state_dict()["step"] == 7
    for bad in ([1, 2], [1, 2, 3, 4]):
        with pytest.raises(ValueError):
            df2.AdamW(opt.params, step=bad)


def test_autograd_notices_a_step(fake):
    """A backward through weights that were saved before a step and stepped since is refused, as
    after any write in place; one through a parameter that was left out is not."""
    p, q = (torch.ones(4, requires_grad=True) for _ in range(2))
    opt = df2.AdamW([p, q], master_weights=True)
    for t, change in ((p, False), (q, True)):
        y = (t * t).sum()
        opt.step([None, zeros(4)])
        if change:
            with pytest.raises(RuntimeError, match="inplace"):
                y.backward()
        else:
            y.backward()
    with torch.inference_mode():
        w = torch.ones(4)
    df2.AdamW([w], [zeros(4)]).step()                 # (keeps no version)


def test_a_handle_before_its_first_step_can_be_copied(fake):
    opt = copy.deepcopy(handle(8))
    opt.step()
    agree(opt, fake.calls[-1][0])


def test_no_parameters(fake):
    opt = df2.AdamW([], [], step=3)
    opt.step()
    assert opt.state_dict()["step"] == 3
    assert not fake.calls
    with pytest.raises(ValueError):
        opt.step([zeros(1)])
