"""dflash2_adamw against AdamW in 64 bits, and its 8-bit states' format.

Tolerances.  The kernel rounds each fp32 operation once.  A first moment is three
rounded operations on terms of its own size: within 4 * 2^-24 of |beta1 m| +
|(1 - beta1) g|.  A second moment (five, all terms positive) within 8 * 2^-24 of
itself.  The update m / den * lr has at most eight more: within 16 * 2^-24 of
lr * (|beta1 m| + |(1 - beta1) g|) / den, and the weight adds two roundings of its
own size.  A weight held in bf16 is the rounding of a value within these bounds."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
B1, B2, EPS, LR = 0.9, 0.999, 1e-8, 3e-3
BLOCK = 256


@pytest.fixture(scope="module")
def df2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dflash2_draft_block_gb300 as m
    m.lib()
    return m


def tensors(seed, sizes, pdt, gdt, first=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda n, s: torch.randn(n, generator=gen, device="cuda") * s
    ps = [r(n, 0.05).to(pdt) for n in sizes]
    gs = [(r(n, 1e-3) * (torch.rand(n, generator=gen, device="cuda") > 0.1)).to(gdt) for n in sizes]
    ms = [r(n, 0.0 if first else 3e-4) for n in sizes]
    vs = [r(n, 0.0 if first else 1e-3).square() for n in sizes]
    return ps, gs, ms, vs


def step64(w, g, m, v, t, wd, scale):
    w, m, v = w.double(), m.double(), v.double()
    g = g.double() * scale
    mn = B1 * m + (1 - B1) * g
    vn = B2 * v + (1 - B2) * g * g
    den = (vn / (1 - B2 ** t)).sqrt() + EPS
    size = (B1 * m).abs() + ((1 - B1) * g).abs()
    return w - LR * wd * w - LR * mn / (1 - B1 ** t) / den, mn, vn, size, LR * size / (1 - B1 ** t) / den


SIZES = [1, 7, 8, 255, 256, 257, 2048, 100003]


@pytest.mark.parametrize("pdt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gdt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("t", [1, 2, 5000])
def test_32bit_states(df2, pdt, gdt, master, t):
    ps, gs, ms, vs = tensors(t, SIZES, pdt, gdt, first=t == 1)
    wd = [0.1 * (i % 2) for i in range(len(SIZES))]
    masters = [p.float() + 1e-6 for p in ps] if master else None
    scale = torch.tensor([0.5], device="cuda")
    w0 = [w.clone() for w in (masters if master else ps)]
    m0, v0 = [m.clone() for m in ms], [v.clone() for v in vs]
    opt = df2.AdamW(ps, gs, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=wd, master_weights=masters,
                    state={"exp_avg": ms, "exp_avg_sq": vs}, step=t - 1)
    opt.step(grad_scale=scale)
    torch.cuda.synchronize()
    for i in range(len(SIZES)):
        w, m, v, size, upd = step64(w0[i], gs[i], m0[i], v0[i], t, wd[i], 0.5)
        assert torch.all((ms[i].double() - m).abs() <= 4 * U * size + 1e-45)
        assert torch.all((vs[i].double() - v).abs() <= 8 * U * v + 1e-44)
        tol = 16 * U * upd + 4 * U * (w.abs() + upd)
        if master:
            assert torch.all((masters[i].double() - w).abs() <= tol)
            assert torch.equal(ps[i], masters[i].to(pdt))
        else:
            # rounding is monotonic: between the roundings of the interval's ends
            assert torch.all(ps[i] >= (w - tol).to(pdt)) and torch.all(ps[i] <= (w + tol).to(pdt))


def quantise64(x, root):
    """x (fp32) to e4m3 values and scales by the header's rule, in 64 bits with one fp32
    rounding where the rule has one."""
    n = x.numel()
    pad = torch.zeros(-(-n // BLOCK) * BLOCK, dtype=torch.float32, device=x.device)
    pad[:n] = x
    b = pad.view(-1, BLOCK)
    top = b.abs().amax(1, keepdim=True)
    ok = top >= 2.0 ** -100
    q = b * torch.where(ok, 448.0 / top, torch.zeros_like(top))
    if root:
        q = torch.where((b > 0) & ok, q.clamp(min=2.0 ** -9), q)
    q = q.to(torch.float8_e4m3fn).view(-1)[:n]
    return q, torch.where(ok, top / 448.0, torch.zeros_like(top)).view(-1)


def value(q, scale):
    return q.float() * scale.repeat_interleave(BLOCK)[:q.numel()]


@pytest.mark.parametrize("pdt, gdt", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16)])
@pytest.mark.parametrize("t", [1, 40])
def test_8bit_states_hold_the_step_of_their_values(df2, pdt, gdt, t):
    """A step from 8-bit states is the 32-bit step from the values they stand for, bit for
    bit, and its states are that step's, rounded by the format's rule."""
    ps, gs, ms, vs = tensors(t, SIZES, pdt, gdt, first=t == 1)
    state = {"exp_avg": [], "exp_avg_scale": [], "exp_avg_rms": [], "exp_avg_rms_scale": []}
    for m, v in zip(ms, vs):
        for name, x, root in (("exp_avg", m, False), ("exp_avg_rms", v.sqrt(), True)):
            q, s = quantise64(x, root)
            state[name].append(q.clone())
            state[name + "_scale"].append(s.clone())
    m32 = [value(q, s) for q, s in zip(state["exp_avg"], state["exp_avg_scale"])]
    v32 = [value(q, s) * value(q, s) for q, s in zip(state["exp_avg_rms"], state["exp_avg_rms_scale"])]
    p32 = [p.clone() for p in ps]
    kw = dict(lr=LR, betas=(B1, B2), eps=EPS, weight_decay=0.02, step=t - 1)
    df2.AdamW(ps, gs, state_bits=8, state=state, **kw).step()
    df2.AdamW(p32, gs, state={"exp_avg": m32, "exp_avg_sq": v32}, **kw).step()
    torch.cuda.synchronize()
    for i in range(len(SIZES)):
        assert torch.equal(ps[i], p32[i])
        for name, x, root in (("exp_avg", m32[i], False), ("exp_avg_rms", v32[i].sqrt(), True)):
            q, s = quantise64(x, root)
            assert torch.equal(state[name + "_scale"][i], s), name
            assert torch.equal(state[name][i].view(torch.uint8), q.view(torch.uint8)), name


def test_8bit_root_never_rounds_to_zero(df2):
    """One gradient 1e8 times the others' in a block: the small ones' root keeps the
    smallest value above zero, so their next step, without gradients, stays bounded."""
    n = BLOCK
    p = torch.zeros(n, device="cuda")
    g = torch.full((n,), 1e-6, device="cuda")
    g[5] = 100.0
    opt = df2.AdamW([p], [g], lr=LR, weight_decay=0.0, state_bits=8)
    opt.step()
    assert torch.all(opt.state["exp_avg_rms"][0].float() >= 2.0 ** -9)
    opt.step([torch.zeros_like(g)])
    torch.cuda.synchronize()
    assert torch.all(p.abs() <= 2.5 * LR)


def test_views_at_odd_offsets_and_strayless_writes(df2):
    """Tensors that start off every vector boundary, inside larger buffers: the same result
    as aligned copies, and nothing written beside them."""
    sizes = [1000, 300, 5]
    for bits in (32, 8):
        ps, gs, _, _ = tensors(9, sizes, torch.bfloat16, torch.float32)
        bufs = [torch.full((n + 16,), 7.0, dtype=torch.bfloat16, device="cuda") for n in sizes]
        views = [b[3:3 + n] for b, n in zip(bufs, sizes)]
        gb = [torch.zeros(n + 1, device="cuda")[1:] for n in sizes]
        for v, p, a, g in zip(views, ps, gb, gs):
            v.copy_(p)
            a.copy_(g)
        for params, grads in ((ps, gs), (views, gb)):
            opt = df2.AdamW(params, grads, lr=LR, state_bits=bits, master_weights=True)
            for _ in range(3):
                opt.step()
        torch.cuda.synchronize()
        for b, v, p, n in zip(bufs, views, ps, sizes):
            assert torch.equal(v, p)
            assert torch.all(b[:3] == 7) and torch.all(b[3 + n:] == 7)


def test_more_tensors_than_one_launch_holds(df2):
    """700 tensors: three launches, every tensor stepped once, empty ones skipped."""
    sizes = [(i * 37) % 300 for i in range(700)]
    ps, gs, _, _ = tensors(4, sizes, torch.float32, torch.float32)
    flat, fgrad = torch.cat(ps), torch.cat(gs)
    opt = df2.AdamW(ps, gs, lr=LR)
    one = df2.AdamW([flat], [fgrad], lr=LR)
    k0 = df2.kernels_launched()
    opt.step()
    assert df2.kernels_launched() - k0 == 3
    one.step()
    torch.cuda.synchronize()
    assert torch.equal(torch.cat(ps), flat)


@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_unusable_grad_scale_leaves_everything(df2, bad):
    ps, gs, _, _ = tensors(2, [1000], torch.float32, torch.float32)
    before = ps[0].clone()
    opt = df2.AdamW(ps, gs, state_bits=8)
    opt.step(grad_scale=torch.tensor([bad], device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(ps[0], before)
    assert all(torch.all(t.view(torch.uint8) == 0) for ts in opt.state.values() for t in ts)


def test_gradients_that_move_and_go_missing(df2):
    """.grad tensors: a new address or type a step is seen, None leaves its parameter out."""
    p = [torch.ones(500, device="cuda", requires_grad=True) for _ in range(2)]
    opt = df2.AdamW(p, lr=LR, weight_decay=0.0)
    p[0].grad = torch.ones(500, device="cuda")
    opt.step()
    assert torch.all(p[1] == 1) and torch.all(p[0] < 1)
    p[0].grad = torch.zeros(500, device="cuda", dtype=torch.float32)
    p[1].grad = -torch.ones(500, device="cuda")
    opt.step()
    torch.cuda.synchronize()
    assert torch.all(p[1] > 1)
    assert opt.step_count == 2


def test_another_stream(df2):
    ps, gs, _, _ = tensors(3, [50000], torch.float32, torch.float32)
    want = [p.clone() for p in ps]
    df2.AdamW(want, gs, lr=LR).step()
    opt = df2.AdamW(ps, gs, lr=LR)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    opt.step(stream=st)
    torch.cuda.current_stream().wait_stream(st)
    torch.cuda.synchronize()
    assert torch.equal(ps[0], want[0])


def test_loss_goes_down_with_either_state(df2):
    """A least-squares fit with gradients 1e4 apart in size: both states reach a tenth of the
    loss they began with."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    size = torch.logspace(-2, 2, 64, device="cuda")
    x = torch.randn(512, 64, generator=gen, device="cuda") * size
    y = x @ torch.randn(64, 8, generator=gen, device="cuda")
    for bits in (32, 8):
        w = torch.zeros(64, 8, device="cuda")
        g = torch.empty_like(w)
        opt = df2.AdamW([w], [g], lr=2e-2, weight_decay=0.0, state_bits=bits)
        first = None
        for _ in range(300):
            e = x @ w - y
            first = first or float(e.square().mean())
            g.copy_(x.t() @ e / 512)
            opt.step()
        assert float((x @ w - y).square().mean()) < 0.1 * first, bits
