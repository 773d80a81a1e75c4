"""Dropout on the GPU against its definition in 64 bits: types, strides, odd sizes, in place,
residuals, NaN where nothing is kept, far element indices, graphs, and streams.

A kept element is x * s, rounded to fp32 (2^-24 of it), where s is 65536 / (65536 - T)
rounded (2^-24); the residual's sum is rounded once more and the result once to its type.
So |error| <= 2^-23 |x s| (1 + 2^-24) + 2^-24 |y| + half a step of y."""
import numpy as np
import pytest

from dropout_words import dropped

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
HALF_STEP = {BF: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.fixture(scope="module")
def df2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dflash2_draft_block_gb300 as m
    return m


def f64(t):
    return t.detach().double().cpu().numpy()


def check(got, x, rate, seed, draw, residual=None, first=0):
    y, keep = dropped(f64(x), rate, seed, draw, first)
    y[~keep] = 0.0
    room = 2.0 ** -22 * np.abs(y)
    if residual is not None:
        y = y + f64(residual)
    room = room + (2.0 ** -23 + HALF_STEP[got.dtype]) * np.abs(y) + 1e-44
    off = np.abs(f64(got) - y)
    assert (off <= room).all(), (off - room).max()


def randn(seed, *shape, dtype=BF):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def apart(x, pad, shift=0):
    """The same matrix, its rows `pad` elements apart and its start moved by `shift` elements."""
    rows, cols = x.shape
    wide = torch.full((rows * (cols + pad) + shift,), 3.0, dtype=x.dtype, device=x.device)
    view = wide[shift:].view(rows, cols + pad)[:, :cols]
    view.copy_(x)
    return view


@pytest.mark.parametrize("N, D", [(1, 1), (1, 7), (3, 8), (5, 1), (17, 251), (8, 4096), (1, 100003), (300, 264), (2049, 24)])
@pytest.mark.parametrize("xd", [BF, F32])
@pytest.mark.parametrize("od", [BF, F32])
@pytest.mark.parametrize("res", [False, True])
def test_against_the_definition(df2, N, D, xd, od, res):
    x = randn(N + D, N, D, dtype=xd)
    r = randn(D, N, D, dtype=od) if res else None
    seed, draw = 0x9E3779B97F4A7C15 + D, (N << 33) + 5
    check(df2.dropout(x, 0.3, seed, draw, residual=r, dtype=od), x, 0.3, seed, draw, r)


@pytest.mark.parametrize("pad, shift", [(0, 0), (8, 0), (1, 0), (5, 3), (16, 8), (0, 1)])
@pytest.mark.parametrize("D", [64, 37])
def test_strides_and_alignment_change_nothing(df2, pad, shift, D):
    x, r = randn(1, 41, D), randn(2, 41, D, dtype=F32)
    want = df2.dropout(x, 0.25, 11, 12, residual=r)
    wide = torch.full((41, D + pad), 9.0, device="cuda")
    got = df2.dropout(apart(x, pad, shift), 0.25, 11, 12, residual=apart(r, pad, shift), out=wide[:, :D])
    assert torch.equal(got, want)
    assert bool((wide[:, D:] == 9.0).all())


def test_rates_at_the_ends(df2):
    x = randn(3, 64, 96)
    assert torch.equal(df2.dropout(x, 0.0, 5), x)
    assert not df2.dropout(x, 1.0, 5).any()
    assert torch.equal(df2.dropout(x, 1.0, 5, residual=x), x)
    check(df2.dropout(x, 65535 / 65536, 5), x, 65535 / 65536, 5, 0)
    check(df2.dropout(x, 1 / 65536, 5), x, 1 / 65536, 5, 0)


def test_what_is_dropped_leaves_no_trace(df2):
    x = randn(4, 40, 72, dtype=F32)
    _, keep = dropped(f64(x), 0.5, 6, 7)
    gone = torch.from_numpy(~keep).cuda()
    y = df2.dropout(x, 0.5, 6, 7)
    for bad in (float("nan"), float("inf"), -float("inf")):
        assert torch.equal(df2.dropout(torch.where(gone, torch.full_like(x, bad), x), 0.5, 6, 7), y)
    kept = df2.dropout(torch.full_like(x, float("nan")), 0.5, 6, 7)
    assert torch.equal(kept.isnan(), ~gone)


def test_in_place(df2):
    for D in (64, 37):
        x, r = randn(5, 50, D), randn(6, 50, D)
        want, sum_ = df2.dropout(x, 0.4, 1), df2.dropout(x, 0.4, 1, residual=r)
        a, b, c = x.clone(), r.clone(), x.clone()
        assert df2.dropout(a, 0.4, 1, out=a) is a and torch.equal(a, want)
        df2.dropout(x, 0.4, 1, residual=b, out=b)
        assert torch.equal(b, sum_)
        df2.dropout(c, 0.4, 1, residual=r, out=c)
        assert torch.equal(c, sum_)
        flat = torch.zeros(50 * D + 8, dtype=BF, device="cuda")
        with pytest.raises(df2.DFlash2Error):
            df2.dropout(flat[:50 * D], 0.4, 1, out=flat[8:])


def test_shapes(df2):
    x = randn(7, 4, 6, 16)
    assert torch.equal(df2.dropout(x, 0.2, 3), df2.dropout(x.view(24, 16), 0.2, 3).view(4, 6, 16))
    assert torch.equal(df2.dropout(x.view(-1), 0.2, 3), df2.dropout(x, 0.2, 3).view(-1))
    assert df2.dropout(x[:0], 0.2, 3).shape == (0, 6, 16)


def test_gradient(df2):
    """The gradient is the formula's, and differences of the (linear) call's."""
    x, dout = randn(8, 30, 40, dtype=F32), randn(9, 30, 40, dtype=F32)
    dx = df2.dropout_grad(dout, 0.35, 21, 22)
    check(dx, dout, 0.35, 21, 22)
    acc = randn(10, 30, 40, dtype=F32)
    want = acc.clone()
    assert df2.dropout_grad(dout, 0.35, 21, 22, accumulate=True, out=acc) is acc
    check(acc, dout, 0.35, 21, 22, want)
    d = randn(11, 30, 40, dtype=F32)
    up, down = (df2.dropout(x + s * d, 0.35, 21, 22) for s in (1.0, -1.0))
    got = float((dout.double() * (up.double() - down.double())).sum() / 2)
    # each value is rounded at most four times (x + d, the scale, the product, twice) near size 10
    room = 1200 * 4 * 2.0 ** -24 * 10 * float(dout.abs().max())
    assert abs(got - float((dx.double() * d.double()).sum())) < room


def test_other_draws_and_seeds_give_other_masks(df2):
    x = torch.ones(64, 1024, device="cuda")
    masks = [df2.dropout(x, 0.5, s, d) > 0 for s, d in ((1, 0), (2, 0), (1, 1), (1 + (1 << 32), 0), (1, 1 << 32))]
    n = x.numel()
    for i, a in enumerate(masks):
        assert abs(float(a.float().mean()) - 0.5) < 5 * 0.5 / n ** 0.5
        for b in masks[:i]:
            assert abs(float((a == b).float().mean()) - 0.5) < 5 * 0.5 / n ** 0.5


def test_elements_past_32_bits(df2):
    """2^32 + 2^20 elements: the counters of the last ones, and their addresses."""
    n = (1 << 32) + (1 << 20) + 3
    x = torch.ones(n, dtype=BF, device="cuda")
    y = df2.dropout(x, 0.5, 77, 78)
    for first in (0, (1 << 31) - 5000, (1 << 32) - 5000, n - 10000):
        check(y[first:first + 10000], x[first:first + 10000], 0.5, 77, 78, first=first)


def test_draw_on_the_gpu_and_graphs(df2):
    x = randn(12, 128, 256)
    draw = torch.full((1,), 5, dtype=torch.int64, device="cuda")
    assert torch.equal(df2.dropout(x, 0.5, 9, draw), df2.dropout(x, 0.5, 9, 5))
    y, dx = torch.empty_like(x), torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        df2.dropout(x, 0.5, 9, draw, out=y)
        df2.dropout_grad(x, 0.5, 9, draw, out=dx)
        draw += 1
    for step in (5, 6, 7):
        graph.replay()
        want = df2.dropout(x, 0.5, 9, step)
        assert torch.equal(y, want) and torch.equal(dx, want)
    draw.fill_((1 << 40) + 1)
    graph.replay()
    assert torch.equal(y, df2.dropout(x, 0.5, 9, (1 << 40) + 1))


def test_capture_with_a_number_is_refused(df2):
    x, y = randn(13, 16, 16), torch.zeros(16, 16, dtype=BF, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y.fill_(1.0)
        with pytest.raises(RuntimeError, match="captured"):
            df2.dropout(x, 0.5, 9, 5, out=y)
    graph.replay()
    assert bool((y == 1.0).all())


def test_side_stream(df2):
    x = randn(14, 512, 512)
    want = df2.dropout(x, 0.1, 3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = df2.dropout(x, 0.1, 3, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
