"""dflash2_embedding and dflash2_embedding_grad against torch in 64 bits.

Tolerances.  A lookup is one fp32 product (exact against torch's own) and one rounding.
A gradient sums c rows in fp32, in any order, then scales: within (c + 1) * 2^-24 of the
sum of the terms' sizes; a result held in bf16 lies between the bf16 roundings of the
ends of that interval."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def df2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dflash2_draft_block_gb300 as m
    m.lib()
    return m


def ids_of(kind, N, V, gen):
    u = torch.rand(N, generator=gen, device="cuda")
    uniform = (u * V).long().clamp(max=V - 1)
    if kind == "uniform":
        ids = uniform
    elif kind == "one":          # a single token everywhere
        ids = torch.full((N,), V // 2, device="cuda")
    elif kind == "mask":         # seven of eight are one token
        ids = torch.where(torch.rand(N, generator=gen, device="cuda") < 0.875, torch.full_like(uniform, V - 1), uniform)
    elif kind == "none":         # nothing but padding
        ids = torch.full((N,), -1, device="cuda")
    elif kind == "runs":         # lengths around the chunks' halves and wholes
        lengths = torch.tensor([1, 7, 8, 9, 15, 16, 17, 23, 24, 25, 31, 32, 33, 40, 100, 3], device="cuda").repeat(N // 300 + 1)
        ids = torch.repeat_interleave(torch.arange(len(lengths), device="cuda") % V, lengths)[:N]
        ids = ids[torch.randperm(len(ids), generator=gen, device="cuda")]
    elif kind == "padded":
        ids = torch.where(torch.rand(N, generator=gen, device="cuda") < 0.4, torch.full_like(uniform, -5), uniform)
    return ids.to(torch.int32)


@pytest.mark.parametrize("N, V, D", [(1, 1, 1), (1, 10, 8), (8, 5000, 4096), (7, 33, 31), (513, 100, 250),
                                     (3000, 257, 264), (20000, 4096, 256)])
@pytest.mark.parametrize("tdt", [BF, F32])
@pytest.mark.parametrize("odt", [BF, F32])
def test_lookup(df2, N, V, D, tdt, odt):
    gen = torch.Generator(device="cuda").manual_seed(N + D)
    table = torch.randn(V, D, generator=gen, device="cuda").to(tdt)
    ids = ids_of("padded", N, V, gen)
    got = df2.embedding(table, ids, scale=1.7, dtype=odt)
    want = table.float()[ids.clamp(min=0)] * 1.7
    want = torch.where((ids >= 0)[:, None], want, torch.zeros_like(want)).to(odt)
    assert torch.equal(got, want)


def test_lookup_strides_shapes_and_bad_ids(df2):
    gen = torch.Generator(device="cuda").manual_seed(3)
    wide = torch.randn(100, 96, generator=gen, device="cuda")
    for a, b in ((0, 64), (3, 40), (8, 72)):
        table = wide[:, a:b]
        ids = torch.randint(0, 100, (4, 6), generator=gen, device="cuda", dtype=torch.int32)
        assert torch.equal(df2.embedding(table, ids), table[ids])
        big = torch.full((24, 200), 9.0, device="cuda")
        df2.embedding(table, ids, out=big[:, 5:5 + b - a])
        assert torch.equal(big[:, 5:5 + b - a], table[ids.view(-1)])
        assert torch.all(big[:, :5] == 9) and torch.all(big[:, 5 + b - a:] == 9)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids = torch.tensor([0, 100, -1, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    got = df2.embedding(wide, ids, dev_status=st)
    assert int(st) == df2.DF2_STATUS_ID_OUT_OF_RANGE
    assert torch.equal(got[0], wide[0]) and torch.all(got[1].isnan()) and torch.all(got[2] == 0) and torch.all(got[3].isnan())
    assert df2.embedding(wide, ids[:0]).shape == (0, 96)


def grad64(dout, ids, V, scale):
    live = ids >= 0
    d = torch.where(live[:, None], dout.double(), torch.zeros_like(dout, dtype=torch.float64)) * scale
    z = lambda: torch.zeros(V, dout.shape[1], dtype=torch.float64, device="cuda")
    at = ids.clamp(min=0).long()
    count = torch.zeros(V, dtype=torch.float64, device="cuda").index_add_(0, at, live.double())
    return z().index_add_(0, at, d), z().index_add_(0, at, d.abs()), count


def check_grad(got, dout, ids, V, scale, before=None):
    want, size, count = grad64(dout, ids, V, scale)
    if before is not None:
        want, size, count = want + before.double(), size + before.double().abs(), count + 1
    tol = (count[:, None] + 1) * U * size
    if got.dtype == F32:
        assert torch.all((got.double() - want).abs() <= tol)
    else:
        assert torch.all(got >= (want - tol).to(BF)) and torch.all(got <= (want + tol).to(BF))


@pytest.mark.parametrize("kind", ["uniform", "one", "mask", "none", "runs", "padded"])
@pytest.mark.parametrize("N, V, D", [(1, 1, 8), (16, 4096, 256), (31, 7, 5), (100, 60, 264), (1023, 40, 100),
                                     (1025, 513, 256), (5003, 1000, 251), (17000, 300, 520), (40000, 70000, 16)])
@pytest.mark.parametrize("gdt, odt", [(BF, F32), (F32, BF), (BF, BF), (F32, F32)])
def test_gradient(df2, kind, N, V, D, gdt, odt):
    gen = torch.Generator(device="cuda").manual_seed(N + V)
    ids = ids_of(kind, N, V, gen)
    dout = torch.randn(N, D, generator=gen, device="cuda").to(gdt)
    dout[ids < 0] = float("nan")      # what padding holds is not read
    out = torch.full((V, D), float("nan"), dtype=odt, device="cuda")
    got = df2.embedding_grad(dout, ids, V, scale=0.6, out=out)
    clean = torch.where((ids >= 0)[:, None], dout, torch.zeros_like(dout))
    check_grad(got, clean, ids, V, 0.6)
    # twice: the same bits
    assert torch.equal(df2.embedding_grad(dout, ids, V, scale=0.6, dtype=odt), got)
    # added to what is there; untouched rows are left alone, bit for bit
    before = torch.randn(V, D, generator=gen, device="cuda").to(odt)
    acc = before.clone()
    df2.embedding_grad(dout, ids, V, scale=0.6, accumulate=True, out=acc)
    check_grad(acc, clean, ids, V, 0.6, before)
    absent = torch.ones(V, dtype=torch.bool, device="cuda")
    absent[ids[ids >= 0].long()] = False
    assert torch.equal(acc[absent], before[absent])


@pytest.mark.parametrize("V", [1, 2, 511, 512, 513, 262143, 262144, (1 << 27) + 5, 1 << 30])
def test_gradient_finds_every_id_of_a_vocabulary(df2, V):
    """One row an id, at the ends of the digits of the sort: added where it belongs.  (The
    table is a single column, so that 2^30 rows fit.)"""
    gen = torch.Generator(device="cuda").manual_seed(V & 0xffff)
    picks = sorted({0, V - 1, V // 2, V // 3, min(V - 1, 511), min(V - 1, 512), min(V - 1, 262144)})
    ids = torch.tensor(picks * 3, dtype=torch.int32, device="cuda")
    dout = torch.arange(1, len(ids) + 1, device="cuda", dtype=F32)[:, None].contiguous()
    out = torch.zeros(V, 1, device="cuda")
    df2.embedding_grad(dout, ids, V, accumulate=True, out=out)
    n = len(picks)
    for i, v in enumerate(picks):
        assert float(out[v]) == 3 * (i + 1) + 3 * n
    assert int((out != 0).sum()) == n


def test_gradient_strides_and_bad_ids(df2):
    gen = torch.Generator(device="cuda").manual_seed(8)
    wide = torch.randn(300, 90, generator=gen, device="cuda")
    ids = torch.randint(0, 50, (300,), generator=gen, device="cuda", dtype=torch.int32)
    for a, b in ((0, 64), (3, 40)):
        big = torch.full((50, 130), 4.0, device="cuda")
        df2.embedding_grad(wide[:, a:b], ids, 50, out=big[:, 6:6 + b - a])
        check_grad(big[:, 6:6 + b - a], wide[:, a:b], ids, 50, 1.0)
        assert torch.all(big[:, :6] == 4) and torch.all(big[:, 6 + b - a:] == 4)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = ids.clone()
    bad[::3] = 50
    got = df2.embedding_grad(wide, bad, 50, dev_status=st)
    assert int(st) == df2.DF2_STATUS_ID_OUT_OF_RANGE
    check_grad(got, torch.where((bad < 50)[:, None], wide, torch.zeros_like(wide)), bad.clamp(max=49), 50, 1.0)
    empty = df2.embedding_grad(wide[:0], ids[:0], 50)
    assert empty.shape == (50, 90) and torch.all(empty == 0)


def test_gradient_against_differences(df2):
    """d/dtable of sum(embedding(table) * c) is what embedding_grad(c) says: by central
    differences, in a table where the map is linear and fp32 differences of 2^-3 are exact
    up to the sum's rounding."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    V, D, N = 12, 9, 40
    table = torch.randn(V, D, generator=gen, device="cuda")
    ids = torch.randint(-1, V, (N,), generator=gen, device="cuda", dtype=torch.int32)
    c = torch.randn(N, D, generator=gen, device="cuda")
    got = df2.embedding_grad(c, ids, V, scale=2.5)
    h = 2.0 ** -3
    f = lambda t: float((df2.embedding(t, ids, scale=2.5).double() * c.double()).sum())
    for v in range(V):
        for d in (0, 4, 8):
            up, down = table.clone(), table.clone()
            up[v, d] += h
            down[v, d] -= h
            want = (f(up) - f(down)) / (2 * h)
            # a lookup's product and the table's sum with h each round within 2^-24 of |t| + h
            room = 4 * U * 2.5 * (abs(float(table[v, d])) + h) * N * 4 / h + 1e-6
            assert abs(float(got[v, d]) - want) <= room


def test_gradient_on_another_stream(df2):
    gen = torch.Generator(device="cuda").manual_seed(6)
    ids = ids_of("mask", 9000, 700, gen)
    dout = torch.randn(9000, 128, generator=gen, device="cuda")
    want = df2.embedding_grad(dout, ids, 700)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = torch.empty(700, 128, device="cuda")
    for _ in range(20):
        df2.embedding_grad(dout, ids, 700, out=out, stream=st)
        torch.empty(1 << 20, device="cuda").fill_(float("nan"))  # would reuse a scratch freed too early
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(out, want)
