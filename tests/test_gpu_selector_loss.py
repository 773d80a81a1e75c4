"""dflash2_selector_loss_grad against the formula in 64 bits.

Tolerances, with u = 2^-24 and |.| the sums of the terms' sizes.  A score is r + 2
rounded operations on exact bf16 values: within (r + 2) u |s|, |s| = |val| + sum |u||Bc|.
Call the row's largest such error e (plus the row's loss arithmetic, 16 u of
max(1, |s|max)).  Probabilities then move by at most 2 e of themselves, so dscores within
w (2 e + (K + 16) u); t, of K terms, within sum_j |Bc| (that + K u); dG and the tables'
gradients follow by products and sums of c terms, each adding its own (c + 2) u of its
terms' sizes.  A table gradient held in bf16 lies between the bf16 roundings of the ends
of its interval."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module")
def df2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dflash2_draft_block_gb300 as m
    m.lib()
    return m


def case(seed, P, K, r, V, covered=0.7, std=0.3):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    ids = torch.rand(P, V, generator=gen, device="cuda").topk(K, dim=1).indices.to(torch.int32) if V <= 4096 else \
        (torch.randint(0, V // K, (P, K), generator=gen, device="cuda") + torch.arange(K, device="cuda") * (V // K)).to(torch.int32)
    col = torch.randint(0, K, (P,), generator=gen, device="cuda")
    hit = torch.rand(P, generator=gen, device="cuda") < covered
    targets = torch.where(hit, ids.gather(1, col[:, None])[:, 0], torch.full((P,), -1, dtype=torch.int32, device="cuda"))
    # a quarter of the uncovered rows name a token that is no candidate
    other = (ids[:, 0] + 1) % V
    away = (ids != other[:, None]).all(1) & ~hit & (torch.rand(P, generator=gen, device="cuda") < 0.25)
    targets = torch.where(away, other, targets).to(torch.int32)
    return dict(pred=torch.randint(0, V, (P,), generator=gen, device="cuda", dtype=torch.int32), targets=targets,
                topk_ids=ids.contiguous(), topk_vals=n(P, K) * 2, G=n(P, r), A=(n(V, r) * std).to(BF),
                Bc=(n(V, r) * std).to(BF), row_weights=torch.rand(P, generator=gen, device="cuda") / P)


def reference(c, live):
    """The values in 64 bits and their tolerances, for the rows `live` (a mask); others hold
    nothing."""
    P, K = c["topk_ids"].shape
    V, r = c["A"].shape
    z = lambda t: torch.where(live.view(-1, *[1] * (t.dim() - 1)), t, torch.zeros_like(t))
    pred = torch.where(live, c["pred"], torch.zeros_like(c["pred"])).long()
    ids = z(c["topk_ids"]).long()
    a, G = c["A"].to(F64)[pred], z(c["G"]).to(F64)
    b, vals = c["Bc"].to(F64)[ids], z(c["topk_vals"]).to(F64)
    w = z(c["row_weights"] if c["row_weights"] is not None else torch.ones(P, device="cuda")).to(F64)[:, None]
    u = a * G
    s = vals + torch.einsum("pr,pkr->pk", u, b)
    size = vals.abs() + torch.einsum("pr,pkr->pk", u.abs(), b.abs())
    size = torch.where(size.isfinite(), size, torch.zeros_like(size))
    e = (r + 2) * U * size.amax(1, keepdim=True) + 16 * U * size.amax(1, keepdim=True).clamp(min=1)
    is_label = (ids == c["targets"][:, None]) & live[:, None]
    first = is_label & (is_label.int().cumsum(1) == 1)
    prob = torch.softmax(s, 1)
    loss = torch.logsumexp(s, 1) - torch.where(first, s, torch.zeros_like(s)).sum(1)
    ds = torch.where(live[:, None], w * (prob - first.to(F64)), torch.zeros_like(s))
    ds_tol = w.abs() * (2 * e + (K + 16) * U)
    t = torch.einsum("pk,pkr->pr", ds, b)
    t_tol = (ds_tol[:, :, None] * b.abs()).sum(1) + (K + 2) * U * torch.einsum("pk,pkr->pr", ds.abs(), b.abs())
    dG, dG_tol = a * t, a.abs() * (t_tol + 2 * U * t.abs())
    gt, gt_tol = G * t, G.abs() * (t_tol + 2 * U * t.abs())
    n_a = torch.zeros(V, dtype=F64, device="cuda").index_add_(0, pred, live.to(F64))[:, None]
    add = lambda at, x: torch.zeros(V, r, dtype=F64, device="cuda").index_add_(0, at, x)
    dA, dA_tol = add(pred, gt), add(pred, gt_tol) + (n_a + 2) * U * add(pred, gt.abs())
    flat = ids.reshape(-1)
    n_b = torch.zeros(V, dtype=F64, device="cuda").index_add_(0, flat, live.to(F64).repeat_interleave(K))[:, None]
    du = lambda d, x: (d[:, :, None] * x[:, None, :]).reshape(-1, r)
    dBc = add(flat, du(ds, u))
    dBc_tol = add(flat, du(ds_tol + 3 * U * ds.abs(), u.abs())) + (n_b + 2) * U * add(flat, du(ds.abs(), u.abs()))
    label = torch.where(live, first.int().argmax(1), torch.full((P,), -1, device="cuda")).to(torch.int32)
    return dict(loss=(loss, 2 * e[:, 0] + (K + 16) * U), label=label, ds=(ds, ds_tol * live[:, None]),
                dG=(dG, dG_tol), dA=(dA, dA_tol), dBc=(dBc, dBc_tol))


def near(got, want, tol, what):
    if got.dtype == BF:
        assert torch.all(got >= (want - tol).to(BF)) and torch.all(got <= (want + tol).to(BF)), what
    else:
        off = (got.to(F64) - want).abs() - tol
        assert torch.all(off <= 0), f"{what}: {float(off.max())} over"


def check(df2, c, live, dtype=F32, **kw):
    P, K = c["topk_ids"].shape
    got = df2.selector_loss_grad(**c, dtype=dtype, **kw)
    ref = reference(c, live)
    loss, label, ds, dG, dA, dBc = got
    assert torch.equal(label, ref["label"])
    assert torch.equal(loss.isnan(), ~live)
    near(loss[live], ref["loss"][0][live], ref["loss"][1][live], "loss")
    for name, x in (("ds", ds), ("dG", dG), ("dA", dA), ("dBc", dBc)):
        if x is not None:
            near(x, *ref[name], name)
    assert torch.all(ds[~live] == 0) and torch.all(dG[~live] == 0)
    return got, ref


def covered_rows(c):
    return (c["topk_ids"] == c["targets"][:, None]).any(1)


@pytest.mark.parametrize("P, K, r, V", [
    (1, 1, 8, 1), (1, 16, 256, 5000), (5, 3, 24, 100), (33, 4, 32, 64), (64, 7, 40, 300), (40, 17, 64, 500),
    (17, 33, 72, 700), (20, 16, 128, 900), (9, 65, 136, 400), (300, 16, 256, 2000), (12, 129, 256, 1000),
    (10, 64, 512, 3000), (6, 65, 520, 600), (5, 10, 1024, 300), (3, 40, 1032, 200), (4, 9, 2048, 100),
    (2, 12, 2056, 60), (3, 9, 4096, 50), (2, 1024, 64, 1500), (1, 1000, 4096, 1100), (700, 2, 16, 9),
])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_shapes(df2, P, K, r, V, dtype):
    c = case(P * 31 + K, P, K, r, V)
    live = covered_rows(c)
    got, _ = check(df2, c, live, dtype)
    again = df2.selector_loss_grad(**c, dtype=dtype)
    for x, y in zip(got, again):
        assert torch.equal(x.nan_to_num(7.0), y.nan_to_num(7.0))
    # the loss is selector_ce's on selector_pair_scores' scores, to the same tolerance
    s = df2.selector_pair_scores(c["pred"], c["topk_ids"], c["topk_vals"], c["G"], c["A"], c["Bc"])
    loss, label = df2.selector_ce(s, c["topk_ids"], c["targets"], V)
    assert torch.equal(label, got[1])
    ref = reference(c, live)
    near(loss[live], ref["loss"][0][live], ref["loss"][1][live], "selector_ce")


@pytest.mark.parametrize("P, K, r, V", [
    (5003, 16, 256, 9000), (2441, 17, 72, 700), (2500, 8, 136, 500), (3001, 1, 1024, 300), (2600, 128, 8, 3000),
    (2433, 33, 40, 900), (1300, 40, 256, 2000), (700, 64, 256, 4000), (650, 100, 200, 1000), (400, 64, 512, 5000),
    (311, 31, 1000, 600), (305, 128, 264, 800), (320, 2, 4096, 200),
])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_many_rows(df2, P, K, r, V, dtype):
    """More rows than the GPU holds at once, and candidate lists long enough to be sorted in
    every size class (up to 16 k, 64 k and more positions, one of several tiles a CTA)."""
    c = case(P + K, P, K, r, V)
    live = covered_rows(c)
    c["G"][~live] = float("nan")
    got, _ = check(df2, c, live, dtype)
    again = df2.selector_loss_grad(**c, dtype=dtype)
    for x, y in zip(got, again):
        assert torch.equal(x.nan_to_num(7.0), y.nan_to_num(7.0))
    # without the tables nothing is sorted, and the rows run by themselves
    part = df2.selector_loss_grad(**c, dA=None, dBc=None)
    for x, y in zip(part[:4], got[:4]):
        assert torch.equal(x.nan_to_num(7.0), y.nan_to_num(7.0))


def test_many_rows_masks_and_bad_ids(df2):
    c = case(21, 3000, 16, 256, 4000, covered=1.0)
    bad = torch.arange(3000, device="cuda") % 97 == 0
    c["topk_ids"][bad, 3] = 4000
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    check(df2, c, covered_rows(c) & ~bad, dev_status=st)
    assert int(st) == df2.DF2_STATUS_ID_OUT_OF_RANGE
    none = torch.arange(3000, device="cuda") % 89 == 0
    c["topk_vals"][none] = float("-inf")
    got = df2.selector_loss_grad(**c)
    dead = bad | none
    assert torch.all(got[1][dead] == -1) and torch.all(got[0][dead].isnan()) and torch.all(got[2][dead] == 0)
    assert torch.all(got[1][~dead] >= 0) and all(torch.all(x.isfinite()) for x in got[2:])


@pytest.mark.parametrize("covered", [0.0, 1.0])
def test_no_row_and_every_row(df2, covered):
    c = case(5, 50, 8, 64, 400, covered)
    got, _ = check(df2, c, covered_rows(c))
    if covered == 0.0:
        assert torch.all(got[4] == 0) and torch.all(got[5] == 0)


def test_accumulate_frozen_and_unweighted(df2):
    c = case(6, 90, 16, 256, 1200)
    live = covered_rows(c)
    c["row_weights"] = None
    for dtype in (F32, BF):
        dA0, dBc0 = (torch.randn(1200, 256, device="cuda").to(dtype) for _ in range(2))
        dA, dBc = dA0.clone(), dBc0.clone()
        df2.selector_loss_grad(**c, dA=dA, dBc=dBc, accumulate=True)
        ref = reference(c, live)
        for got, was, (want, tol) in ((dA, dA0, ref["dA"]), (dBc, dBc0, ref["dBc"])):
            near(got, was.to(F64) + want, tol + 2 * U * (was.to(F64).abs() + want.abs()), "accumulated")
            untouched = want.abs().sum(1) == 0
            assert torch.equal(got[untouched], was[untouched])
    full = df2.selector_loss_grad(**c)
    part = df2.selector_loss_grad(**c, dA=None)
    assert part[4] is None and torch.equal(part[5], full[5])
    part = df2.selector_loss_grad(**c, dBc=None)
    assert part[5] is None and torch.equal(part[4], full[4])


def test_what_dropped_rows_hold_is_not_used(df2):
    """NaN and infinities in the rows without a label, and in their weights, reach nothing."""
    c = case(7, 80, 16, 256, 900)
    live = covered_rows(c)
    clean = df2.selector_loss_grad(**c)
    c["G"][~live] = float("nan")
    c["topk_vals"][~live] = float("inf")
    c["row_weights"][~live] = float("nan")
    dirty = df2.selector_loss_grad(**c)
    for x, y in zip(clean, dirty):
        assert torch.equal(x.nan_to_num(3.0), y.nan_to_num(3.0))


def test_masked_candidates(df2):
    """-inf and the lowest fp32 as masks: no probability, no gradient; a row of nothing but
    -inf contributes nothing."""
    c = case(8, 60, 16, 64, 500, covered=1.0)
    live = covered_rows(c)
    is_label = c["topk_ids"] == c["targets"][:, None]
    mask = (torch.rand(60, 16, device="cuda") < 0.5) & ~is_label
    low = torch.finfo(F32).min
    for value in (float("-inf"), low):
        m = dict(c, topk_vals=torch.where(mask, torch.full_like(c["topk_vals"], value), c["topk_vals"]))
        m["topk_vals"][3] = float("-inf")
        got = df2.selector_loss_grad(**m)
        assert int(got[1][3]) == -1 and bool(got[0][3].isnan())
        assert torch.all(got[2][3] == 0) and torch.all(got[3][3] == 0)
        keep = torch.arange(60, device="cuda") != 3
        assert torch.all(got[2][mask & keep[:, None]] == 0)
        assert all(torch.all(x[keep].isfinite()) for x in got[:4]) and all(torch.all(x.isfinite()) for x in got[4:])
        # against the row without its masked candidates
        for p in (0, 1, 2, 59):
            s = c["topk_vals"][p].to(F64) + c["Bc"][c["topk_ids"][p].long()].to(F64) @ (
                c["A"][int(c["pred"][p])].to(F64) * c["G"][p].to(F64))
            s = s[~mask[p]]
            prob = torch.softmax(s, 0) - is_label[p][~mask[p]].to(F64)
            tol = 64 * 2 * U * (1 + s.abs().max()) * 3 + 32 * U
            near(got[2][p][~mask[p]], prob * float(c["row_weights"][p]), tol * float(c["row_weights"][p]), "masked row")


@pytest.mark.parametrize("where", ["pred", "candidate", "target", "negative candidate", "negative pred"])
def test_bad_ids_drop_their_row(df2, where):
    c = case(9, 40, 16, 128, 300, covered=1.0)
    V = 300
    bad = torch.zeros(40, dtype=torch.bool, device="cuda")
    bad[[0, 17, 39]] = True
    if where == "pred":
        c["pred"][bad] = V
    elif where == "negative pred":
        c["pred"][bad] = -1
    elif where == "target":
        c["targets"][bad] = V + 5
    else:
        c["topk_ids"][bad, 11] = -1 if where == "negative candidate" else 2 ** 31 - 1
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    check(df2, c, covered_rows(c) & ~bad, dev_status=st)
    assert int(st) == df2.DF2_STATUS_ID_OUT_OF_RANGE


def test_same_candidate_twice_and_shared_tokens(df2):
    """Repeated candidates in a row, one token in every row, one predecessor for all: the
    sums over them are whole."""
    c = case(10, 500, 8, 64, 50, covered=1.0)
    c["topk_ids"][:, 0] = 7
    c["topk_ids"][::3, 5] = c["topk_ids"][::3, 4]
    c["pred"][:] = 11
    c["targets"] = c["topk_ids"][:, 4].contiguous()
    check(df2, c, covered_rows(c))


def test_gradients_against_differences(df2):
    """Central differences of sum(w * loss) in 64 bits of the loss formula, at coordinates of
    every input (the truncation error of h = 1e-4 is below 1e-6 of the gradients' size)."""
    c = case(11, 6, 5, 16, 30, covered=1.0)
    loss, label, ds, dG, dA, dBc = df2.selector_loss_grad(**c)
    x = {k: c[k].to(F64) for k in ("topk_vals", "G", "A", "Bc")}
    w = c["row_weights"].to(F64)

    def f():
        u = x["A"][c["pred"].long()] * x["G"]
        s = x["topk_vals"] + (u[:, None] * x["Bc"][c["topk_ids"].long()]).sum(2)
        return (w * (torch.logsumexp(s, 1) - s.gather(1, label.long()[:, None])[:, 0])).sum()

    h = 1e-4
    for name, grad in (("topk_vals", ds), ("G", dG), ("A", dA), ("Bc", dBc)):
        t = x[name]
        rows = torch.randperm(t.shape[0], device="cuda")[:6]
        if name == "A":
            rows = c["pred"].long()
        if name == "Bc":
            rows = c["topk_ids"].long()[:, 0]
        for i in rows.tolist():
            for j in (0, t.shape[1] // 2, t.shape[1] - 1):
                v = float(t[i, j])
                t[i, j] = v + h
                up = float(f())
                t[i, j] = v - h
                down = float(f())
                t[i, j] = v
                assert abs((up - down) / (2 * h) - float(grad[i, j])) <= 1e-6 * float(w.max()) * 10, (name, i, j)


def test_empty_and_another_stream(df2):
    c = case(12, 2000, 16, 256, 5000)
    e = {k: (v[:0] if k not in ("A", "Bc") else v) for k, v in c.items()}
    got = df2.selector_loss_grad(**e)
    assert got[0].shape == (0,) and torch.all(got[4] == 0) and torch.all(got[5] == 0)
    want = df2.selector_loss_grad(**c)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = tuple(torch.empty_like(t) for t in want)
    for _ in range(10):
        df2.selector_loss_grad(**c, dA=out[4], dBc=out[5], out=out[:4], stream=st)
        torch.empty(1 << 22, device="cuda").fill_(float("nan"))
    torch.cuda.current_stream().wait_stream(st)
    for x, y in zip(out, want):
        assert torch.equal(x.nan_to_num(3.0), y.nan_to_num(3.0))
