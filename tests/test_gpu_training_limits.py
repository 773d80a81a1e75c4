"""The training calls past 32-bit offsets, inside CUDA graphs, and launched back to back
through one workspace."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def df2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dflash2_draft_block_gb300 as m
    m.lib()
    return m


def test_tables_past_four_gigabytes(df2):
    """Rows whose byte and element offsets pass 2^32: looked up, added to, written among
    zeros."""
    V, D = 540_000, 8200          # 4.4 G elements, 8.9 GB in bf16
    gen = torch.Generator(device="cuda").manual_seed(0)
    table = torch.zeros(V, D, dtype=BF, device="cuda")
    ids = torch.tensor([0, V - 1, V // 2, V - 2, 523_776, 262_144, V - 1], dtype=I32, device="cuda")
    rows = torch.randn(len(ids), D, generator=gen, device="cuda").to(BF)
    table[ids.long()] = rows
    assert torch.equal(df2.embedding(table, ids), table[ids.long()])
    del table
    torch.cuda.empty_cache()
    many = ids.repeat(100)        # long enough to be sorted
    for n, x in ((len(ids), ids), (len(many), many)):
        dout = torch.randn(n, D, generator=gen, device="cuda").to(BF)
        out = torch.full((V, D), 3.0, dtype=BF, device="cuda")
        df2.embedding_grad(dout, x, V, out=out)
        names = x.unique().long()
        want = torch.zeros(len(names), D, device="cuda")
        want.index_add_(0, torch.searchsorted(names, x.long()), dout.float())
        # n / 6 fp32 additions a row, then bf16: half a bf16 step of the terms' size at most
        assert torch.all((out[names].float() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * n)
        mask = torch.ones(V, dtype=torch.bool, device="cuda")
        mask[names] = False
        assert int((out.view(torch.int16).amax(1) != 0)[mask].sum()) == 0 and int((out.view(torch.int16).amin(1) != 0)[mask].sum()) == 0
        del out, mask
        torch.cuda.empty_cache()


def test_a_tensor_past_two_to_the_31(df2):
    """AdamW on one tensor of more than 2^31 elements: its ends step as a small tensor does."""
    n, k = 2 ** 31 + 1003, 100_000
    gen = torch.Generator(device="cuda").manual_seed(1)
    p, g = torch.zeros(n, dtype=BF, device="cuda"), torch.zeros(n, dtype=BF, device="cuda")
    small_p = torch.randn(2 * k + 1000, generator=gen, device="cuda").to(BF)
    small_g = torch.randn(2 * k + 1000, generator=gen, device="cuda").to(BF)
    tail = n // 256 * 256 - k // 256 * 256          # on a block of the states
    p[:k], g[:k] = small_p[:k], small_g[:k]
    p[tail:], g[tail:] = small_p[k:k + n - tail], small_g[k:k + n - tail]
    want = [small_p[:k].clone(), small_p[k:k + n - tail].clone()]
    opt = df2.AdamW([p], [g], lr=0.1, state_bits=8)
    ref = df2.AdamW(want, [small_g[:k].clone(), small_g[k:k + n - tail].clone()], lr=0.1, state_bits=8)
    for _ in range(2):
        opt.step()
        ref.step()
    assert torch.equal(p[:k // 256 * 256], want[0][:k // 256 * 256]) and torch.equal(p[tail:], want[1])
    assert int((p[k + 256:tail - 256] != 0).sum()) == 0


def selector_case(P, K, r, V, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ids = (torch.randint(0, V // K, (P, K), generator=gen, device="cuda") + torch.arange(K, device="cuda") * (V // K)).to(I32)
    return dict(pred=torch.randint(0, V, (P,), generator=gen, device="cuda", dtype=I32),
                targets=ids[:, K // 2].contiguous(), topk_ids=ids,
                topk_vals=torch.randn(P, K, generator=gen, device="cuda"), G=torch.randn(P, r, generator=gen, device="cuda"),
                A=torch.randn(V, r, generator=gen, device="cuda").to(BF), Bc=torch.randn(V, r, generator=gen, device="cuda").to(BF))


@pytest.mark.parametrize("P, K, r, V", [(16, 4, 32, 400), (300, 16, 256, 3000), (9000, 16, 64, 8000)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_a_step_in_a_cuda_graph(df2, P, K, r, V, accumulate):
    """Captured once, replayed on other inputs: what the direct calls give, bit for bit."""
    c = selector_case(P, K, r, V)
    A0, B0 = c["A"].clone(), c["Bc"].clone()
    dA, dBc, dE = (torch.zeros(V, r, device="cuda") for _ in range(3))
    out = (torch.empty(P, device="cuda"), torch.empty(P, dtype=I32, device="cuda"), torch.empty(P, K, device="cuda"),
           torch.empty(P, r, device="cuda"))

    def step():
        rows = df2.embedding(c["A"], c["pred"], dtype=F32)
        df2.selector_loss_grad(**c, dA=dA, dBc=dBc, accumulate=accumulate, out=out)
        df2.embedding_grad(rows, c["pred"], V, out=dE, accumulate=accumulate)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                     # attributes and queries before the capture
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        fresh = selector_case(P, K, r, V, seed)
        for k in c:
            c[k].copy_(fresh[k])
        for t in (dA, dBc, dE):
            t.fill_(0.5)
        graph.replay()
        got = [t.clone() for t in (*out, dA, dBc, dE)]
        for t in (dA, dBc, dE):
            t.fill_(0.5)
        step()
        torch.cuda.synchronize()
        for x, y in zip(got, (*out, dA, dBc, dE)):
            assert torch.equal(x, y)
    assert not torch.equal(A0, c["A"]) and not torch.equal(B0, c["Bc"])


def test_back_to_back_through_one_workspace(df2):
    """Calls of different sizes that share a workspace, not waited for in between: the sort of
    one must not start before the join of the last is done."""
    shapes = [(9000, 16, 64, 8000), (40, 4, 64, 8000), (2000, 16, 64, 8000)]
    cases = [selector_case(*s, seed=i) for i, s in enumerate(shapes)]
    ws = torch.empty(max(df2.selector_loss_grad_workspace_size(s[0], s[3], s[1], s[2]) for s in shapes),
                     dtype=torch.uint8, device="cuda")
    want = [df2.selector_loss_grad(**c) for c in cases]
    torch.cuda.synchronize()
    got = [[df2.selector_loss_grad(**c, workspace=ws) for c in cases] for _ in range(10)]
    torch.cuda.synchronize()
    for rnd in got:
        for a, b in zip(rnd, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
