"""The AdamW handle on the GPU: states that move between steps, steps under capture, and
parameters whose gradients come late."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def df2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dflash2_draft_block_gb300 as m
    m.lib()
    return m


def randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("first", [2, 7])
def test_a_late_gradient_starts_at_step_one(df2, bits, first):
    """A parameter counts its own steps: one whose gradient comes at step `first` moves as in an
    optimiser of its own, also after the states went through state_dict()."""
    p, q = randn(0, 1000), randn(1, 700)
    p1, q1 = p.clone(), q.clone()
    kw = dict(lr=1e-2, weight_decay=0.1, state_bits=bits)
    both, a, b = df2.AdamW([p, q], **kw), df2.AdamW([p1], **kw), df2.AdamW([q1], **kw)
    for t in range(1, 12):
        gp, gq = randn(10 + t, 1000), randn(50 + t, 700)
        both.step([gp, gq if t >= first else None])
        a.step([gp])
        if t >= first:
            b.step([gq])
        if t == first + 2:
            both = df2.AdamW([p, q], **kw, **both.state_dict())
    torch.cuda.synchronize()
    assert torch.equal(p, p1) and torch.equal(q, q1)
    assert both.step_count == 11


def test_a_step_is_not_captured(df2):
    """A replayed step would be the same step for ever: capture is refused, and nothing counts."""
    p, g = randn(2, 5000), randn(3, 5000)
    opt = df2.AdamW([p], [g])
    opt.step()
    torch.cuda.synchronize()
    was = p.clone()
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="captur"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            opt.step()
    torch.cuda.synchronize()
    assert opt.step_count == 1 and torch.equal(p, was)
    opt.step()
    torch.cuda.synchronize()
    assert opt.step_count == 2 and not torch.equal(p, was)


@pytest.mark.parametrize("bits", [32, 8])
def test_states_that_went_to_the_host_and_back(df2, bits):
    """Every state, scale and master moved through host memory between two steps, in place and as
    replaced lists: the same weights as without."""
    p, gs = randn(4, 3000).to(BF), [randn(20 + t, 3000) for t in range(6)]
    q = p.clone()
    kw = dict(lr=1e-2, state_bits=bits, master_weights=True)
    stay, move = df2.AdamW([p], **kw), df2.AdamW([q], **kw)
    for t, g in enumerate(gs):
        if t in (2, 3):
            for ts in (*move.state.values(), move.master_weights):
                for x in ts:
                    x.data = x.data.cpu()
            torch.empty(1 << 20, device="cuda").fill_(float("nan"))   # takes what they left
            for ts in (*move.state.values(), move.master_weights):
                for x in ts:
                    x.data = x.data.cuda()
        if t == 4:
            move.state = {k: [x.clone() for x in ts] for k, ts in move.state.items()}
            move.master_weights = [x.clone() for x in move.master_weights]
        stay.step([g])
        move.step([g])
    torch.cuda.synchronize()
    assert torch.equal(p, q)
    for k in stay.state:
        assert torch.equal(stay.state[k][0].view(torch.uint8), move.state[k][0].view(torch.uint8)), k
