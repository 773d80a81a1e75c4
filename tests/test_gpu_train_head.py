"""The head's training calls as a step uses them: dropout with the residual stream, the unary loss with
its gradients, dropout's gradient and the embedding's, against the same chain in 64 bits; and the
example's run with both."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from dropout_words import dropped  # noqa: E402
from unary_loss_ref import reference  # noqa: E402

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def df2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dflash2_draft_block_gb300 as m
    return m


def test_a_step_against_64_bits(df2):
    """x = E[ids], h = x + dropout(x2), loss(h W^T), back to E and W, step by step: each call's own
    roundings are what its tests allow, so the inputs of each are taken as they are held."""
    P, V, D, rate, seed, draw = 96, 700, 128, 0.2, 99, 12345
    g = torch.Generator().manual_seed(3)
    E, W = (torch.randn(V, D, generator=g).to(BF).cuda(), (torch.randn(V, D, generator=g) / 6).to(BF).cuda())
    x2 = torch.randn(P, D, generator=g).to(BF).cuda()
    ids = torch.randint(-1, V, (P,), generator=g).to(I32).cuda()
    t = torch.randint(-1, V, (P,), generator=g).to(I32).cuda()
    w = torch.rand(P, generator=g).cuda()
    x = df2.embedding(E, ids)
    h = df2.dropout(x2, rate, seed, draw, residual=x)
    loss, lse, dh, dW = df2.unary_loss_grad(h, W, t, row_weights=w, dW=True, dtype=F32)
    dx2 = df2.dropout_grad(dh, rate, seed, draw)
    dE = df2.embedding_grad(dh, ids, V)
    torch.cuda.synchronize()
    y, keep = dropped(x2.double().cpu().numpy(), rate, seed, draw)
    y = torch.from_numpy(y).cuda() + x.double()
    assert bool(((h.double() - y).abs() <= (2.0 ** -8 + 2.0 ** -21) * y.abs() + 2.0 ** -21 * x2.double().abs()).all())
    (_, _, rdh, rdW), room = reference(h, W, t, w)
    assert bool(((dh.double() - rdh).abs() <= room["dh"] + 2.0 ** -23 * rdh.abs()).all())
    assert bool(((dW.double() - rdW).abs() <= room["dW"] + 2.0 ** -23 * rdW.abs()).all())
    scale = 65536.0 / (65536 - 13107)
    want = torch.where(torch.from_numpy(keep).cuda(), dh.double() * scale, torch.zeros_like(rdh))
    assert bool(((dx2.double() - want).abs() <= 2.0 ** -22 * want.abs()).all())
    sums = torch.zeros(V, D, dtype=torch.float64, device="cuda")
    sums.index_add_(0, ids.clamp(min=0).long(), torch.where(ids[:, None] >= 0, dh.double(), torch.zeros_like(rdh)))
    parts = torch.zeros_like(sums).index_add_(0, ids.clamp(min=0).long(), dh.double().abs())
    assert bool(((dE.double() - sums).abs() <= 2.0 ** -20 * parts).all())


def test_micro_batches_add_up(df2):
    """dW of two halves, the second added to the first, is dW of both within a few roundings."""
    g = torch.Generator().manual_seed(4)
    h, W = torch.randn(400, 192, generator=g).to(BF).cuda(), (torch.randn(900, 192, generator=g) / 8).to(BF).cuda()
    t = torch.randint(-1, 900, (400,), generator=g).to(I32).cuda()
    dW = torch.empty(900, 192, device="cuda")
    df2.unary_loss_grad(h[:256], W, t[:256], dW=dW)
    df2.unary_loss_grad(h[256:], W, t[256:], dW=dW, accumulate=True)
    (_, _, _, want), room = reference(h, W, t)
    assert bool(((dW.double() - want).abs() <= room["dW"] + 2.0 ** -22 * want.abs()).all())


@pytest.fixture(scope="module")
def example(df2):
    spec = importlib.util.spec_from_file_location("train_selector", os.path.join(ROOT, "examples", "train_selector.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_the_example_runs_with_both(example):
    a, b = (example.train(steps=6, positions=600, head_loss=0.2, dropout=0.1) for _ in range(2))
    assert a == b and all(x == x for x in a)
    assert example.train(steps=6, positions=600) != a
