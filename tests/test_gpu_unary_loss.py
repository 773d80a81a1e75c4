"""unary_ce and unary_loss_grad on the GPU against their definition in 64 bits, element by
element within what the roundings allow (unary_loss_ref)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from unary_loss_ref import check, reference  # noqa: E402

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def df2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dflash2_draft_block_gb300 as m
    return m


def inputs(seed, P, V, D, spread=2.5, raised=12.0, masked=0.2):
    """Logits of deviation `spread`, targets raised by up to `raised`, a share without a target."""
    g = torch.Generator().manual_seed(seed)
    W = (torch.randn(V, D, generator=g) * (spread / D ** 0.5)).to(BF)
    t = torch.randint(0, V, (P,), generator=g)
    up = torch.rand(P, 1, generator=g) * raised / spread ** 2
    h = (torch.randn(P, D, generator=g) + up * W[t].float()).to(BF)
    t = torch.where(torch.rand(P, generator=g) < masked, torch.full_like(t, -1), t).to(I32)
    w = torch.rand(P, generator=g) * 2
    return h.cuda(), W.cuda(), t.cuda(), w.cuda()


def compare(df2, h, W, t, w, mul=1.0, cap=0.0, dtype=BF, dW=True, accumulate=False, **more):
    keep = dW.clone() if isinstance(dW, torch.Tensor) else None
    want, room = reference(h, W, t, w, mul, cap, keep if accumulate else None)
    got = df2.unary_loss_grad(h, W, t, row_weights=w, output_multiplier=mul, final_logit_softcapping=cap, dtype=dtype,
                              dW=dW, accumulate=accumulate, **more)
    if accumulate:  # the old value, as it is held, is added in fp32
        room["dW"] = room["dW"] + 2.0 ** -24 * (want[3].abs() + keep.double().abs())
    worst = {n: check(n, a, b, room[n]) for n, a, b in zip(("loss", "lse", "dh", "dW"), got, want) if a is not None}
    loss, lse = df2.unary_ce(h, W, t, output_multiplier=mul, final_logit_softcapping=cap)
    assert torch.equal(loss.nan_to_num(-1.0), got[0].nan_to_num(-1.0))
    assert torch.equal(lse.nan_to_num(-1.0), got[1].nan_to_num(-1.0))
    return worst


SIZES = [(1, 1, 8), (1, 2, 8), (3, 5, 16), (8, 127, 64), (8, 1000, 72), (16, 4096, 256), (63, 129, 520), (64, 257, 64),
         (65, 255, 8), (130, 777, 1032), (256, 256, 512), (257, 513, 264), (300, 2050, 576), (600, 9001, 136),
         (5, 33001, 1024)]


@pytest.mark.parametrize("P, V, D", SIZES)
def test_sizes(df2, P, V, D):
    compare(df2, *inputs(P + V, P, V, D))


@pytest.mark.parametrize("mul, cap", [(1.0, 0.0), (0.8, 0.0), (1.0, 30.0), (0.5, 5.0), (3.0, 2.0)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_maps_and_types(df2, mul, cap, dtype):
    compare(df2, *inputs(3, 140, 1500, 200), mul=mul, cap=cap, dtype=dtype)
