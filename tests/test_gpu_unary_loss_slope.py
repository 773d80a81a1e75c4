"""The softcap's slope where logits saturate it: m (1 - tanh^2 y), y = m u / c, falls off as
4 exp(-2 |y|) and keeps its bits.

Two columns: u = (0, h) or (h, 0), so that dh in fp32 is a row's two factors g as they are held.
Each is off by its rounding to bf16 (2^-8) and, where it is not the target's, to fp16 (2^-11, and 2^-40
of the row's largest); by the errors of exp and the logarithm (2^-17, and 2^-20 of the cap for a
logit); and by the slope's: y is rounded (2^-23 of it), and so is exp's argument (2^-22 of 2 |y|), each
times 2, with a few roundings more: 2^-20 |y| + 2^-19."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def df2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dflash2_draft_block_gb300 as m
    return m


@pytest.mark.parametrize("far", [0, 1])
@pytest.mark.parametrize("target", [0, 1])
@pytest.mark.parametrize("mul, cap", [(1.0, 8.0), (1.0, 30.0), (2.5, 1.5), (0.25, 0.125)])
def test_saturated(df2, mul, cap, target, far):
    y = torch.cat([torch.linspace(0.01, 1.0, 40), torch.linspace(1.0, 14.0, 200)])
    y = torch.cat([y, -y])
    h = torch.zeros(len(y), 8)
    h[:, 1] = y * cap / mul
    h = h.to(BF).cuda()
    W = torch.zeros(2, 8)
    W[far, 1] = 1.0
    W[1 - far, 2] = 1.0
    t = torch.full((len(y),), target, dtype=I32, device="cuda")
    dh = df2.unary_loss_grad(h, W.to(BF).cuda(), t, output_multiplier=mul, final_logit_softcapping=cap, dtype=F32)[2]
    u = h.double() @ W.double().T.cuda()
    y = mul * u / cap
    x = cap * torch.tanh(y)
    slope = mul / torch.cosh(y) ** 2
    lse = torch.logsumexp(x, 1, keepdim=True)
    other = torch.exp(x[:, 1 - target:2 - target] - lse)  # of two, the target's factor is minus the other's
    g = torch.cat([other, other], 1)
    g[:, target] *= -1
    g = g * slope
    room = g.abs() * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -17 + 2.0 ** -20 * cap + 2.0 ** -20 * y.abs() + 2.0 ** -19)
    held = mul * 2.0 ** -40 * torch.exp(x.amax(1) - lse[:, 0])
    got = torch.stack([dh[:, 1 + far], dh[:, 2 - far]], 1).double()  # of columns 0 and 1
    room[:, 1 - target] += held
    off = (got - g).abs() / room
    assert bool((off <= 1.0).all()), (float(off.max()), off.argmax())


def test_far_saturated_targets(df2):
    """The target's factor has a slope of its own, held in fp32 until g: down to exp(-80)."""
    y = torch.linspace(14.0, 40.0, 100)
    y = torch.cat([y, -y])
    cap = 4.0
    h = torch.zeros(len(y), 8)
    h[:, 1] = y * cap
    h = h.to(BF).cuda()
    W = torch.zeros(2, 8)
    W[0, 1] = 1.0
    t = torch.zeros(len(y), dtype=I32, device="cuda")
    dh = df2.unary_loss_grad(h, W.to(BF).cuda(), t, final_logit_softcapping=cap, dtype=F32)[2]
    y = h[:, 1].double() / cap
    x = cap * torch.tanh(y)
    g = -1.0 / (1.0 + torch.exp(x)) / torch.cosh(y) ** 2
    off = (dh[:, 1].double() - g).abs() / g.abs()
    assert bool((off <= 2.0 ** -8 + 2.0 ** -17 + 2.0 ** -18 + 2.0 ** -20 * y.abs() + 2.0 ** -19).all()), float(off.max())
