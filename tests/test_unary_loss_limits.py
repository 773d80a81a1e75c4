"""Multipliers and caps that the unary loss's fp32 arithmetic cannot carry are refused, and their
neighbours are not.  (The library's own checks, which return before they touch a device: every call here
has no workspace and ends at that check at the latest.)"""
import numpy as np
import pytest

from dflash2_draft_block_gb300 import _abi, build

P, D, V = 12, 24, 50
UNSUPPORTED, NO_DEVICE, NO_WORKSPACE = 2, 3, 4


@pytest.fixture(scope="module")
def calls():
    build.build()
    lib, base = _abi.load(), 1 << 24

    def both(mul, cap):
        ce = lib.dflash2_unary_ce(base, P, D, 2 * base, V, mul, cap, 3 * base, 4 * base, 5 * base, 0, 0, 0, None)
        grad = lib.dflash2_unary_loss_grad(base, P, D, 2 * base, V, mul, cap, 3 * base, 0, 0, 4 * base, 5 * base, 6 * base, 0,
                                           7 * base, 0, 0, 0, 0, None)
        assert ce == grad
        return ce
    return both


def test_multipliers_whose_exponent_overflows(calls):
    """Without a cap exp's argument is the raw difference times log2(e) m, which is infinite for a
    finite m above FLT_MAX / log2(e): times the largest column's 0 it was NaN."""
    log2e, most = np.float32(1.4426950408889634), np.finfo(np.float32).max
    edge = np.float32(np.float64(most) / np.float64(log2e))
    with np.errstate(over="ignore"):
        for mul in (np.nextafter(edge, np.float32(0)), edge, np.nextafter(edge, most), np.float32(3e38), most):
            fits = bool(np.isfinite(log2e * mul))
            assert calls(float(mul), 0.0) in ((NO_DEVICE, NO_WORKSPACE) if fits else (UNSUPPORTED,)), mul
        assert not np.isfinite(log2e * np.float32(2.4e38)) and np.isfinite(log2e * np.float32(2.3e38))
    assert calls(2.4e38, 1e10) in (NO_DEVICE, NO_WORKSPACE)  # (m / c and log2(e) apart)


def test_caps_whose_quotient_is_subnormal(calls):
    """tanh's argument is the logit times m / c: below 2^-126 that has lost bits (1e-5 / 1e38 is off by
    half a percent, and every logit with it)."""
    quotient = np.float32(1e-5) / np.float32(1e38)
    assert abs(float(quotient) / (float(np.float32(1e-5)) / float(np.float32(1e38))) - 1.0) > 1e-3
    least = np.finfo(np.float32).tiny
    for mul, cap in ((1e-5, 1e38), (1e-30, 1e30), (1.0, 3e38), (1e-37, 30.0), (1e-38, 0.5)):
        fits = bool(np.float32(mul) / np.float32(cap) >= least)
        assert calls(mul, cap) in ((NO_DEVICE, NO_WORKSPACE) if fits else (UNSUPPORTED,)), (mul, cap)
    assert calls(1.0, 8e37) in (NO_DEVICE, NO_WORKSPACE) and calls(1e-37, 0.0) in (NO_DEVICE, NO_WORKSPACE)
