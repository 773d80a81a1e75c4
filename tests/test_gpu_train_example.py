"""The training example end to end: the loss of either state width falls well below the
loss of an untrained selector (ln K = 2.77 and more at the start)."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("train_selector", os.path.join(ROOT, "examples", "train_selector.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("bits", [32, 8])
def test_the_selector_learns(example, bits):
    losses = example.train(steps=60, state_bits=bits)
    assert all(x == x for x in losses)
    assert min(losses[-5:]) < 0.5 * losses[0]


def test_the_same_run_twice_is_the_same_bit_for_bit(example):
    """Nothing in a step depends on the order in which threads arrive."""
    assert example.train(steps=8, positions=3000) == example.train(steps=8, positions=3000)
