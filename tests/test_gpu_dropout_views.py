"""Dropout on views that share no element but lie between one another: parts of one wide matrix, and
every other row.  The mask is the index's, so each gives what separate tensors give, bit for bit, and
nothing beside it is written."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def df2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dflash2_draft_block_gb300 as m
    return m


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N, D, gap", [(50, 64, 0), (50, 64, 8), (33, 37, 0), (7, 1, 0), (2, 4096, 3)])
def test_parts_of_a_wide_matrix(df2, dtype, N, D, gap):
    wide = torch.randn(N, 3 * D + 2 * gap, generator=torch.Generator().manual_seed(D)).to(dtype).cuda()
    x, r, y = (wide[:, k * (D + gap): k * (D + gap) + D] for k in range(3))
    before = wide.clone()
    want = df2.dropout(x.contiguous(), 0.3, 5, 6, residual=r.contiguous())
    assert df2.dropout(x, 0.3, 5, 6, residual=r, out=y) is y
    assert torch.equal(y, want)
    y.copy_(before[:, 2 * (D + gap):])
    assert torch.equal(wide, before)
    df2.dropout(y, 0.3, 5, 6, out=x)  # the other way round
    assert torch.equal(x, df2.dropout(y.contiguous(), 0.3, 5, 6))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 37])
def test_every_other_row(df2, dtype, D):
    rows = torch.randn(40, D, generator=torch.Generator().manual_seed(D)).to(dtype).cuda()
    x, y = rows[0::2], rows[1::2]
    want, kept = df2.dropout(x.contiguous(), 0.5, 1, 2), x.clone()
    df2.dropout(x, 0.5, 1, 2, out=y)
    assert torch.equal(y, want) and torch.equal(x, kept)


def test_shared_elements_are_refused(df2):
    wide = torch.zeros(20, 64, device="cuda")
    for x, y in ((wide[:, :40], wide[:, 24:]), (wide[:, 24:], wide[:, :40]), (wide[:10], wide[5:15]),
                 (wide[:19, :32], wide[1:, :32])):
        with pytest.raises(df2.DFlash2Error):
            df2.dropout(x, 0.5, 1, out=y)
        if x.shape == y.shape:
            with pytest.raises(df2.DFlash2Error):
                df2.dropout(torch.zeros_like(x), 0.5, 1, residual=x, out=y)
