"""The training calls from several host threads at once, each on a stream of its own."""
import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def df2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dflash2_draft_block_gb300 as m
    m.lib()
    return m


def test_two_ranks_of_one_kernel_at_once(df2):
    """Calls that need different amounts of shared memory of the same kernel: neither thread's
    launch is refused, whatever the other asks for in between."""
    P, K, V = 4, 16, 200
    jobs, failed = [], []
    for i, r in enumerate((4096, 2064)):
        gen = torch.Generator(device="cuda").manual_seed(i)
        ids = torch.rand(P, V, generator=gen, device="cuda").topk(K, dim=1).indices.to(torch.int32).contiguous()
        jobs.append(dict(pred=ids[:, 1].contiguous(), targets=ids[:, 0].contiguous(), topk_ids=ids,
                         topk_vals=torch.randn(P, K, generator=gen, device="cuda"),
                         G=torch.randn(P, r, generator=gen, device="cuda") * 0.01,
                         A=torch.randn(V, r, generator=gen, device="cuda").to(torch.bfloat16),
                         Bc=torch.randn(V, r, generator=gen, device="cuda").to(torch.bfloat16), dA=None, dBc=None))
    want = [df2.selector_loss_grad(**c)[:4] for c in jobs]
    outs = [tuple(torch.empty_like(t) for t in w) for w in want]
    torch.cuda.synchronize()
    begin = threading.Barrier(2)

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            begin.wait()
            for _ in range(5000):
                try:
                    df2.selector_loss_grad(**jobs[i], out=outs[i])
                except df2.DFlash2Error as e:
                    failed.append((i, str(e)))
                    return

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for got, was in zip(outs, want):
        assert all(torch.equal(x, y) for x, y in zip(got, was))
