"""Graph-reading calls of several host threads and streams."""
import threading

import pytest

pytestmark = pytest.mark.gpu

K = pytest.importorskip("compressed_graph_spmv_gb300.k2t")
import compressed_graph_spmv_gb300 as pkg  # noqa: E402

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    K.load()


def together(jobs):
    """Run the jobs in a thread each; the first error of any of them is raised."""
    errors, start = [], threading.Barrier(len(jobs))

    def body(job):
        try:
            start.wait()
            job()
        except Exception as e:   # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=body, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    if errors:
        raise errors[0]


@pytest.mark.parametrize("dims", [(2100, 4001), (2055, 3055)])
def test_norms_of_two_widths_in_two_threads(dims):
    """Widths that share a kernel and need different amounts of shared memory."""
    def job(dim):
        n = 2500                                # several rows a batch, and little time on the GPU
        x = torch.randn(n * dim + 1, device="cuda").to(torch.bfloat16)[1:].view(n, dim)    # not on a 16-byte boundary
        w, op = torch.ones(dim, dtype=torch.bfloat16, device="cuda"), pkg.LayerNorm(n, dim, torch.bfloat16)
        dx, dw = torch.empty_like(x), torch.empty_like(w)

        def go():
            for _ in range(4000):
                op.backward(x, x, w, dx, dw)
        return go
    jobs = [job(d) for d in dims for _ in range(3)]
    torch.cuda.synchronize()
    together(jobs)
