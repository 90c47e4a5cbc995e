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


def attention(n=5000):
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    t = dict(q=rand(9, 4, 64), k=rand(n, 2, 64), v=rand(n, 2, 64), dout=rand(9, 4, 64))
    t.update({"d" + x: torch.empty_like(t[x]) for x in "qkv"}, out=torch.empty_like(t["q"]), lse=torch.empty(9, 4, device="cuda"))
    op = pkg.HopAttention(9, n, 4, 2, 64, torch.bfloat16)
    fwd = lambda stream=None: op.forward(t["q"], t["k"], t["v"], t["out"], t["lse"], stream=stream)  # noqa: E731
    bwd = lambda stream=None: op.backward(t["dout"], t["q"], t["k"], t["v"], t["out"], t["lse"], t["dq"], t["dk"], t["dv"],  # noqa: E731
                                          stream=stream)
    return op, t, fwd, bwd


def test_first_call_on_another_stream_than_the_current():
    """The work buffers and their cleared status words belong to the stream of the call: nothing waits for the current one."""
    op, t, fwd, bwd = attention()
    fwd()
    bwd()
    want = {x: t[x].clone() for x in ("out", "lse", "dq", "dk", "dv")}
    op, t, fwd, bwd = attention()
    stale = [torch.full((op.work_bytes(b),), 0xff, dtype=torch.uint8, device="cuda") for b in (False, True)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    del stale
    torch.cuda._sleep(500_000_000)                     # the current stream is busy for a quarter of a second
    fwd(side)
    bwd(side)
    with torch.cuda.stream(side):
        words = [w[:4].cpu() for w in op._work]         # ordered after the calls on their stream alone
        got = {x: t[x].clone() for x in want}
    assert not torch.cuda.current_stream().query(), "the current stream was to be busy all along"
    assert all((w == 0).all() for w in words)
    torch.cuda.synchronize()
    assert op.status() == 0 and all(torch.equal(want[x], got[x]) for x in want)


@pytest.mark.parametrize("first", ["current", "side"])
def test_buffers_of_an_object_that_goes_while_its_calls_run(first):
    """Memory that another stream still uses is not handed out again."""
    for call in attention()[2:]:
        call()                       # kernels are loaded
    op, t, fwd, bwd = attention()
    warm, norm = (pkg.LayerNorm(4000, 512, torch.bfloat16) for _ in range(2))
    x, w = torch.randn(4000, 512, device="cuda").to(torch.bfloat16), torch.ones(512, dtype=torch.bfloat16, device="cuda")
    y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)
    warm.forward(x, w, None, y)
    warm.backward(x, x, w, dx, dw)
    del warm
    side = torch.cuda.Stream()

    def call(stream):
        fwd(stream)
        bwd(stream)
        norm.forward(x, w, None, y, stream=stream)
        norm.backward(x, x, w, dx, dw, stream=stream)
    if first == "current":
        call(None)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(500_000_000)
    call(side)
    sizes = [op.work_bytes(False), op.work_bytes(True), norm.work_bytes(), 8 * 4000, 4 * 4000]
    held = [(b.at, b.tensor.numel()) for b in (*op._buffers, norm._work, norm._own)]
    del op, fwd, bwd, norm, call
    again = [torch.empty(s, dtype=torch.uint8, device="cuda") for s in sizes for _ in range(3)]
    assert not side.query()
    for a in again:
        assert all(a.data_ptr() + a.numel() <= at or at + size <= a.data_ptr() for at, size in held)
    torch.cuda.synchronize()
