"""Norm and rotation of each head on the GPU against 64-bit references, element
by element within the bounds of tests/cache_ref.py."""
import numpy as np
import pytest

import cache_ref as ref
from test_gpu_reader import DT, close, dev, f64, padded

pytestmark = pytest.mark.gpu

K = pytest.importorskip("compressed_graph_spmv_gb300.k2t")
import compressed_graph_spmv_gb300 as pkg  # noqa: E402

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    K.load()


def problem(n, heads, d, dtype, span, seed, weighted=True):
    rng = np.random.default_rng(seed)
    p = dict(x=dev(rng, dtype, n, heads, d), dy=dev(rng, dtype, n, heads, d),
             weight=(1 + dev(rng, "fp32", d, scale=0.2)).to(DT[dtype]) if weighted else None,
             positions=torch.from_numpy(rng.integers(-span, span + 1, size=n).astype(np.int32)).cuda())
    p["x"] *= torch.from_numpy(np.exp(rng.uniform(-3, 3, size=(n, heads, 1)))).to(DT[dtype]).cuda()
    return p


def check(p, dtype, rotary=None, paired=False, eps=1e-6, base=10000.0, layout=lambda t: t, positions=True, inplace=False):
    x, dy, w, pos = p["x"], p["dy"], p["weight"], p["positions"] if positions else None
    n, heads, d = x.shape
    rotary = d if rotary is None else rotary
    op = pkg.HeadNorm(n, heads, d, DT[dtype], rotary_dim=rotary, paired=paired, eps=eps, base=base)
    if w is not None:
        op._work.get(max(16, op.work_bytes()), torch.cuda.current_stream().cuda_stream, 0)
        op._work.tensor.fill_(0xff)            # nothing in the work buffer may be relied on
    where = np.arange(n) if pos is None else pos.cpu().numpy()
    a = ref.angles(where, rotary, base)
    xs, gs, ws = f64(x), f64(dy), np.ones(d) if w is None else f64(w)
    tol = ref.head_norm_tolerances(dtype, xs, gs, ws, a, rotary, paired, eps)
    x, dy = layout(x), layout(dy)
    dw = None if w is None else torch.full_like(w, float("nan"))
    dx = dy.clone() if inplace else layout(torch.full_like(dy, float("nan")))
    op.backward(dx if inplace else dy, x, w, dx, dw, positions=pos)
    y = x.clone() if inplace else layout(torch.full_like(x, float("nan")))
    op.forward(y if inplace else x, w, y, positions=pos)
    torch.cuda.synchronize()
    close("y", y, ref.head_norm(xs, ws, a, rotary, paired, eps)[0], tol["y"])
    want = ref.head_norm_gradients(gs, xs, ws, a, rotary, paired, eps)
    close("dx", dx, want[0], tol["dx"])
    if w is not None:
        close("dweight", dw, want[1], tol["dweight"])
    return y, dx, dw


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("paired", [False, True])
@pytest.mark.parametrize("n,heads,d,rotary", [
    (1, 1, 8, 8), (1, 16, 128, 128), (7, 3, 64, 32), (33, 2, 72, 72), (5, 6, 72, 36), (9, 1, 40, 10), (4, 5, 256, 256),
    (3, 2, 248, 246), (1000, 4, 128, 128), (257, 8, 64, 0), (130, 7, 96, 2), (2, 33, 16, 16), (5000, 6, 72, 72),
])
def test_head_norm_matches(n, heads, d, rotary, paired, dtype):
    check(problem(n, heads, d, dtype, 1 << 17, n * 7 + d), dtype, rotary, paired)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,heads,d", [(70000, 4, 128), (40001, 5, 72), (300000, 1, 8), (20011, 16, 64)])
def test_many_rows(n, heads, d, dtype):
    check(problem(n, heads, d, dtype, 1 << 20, 3), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_far_positions(dtype):
    """The farthest positions either way: angles of 2^31 turns of rate 1, in 64 bits off by 2^31 2^-53 at most."""
    p = problem(64, 2, 64, dtype, 1, 5)
    at = np.concatenate([[-2 ** 31, 2 ** 31 - 1, 0, -1], 2 ** np.arange(30), -(2 ** np.arange(30))]).astype(np.int32)
    p["positions"] = torch.from_numpy(at).cuda()
    check(p, dtype)
    check(p, dtype, base=1.0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_layouts(dtype):
    p = problem(37, 3, 64, dtype, 100, 6)
    check(p, dtype, layout=lambda t: padded(t, 8))
    check(p, dtype, layout=lambda t: t.transpose(0, 1).contiguous().transpose(0, 1))     # heads outermost
    check(p, dtype, positions=False)
    check(p, dtype, inplace=True)
    # one row for all, and one head for all
    row, head = p["x"][:1].expand(37, 3, 64), p["x"][:, :1].expand(37, 3, 64)
    for x in (row, head):
        check(dict(p, x=x), dtype)
        check(dict(p, dy=x), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_values(dtype):
    """Heads of zeros (their square root is of eps alone), a head with one value, none without a weight."""
    p = problem(6, 2, 64, dtype, 50, 8, weighted=False)
    p["x"][0] = 0
    p["x"][1, 0] = 0
    p["x"][1, 0, 5] = 3.0
    check(p, dtype, 32)
    p = problem(6, 2, 64, dtype, 50, 8)
    p["x"][3] = 0
    check(p, dtype, eps=1e-3)
    p["x"][4, 1, 7] = float("nan")
    y = torch.empty_like(p["x"])
    pkg.HeadNorm(6, 2, 64, DT[dtype]).forward(p["x"], p["weight"], y)
    bad = torch.isnan(y).any(2).cpu().numpy()
    assert bad[4, 1] and bad.sum() == 1


def test_no_rows():
    x, w = torch.empty(0, 2, 64, device="cuda"), torch.ones(64, device="cuda")
    op = pkg.HeadNorm(0, 2, 64, torch.float32)
    op.forward(x, w, x)
    dw = torch.full_like(w, 7)
    op.backward(x, x, w, x, dw)
    assert not dw.any()


def test_same_results_every_time_and_in_a_graph():
    p = problem(9001, 4, 64, "bf16", 1000, 9)
    op = pkg.HeadNorm(9001, 4, 64, torch.bfloat16)
    y, dx, dw = torch.empty_like(p["x"]), torch.empty_like(p["x"]), torch.empty_like(p["weight"])

    def call():
        op.forward(p["x"], p["weight"], y, positions=p["positions"])
        op.backward(p["dy"], p["x"], p["weight"], dx, dw, positions=p["positions"])
    call()
    first = [t.clone() for t in (y, dx, dw)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for t in (y, dx, dw):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (y, dx, dw)))


def test_gradients_against_differences():
    """Central differences in fp32 with steps of 1/64: a cubic term of about step^2 / 6 and rounding of 2^-22 64 a value."""
    p = problem(2, 2, 16, "fp32", 9, 11)
    p["x"] = torch.randn(2, 2, 16, generator=torch.Generator().manual_seed(1)).cuda() + 2.0
    op = pkg.HeadNorm(2, 2, 16, torch.float32, rotary_dim=8, eps=1e-2)
    y, dx, dw = torch.empty_like(p["x"]), torch.empty_like(p["x"]), torch.empty_like(p["weight"])
    op.backward(p["dy"], p["x"], p["weight"], dx, dw, positions=p["positions"])

    def loss():
        op.forward(p["x"], p["weight"], y, positions=p["positions"])
        return float((y.double() * p["dy"].double()).sum())
    for t, g in ((p["x"], dx), (p["weight"], dw)):
        flat, got = t.view(-1), g.reshape(-1).cpu().numpy()
        for i in range(0, flat.numel(), 3):
            keep = float(flat[i])
            flat[i] = keep + 1 / 64
            up = loss()
            flat[i] = keep - 1 / 64
            down = loss()
            flat[i] = keep
            assert abs((up - down) * 32 - got[i]) < 2e-3
