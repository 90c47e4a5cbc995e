"""Layer norm backward: whose statistics it uses."""
import numpy as np
import pytest

import reader_ref as ref
from test_gpu_reader import close, f64, norm_tolerances

pytestmark = pytest.mark.gpu

K = pytest.importorskip("compressed_graph_spmv_gb300.k2t")
import compressed_graph_spmv_gb300 as pkg  # noqa: E402

torch = pytest.importorskip("torch")
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    K.load()


SHAPES = [(300, 512, "bf16"), (40001, 64, "bf16"), (9000, 1024, "fp16"), (33, 63, "fp32"), (20011, 333, "bf16"), (2500, 3999, "fp16"),
          (16391, 517, "fp32"), (5, 8200, "bf16"), (3, 16384, "fp32"), (70, 7001, "bf16"), (1, 1, "fp32")]


def states(n, dim, dtype, residual, seed, shift):
    rng = np.random.default_rng(seed)
    mk = lambda *s, scale=1.0, shift=0.0: torch.from_numpy(rng.standard_normal(s) * scale + shift).to(DT[dtype]).cuda()  # noqa: E731
    x = dict(x=mk(n, dim, scale=1 + shift, shift=shift), r=mk(n, dim) if residual else None, dy=mk(n, dim),
             dz=mk(n, dim) if residual else None)
    x["y"], x["dx"] = (torch.full_like(x["x"], float("nan")) for _ in range(2))
    x["z"] = torch.full_like(x["x"], float("nan")) if residual else None
    x["dw"], x["db"] = (torch.full((dim,), float("nan"), dtype=DT[dtype], device="cuda") for _ in range(2))
    return x


def check_gradients(s, w, dtype):
    z = f64(s["x"] if s["z"] is None else s["z"])
    y, _, _, rstd, xh = ref.norm(z, f64(w), None, 1e-5)
    dz = None if s["dz"] is None else f64(s["dz"])
    dx, dw, db = ref.norm_gradients(f64(s["dy"]), xh, rstd, f64(w), dz)
    tol = norm_tolerances(dtype, f64(s["x"]), z, xh, rstd, f64(w), np.zeros_like(f64(w)), f64(s["dy"]), dz, y, dx, dw, db)
    for name, want in (("dx", dx), ("dw", dw), ("db", db)):
        close(name, s[name], want, tol[name])


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("n,dim,dtype", SHAPES)
def test_two_forward_calls_before_their_backward_calls(n, dim, dtype, residual, given):
    """Micro-batches, a layer used twice, recomputation: each backward call is of the states it is given."""
    op = pkg.LayerNorm(n, dim, DT[dtype], residual=residual, eps=1e-5)
    w = torch.from_numpy(np.random.default_rng(1).standard_normal(dim) + 1).to(DT[dtype]).cuda()
    both = [states(n, dim, dtype, residual, 2, 0.0), states(n, dim, dtype, residual, 3, 3.0)]
    for s in both:
        s["st"] = dict(mean=torch.empty(n, device="cuda"), rstd=torch.empty(n, device="cuda")) if given else {}
        op.forward(s["x"], w, None, s["y"], residual=s["r"], z=s["z"], **s["st"])
    for s in both:
        op.backward(s["dy"], s["x"] if s["z"] is None else s["z"], w, s["dx"], s["dw"], s["db"], dz=s["dz"], **s["st"])
    for s in both:
        check_gradients(s, w, dtype)


@pytest.mark.parametrize("n,dim,dtype", SHAPES)
def test_backward_without_a_forward_call(n, dim, dtype):
    op = pkg.LayerNorm(n, dim, DT[dtype])
    op.mean.fill_(float("nan"))
    op.rstd.fill_(float("nan"))
    w = torch.ones(dim, dtype=DT[dtype], device="cuda")
    s = states(n, dim, dtype, False, 4, 1.0)
    op.backward(s["dy"], s["x"], w, s["dx"], s["dw"], s["db"])
    check_gradients(s, w, dtype)


def test_statistics_come_in_pairs():
    op = pkg.LayerNorm(4, 8, torch.float32)
    x, w = torch.zeros(4, 8, device="cuda"), torch.ones(8, device="cuda")
    one = torch.zeros(4, device="cuda")
    for kw in (dict(mean=one), dict(rstd=one)):
        with pytest.raises(ValueError):
            op.forward(x, w, None, x.clone(), **kw)
        with pytest.raises(ValueError):
            op.backward(x, x, w, x.clone(), w.clone(), **kw)
    with pytest.raises(ValueError):
        op.backward(x, x, w, x.clone(), w.clone(), mean=one[:3], rstd=one)
