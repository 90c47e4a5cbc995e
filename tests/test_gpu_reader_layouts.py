"""Attention of tensors in other orders than rows of heads: the same values as of contiguous ones, and nothing written beside
them."""
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


def head_major(t, fill=None):
    """The values of t (or `fill`) with heads outermost, three rows apart at each end of a head, and the whole storage."""
    n, h, d = t.shape
    store = torch.full((h, n + 6, d + 8), 7.0 if fill is not None else float("nan"), dtype=t.dtype, device=t.device)
    view = store[:, 3:3 + n, :d].permute(1, 0, 2)
    view.copy_(t if fill is None else torch.full_like(t, fill))
    return view, store


def both(x, table, T, n, hq, hkv, d, out, grads):
    op = pkg.HopAttention(T, n, hq, hkv, d, x["q"].dtype, sources=table["hops"].shape[1], edges=[0, 1, 3, 5])
    lse, db = torch.empty(T, hq, device="cuda"), torch.empty_like(table["bias"])
    op.forward(x["q"], x["k"], x["v"], out, lse, **table)
    op.backward(x["dout"], x["q"], x["k"], x["v"], out, lse, *grads, dbias=db, **table)
    assert op.status() == 0
    return dict(out=out, lse=lse, dq=grads[0], dk=grads[1], dv=grads[2], dbias=db)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,n,hq,hkv,d", [(6, 150, 4, 2, 72), (6, 1, 4, 4, 64), (1, 700, 2, 2, 128), (90, 333, 4, 2, 64), (130, 200, 3, 3, 128)])
def test_heads_outermost(T, n, hq, hkv, d, dtype):
    g = torch.Generator(device="cuda").manual_seed(T + n)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    x = dict(q=rand(T, hq, d), k=rand(n, hkv, d), v=rand(n, hkv, d), dout=rand(T, hq, d))
    table = dict(hops=torch.randint(-1, 8, (n, 6), generator=g, device="cuda", dtype=torch.int32), bias=rand(hq, 4),
                 query_source=torch.randint(-1, 6, (T,), generator=g, device="cuda", dtype=torch.int32))
    want = both(x, table, T, n, hq, hkv, d, torch.empty_like(x["q"]), [torch.empty_like(x[y]) for y in "qkv"])
    moved = {y: head_major(t)[0] for y, t in x.items()}
    made = {y: head_major(x[z], fill=7.0) for y, z in (("out", "q"), ("dq", "q"), ("dk", "k"), ("dv", "v"))}
    got = both(moved, table, T, n, hq, hkv, d, made["out"][0], [made[y][0] for y in ("dq", "dk", "dv")])
    for y in want:
        assert torch.equal(want[y], got[y]), y
    for y, (view, store) in made.items():
        view.fill_(7.0)
        assert (store == 7).all(), y


@pytest.mark.parametrize("T", [6, 90])
def test_broadcast_inputs(T):
    """One head's states for all, one query for all: gradients are of each place."""
    n, hq, hkv, d = 300, 4, 2, 64
    g = torch.Generator(device="cuda").manual_seed(T)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    x = dict(q=rand(1, hq, d).expand(T, hq, d), k=rand(n, 1, d).expand(n, hkv, d), v=rand(1, hkv, d).expand(n, hkv, d),
             dout=rand(1, 1, d).expand(T, hq, d))
    table = dict(hops=torch.randint(-1, 8, (n, 6), generator=g, device="cuda", dtype=torch.int32), bias=rand(hq, 4),
                 query_source=torch.randint(-1, 6, (T,), generator=g, device="cuda", dtype=torch.int32))
    new = lambda y: torch.empty(x[y].shape, dtype=x[y].dtype, device="cuda")  # noqa: E731
    got = both(x, table, T, n, hq, hkv, d, new("q"), [new(y) for y in "qkv"])
    want = both({y: t.contiguous() for y, t in x.items()}, table, T, n, hq, hkv, d, new("q"), [new(y) for y in "qkv"])
    for y in want:
        assert torch.equal(want[y], got[y]), y
