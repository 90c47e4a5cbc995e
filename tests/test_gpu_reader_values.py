"""Attention of values at the edges of their types."""
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


@pytest.mark.parametrize("T,hkv", [(1, 1), (128, 152), (40, 2), (150, 76)])
def test_half_weights_below_the_least_number(T, hkv):
    """2^20 nodes of relative weight 1.4 2^-24 each beside one of weight 1: together a twelfth of a row.  Scores are the
    bias alone (q is 0).  Every value is v = 1 but the one node's, 0, so that out is that share.  Weights times 2^7 are
    rounded to steps of 2^-24, 1/179 of each: off by 2^-8.5 at most, and the result by 2^-11."""
    n, d = 1 << 20, 32
    low = torch.tensor(-16.3, dtype=torch.float16)
    k = torch.zeros(1, 1, d, dtype=torch.float16, device="cuda").expand(n, hkv, d)
    v = torch.ones(n, 1, d, dtype=torch.float16, device="cuda")
    v[n // 2] = 0
    hops = torch.ones(n, 1, dtype=torch.int32, device="cuda")
    hops[n // 2] = 0
    q, out = (torch.zeros(T, hkv, d, dtype=torch.float16, device="cuda") for _ in range(2))
    lse = torch.zeros(T, hkv, device="cuda")
    bias = torch.tensor([0.0, float(low)], dtype=torch.float16, device="cuda").expand(hkv, 2).contiguous()
    op = pkg.HopAttention(T, n, hkv, hkv, d, torch.float16, sources=1, edges=[0, 1])
    op.forward(q, k, v.expand(n, hkv, d), out, lse, hops=hops, bias=bias, query_source=torch.zeros(T, dtype=torch.int32, device="cuda"))
    rest = (n - 1) * torch.exp(low.double())
    want = float(rest / (1 + rest))
    assert abs(out.double() - want).max() <= want * (2.0 ** -8.5 + 2.0 ** -11)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,hkv", [(128, 152), (40, 160), (150, 76), (1, 200)])
def test_sum_of_weights_over_very_many_nodes(T, hkv, dtype):
    """2^20 nodes of relative weight 2^-23.5 each beside one of weight 1, all of them one block's: their sum is not lost
    beside the one.  Scores are the bias alone."""
    n, d = 1 << 20, 32
    low = torch.tensor(-16.3, dtype=dtype)
    states = torch.ones(n, 1, d, dtype=dtype, device="cuda").expand(n, hkv, d)
    hops = torch.ones(n, 1, dtype=torch.int32, device="cuda")
    hops[0] = 0
    q, out = (torch.zeros(T, hkv, d, dtype=dtype, device="cuda") for _ in range(2))
    lse = torch.zeros(T, hkv, device="cuda")
    bias = torch.tensor([0.0, float(low)], dtype=dtype, device="cuda").expand(hkv, 2).contiguous()
    op = pkg.HopAttention(T, n, hkv, hkv, d, dtype, sources=1, edges=[0, 1])
    table = dict(hops=hops, bias=bias, query_source=torch.zeros(T, dtype=torch.int32, device="cuda"))
    op.forward(q, states, states, out, lse, **table)
    rest = (n - 1) * torch.exp(low.double())
    assert abs(lse.double() - float(torch.log1p(rest))).max() <= 1e-5


@pytest.mark.parametrize("n,hkv", [(70, 2), (5000, 1)])
@pytest.mark.parametrize("T", [3, 40, 140])
@pytest.mark.parametrize("what", ["nan", "inf"])
def test_rows_that_hold_no_number(T, n, hkv, what):
    """A query that is NaN, or whose scores overflow, says so in out and lse: -inf means that nothing was seen."""
    g = torch.Generator(device="cuda").manual_seed(T + n)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, k, v = rand(T, hkv, 64), rand(n, hkv, 64), rand(n, hkv, 64)
    op = pkg.HopAttention(T, n, hkv, hkv, 64, torch.bfloat16)
    out, lse = torch.zeros_like(q), torch.zeros(T, hkv, device="cuda")
    op.forward(q, k, v, out, lse)
    good, good_lse = out.clone(), lse.clone()
    q[1] = float("nan") if what == "nan" else 3e38
    op.forward(q, k, v, out, lse)
    others = [t for t in range(T) if t != 1]
    assert torch.equal(out[others], good[others]) and torch.equal(lse[others], good_lse[others])
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
