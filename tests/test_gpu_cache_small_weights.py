"""Attention over the 8-bit cache where one node outweighs each of very many others, which together still count: no weight is
rounded away that the header does not name."""
import numpy as np
import pytest

import reader_ref as ref
from test_gpu_reader import DT, close

pytestmark = pytest.mark.gpu

K = pytest.importorskip("compressed_graph_spmv_gb300.k2t")
import compressed_graph_spmv_gb300 as pkg  # noqa: E402

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    K.load()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,G", [(1, 1), (2, 4), (9, 1), (20, 2), (70, 2)])
@pytest.mark.parametrize("x", [12.0, 15.0, 16.0, 16.5, 17.0, 17.5, 18.0])
def test_one_node_beside_very_many(x, T, G, dtype):
    """Weight e^x of one node, whose value is -1, beside 2^19 of weight 1 and value 1: 3 to 0.008 times its weight.  With 152
    heads one block takes all nodes of a head, so that all weights are against the one node's.

    out <= u |out| + u (weights) + 2^-18 (sums) + the part of the others times u, and for each of them 2^-29 of the largest weight
    (2^-31 in fp16 or with more than 8 rows), which is the weight e^x: at most 2^-10 (2^-12) of the sum.
    """
    n, hkv, d = 1 << 19, 152, 8
    q = torch.zeros(T, G * hkv, d, device="cuda", dtype=DT[dtype])
    k = torch.zeros(n, hkv, d, device="cuda", dtype=DT[dtype])
    v = torch.ones(n, hkv, d, device="cuda", dtype=DT[dtype])
    at = 7777
    q[..., 0], k[at, :, 0], v[at] = 1, 16, -1                       # e4m3 holds 16
    cache = pkg.NodeCache(n, hkv, d, DT[dtype])
    cache.write(k, v)
    out, lse = torch.empty_like(q), torch.empty(T, G * hkv, device="cuda")
    pkg.CachedAttention(T, n, G * hkv, hkv, d, DT[dtype], scale=x / 16).forward(q, cache, out, lse)
    total = np.exp(x) + n - 1
    want, u = (n - 1 - np.exp(x)) / total, ref.U[dtype]
    least = 2.0 ** -29 if dtype == "bf16" and T * G <= 8 else 2.0 ** -31
    tol = u * abs(want) + u + 2.0 ** -18 + n * least * np.exp(x) / total
    close("out", out, np.full((T, G * hkv, d), want), np.full((T, G * hkv, d), tol))
    close("lse", lse, np.full((T, G * hkv), np.log(total)), np.full((T, G * hkv), 2e-5))
