"""Attention over the 8-bit cache where scores are so large that fp32 does not hold a value block's exponent beside them:
soft masks of -1e9, large scales.

Scores are all equal, or differ by far more than what weights reach, so that weights are exactly alike or none whatever
the size of the scores: outputs are off by rounding alone (weights u, as tests/reader_ref.py has it), and lse by at most seven
roundings of 2^-24 of it (scale, log2(e), their product, the score, the sum with the logarithm, ln(2), the product with it).
"""
import numpy as np
import pytest

import reader_ref as ref
from test_gpu_cache import ask, cached
from test_gpu_reader import DT, close, dev, f64

pytestmark = pytest.mark.gpu

K = pytest.importorskip("compressed_graph_spmv_gb300.k2t")
import compressed_graph_spmv_gb300 as pkg  # noqa: E402

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    K.load()


SHAPES = [(1, 1), (1, 4), (2, 4), (9, 1), (20, 2), (40, 1), (64, 2), (150, 1)]     # queries, heads that share keys


def problem(T, G, n, d, dtype, seed, hkv=2, sources=0, reach=15):
    """Values whose blocks differ by 2^(2 reach) in size, and queries and keys that are one constant product."""
    rng = np.random.default_rng(seed)
    p = dict(q=torch.zeros(T, hkv * G, d, dtype=DT[dtype], device="cuda"), k=torch.zeros(n, hkv, d, dtype=DT[dtype], device="cuda"),
             v=dev(rng, dtype, n, hkv, d), hops=None, bias=None, edges=None, source=None)
    size = torch.from_numpy(2.0 ** rng.integers(-reach, reach + 1 if dtype == "bf16" else 3, size=(n // 32 + 1, hkv, 1))).repeat_interleave(32, 0)[:n].cuda()
    p["v"] = (p["v"].double() * size).to(DT[dtype])
    p["q"][..., 0], p["k"][..., 0] = 2, 0.5
    if sources:
        p["hops"] = torch.zeros(n, sources, dtype=torch.int32, device="cuda")
        p["source"] = torch.from_numpy(rng.integers(0, sources, size=T).astype(np.int32)).cuda()
    return p


def check(p, dtype, scale, levels=None):
    """levels: bias of each node and column; of a query those of its column, and only the nodes of the highest weigh anything."""
    cache, held = cached(p, dtype)
    out, lse = ask(p, dtype, cache, scale=scale)
    T, hq, d = p["q"].shape
    n, hkv = p["k"].shape[:2]
    v, u = np.repeat(held["v"], hq // hkv, axis=1), ref.U[dtype]
    want, size, wlse = np.zeros((T, hq, d)), np.zeros((T, hq, d)), np.zeros((T, hq))
    for t in range(T):
        level = np.zeros(n) if levels is None else levels[:, 0 if p["source"] is None else int(p["source"][t])]
        top = level == level.max()
        want[t], size[t] = v[top].mean(axis=0), np.abs(v[top]).mean(axis=0)
        wlse[t] = scale + level.max() + np.log(top.sum())
    tol = u * np.abs(want) + (u + 2.0 ** -18) * size + (2.0 ** -25 if dtype == "fp16" else 0.0)
    close("out", out, want, tol)
    close("lse", lse, wlse, 7 * 2.0 ** -24 * np.abs(wlse) + 1e-5)


@pytest.mark.parametrize("scale", [1e9, -1e9, 3e7, 2e6, 2.0 ** 22, -(2.0 ** 23), 1e20, -3e37])
@pytest.mark.parametrize("T,G", SHAPES)
def test_equal_scores_of_any_size(T, G, scale):
    for dtype, n, reach in (("bf16", 45, 15), ("bf16", 3000, 15), ("bf16", 3000, 45), ("fp16", 1001, 15)):
        check(problem(T, G, n, 40, dtype, T + n, reach=reach), dtype, scale)


@pytest.mark.parametrize("T,G", SHAPES)
@pytest.mark.parametrize("hkv", [2, 76])
def test_soft_masks(T, G, hkv):
    """Columns of which all nodes are at -1e9, or some, first or last or between, the others at 0, -2e9 or 3e8; with many heads
    a block has many tiles."""
    n, sources = 1500, 7
    table = [0.0, -1e9, -2e9, 3e8, -5e6]
    p = problem(T, G, n, 24, "bf16", T, hkv, sources)
    h = p["hops"]
    h[:, 0] = 1
    h[:, 1] = 1
    h[700:, 1] = 0
    h[:, 2] = 0
    h[600:, 2] = 1
    h[:, 3] = 2
    h[800:900, 3] = 1
    h[:, 4] = torch.from_numpy(np.random.default_rng(T).integers(0, 5, size=n).astype(np.int32)).cuda()
    h[:, 5] = 4
    h[:20, 5] = 1
    h[:, 6] = 1
    h[1490:, 6] = 4
    p["edges"] = list(range(5))
    p["bias"] = torch.tensor(table, device="cuda").bfloat16().expand(hkv * G, 5).contiguous()
    check(p, "bf16", 1.0, f64(p["bias"])[0][h.cpu().numpy()])


@pytest.mark.parametrize("T,G", SHAPES)
def test_as_over_16_bits(T, G):
    """Random queries, and a soft mask on all that a row sees: what the score's rounding leaves of it weighs as it does over the
    states read back.  Scores of 1.4e9 are multiples of 128 there, so that both have the same highest ones; weights are
    exactly alike or none."""
    rng = np.random.default_rng(T)
    n, hkv, d = 900, 2, 64
    p = problem(T, G, n, d, "bf16", T, hkv, 3)
    p["q"], p["k"] = dev(rng, "bf16", T, hkv * G, d), dev(rng, "bf16", n, hkv, d)
    p["edges"], p["bias"] = [0], torch.full((hkv * G, 1), -1e9, device="cuda").bfloat16()
    cache, held = cached(p, "bf16")
    out, lse = ask(p, "bf16", cache)
    k, v = (torch.from_numpy(held[s]).bfloat16().cuda() for s in "kv")
    op = pkg.HopAttention(T, n, hkv * G, hkv, d, torch.bfloat16, sources=3, edges=p["edges"])
    o, l = torch.empty_like(out), torch.empty_like(lse)
    op.forward(p["q"], k, v, o, l, hops=p["hops"], bias=p["bias"], query_source=p["source"])
    mean = np.repeat(held["v"].mean(axis=0), G, axis=0)[None]
    size = np.repeat(np.abs(held["v"]).mean(axis=0), G, axis=0)[None]
    u = ref.U["bf16"]
    for got in (o, out):          # every score is the bias: 64 values of a few units each times 1/8 are below half of 128
        close("out", got, np.broadcast_to(mean, got.shape), np.broadcast_to(u * np.abs(mean) + (u + 2.0 ** -18) * size, got.shape))
    assert torch.equal(lse, l)


@pytest.mark.parametrize("order", ["rising", "falling", "shuffled"])
@pytest.mark.parametrize("T,G", SHAPES)
def test_levels_that_change(T, G, order):
    """Runs of nodes at one of ten levels after another, so that a row's origin moves many times in a block of many tiles; runs end
    inside tiles, and a column sees some of them alone."""
    rng = np.random.default_rng(T * 3 + G)
    n, hkv, sources = 5000, 152 if T < 9 else 40, 4
    p = problem(T, G, n, 8, "bf16", T, hkv, sources)
    table = np.array([-3e9, -2e9, -1.01e9, -1e9, -6e6, 0.0, 4.0, 9e6, 3e8, 2e9])
    for c in range(sources):
        level = np.sort(rng.permutation(10)[:10 - c])
        level = {"rising": level, "falling": level[::-1], "shuffled": rng.permutation(level)}[order]
        ends = np.sort(rng.choice(np.arange(1, n), size=len(level) - 1, replace=False))
        column = np.repeat(level, np.diff(np.concatenate([[0], ends, [n]])))
        p["hops"][:, c] = torch.from_numpy(column.astype(np.int32)).cuda()
    p["edges"] = list(range(10))
    p["bias"] = torch.from_numpy(table).cuda().bfloat16().expand(hkv * G, 10).contiguous()
    levels = f64(p["bias"])[0][p["hops"].cpu().numpy()]
    top = levels.max(axis=0)
    for c in range(sources):          # 0 and 4 together are no test of levels alone
        if top[c] == 4.0:
            p["hops"][:, c][p["hops"][:, c] == 5] = -1
    levels = np.where(p["hops"].cpu().numpy() < 0, -np.inf, f64(p["bias"])[0][np.maximum(p["hops"].cpu().numpy(), 0)])
    check(p, "bf16", 1.0, levels)
