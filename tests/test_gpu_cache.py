"""The 8-bit node cache on the GPU against 64-bit references (tests/cache_ref.py: values and scales exactly), and
attention over it within the bounds of tests/reader_ref.py."""
import numpy as np
import pytest

import cache_ref
import reader_ref as ref
from test_gpu_reader import DT, close, dev, f64, padded, problem, ref_table

pytestmark = pytest.mark.gpu

K = pytest.importorskip("compressed_graph_spmv_gb300.k2t")
import compressed_graph_spmv_gb300 as pkg  # noqa: E402

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    K.load()


def states(rng, dtype, n, heads, d):
    size = np.exp(rng.uniform(-6, 6, size=(n, heads, 1)))
    return torch.from_numpy(rng.standard_normal((n, heads, d)) * size).to(DT[dtype]).cuda()


class Both:
    """A cache and its reference, written together."""

    def __init__(self, n, heads, d, dtype):
        self.cache, self.n, self.shape, self.dtype = pkg.NodeCache(n, heads, d, DT[dtype]), n, (heads, d), dtype
        self.k, self.v = cache_ref.Cache(n, heads, d), cache_ref.Cache(n, heads, d)

    def write(self, k, v, first=0):
        self.cache.write(k, v, first=first)
        self.k.write(f64(k), first)
        self.v.write(f64(v), first)

    def back(self, dtype="fp32", first=0, count=None, nodes=None):
        """What is read, in a type that holds it."""
        count = nodes.shape[0] if nodes is not None else self.n - first if count is None else count
        reader = self.cache
        if dtype != self.dtype:
            reader = pkg.NodeCache(self.n, *self.shape, DT[dtype])
            for a, b in ((reader.k, self.cache.k), (reader.v, self.cache.v)):
                a.view(torch.uint8).copy_(b.view(torch.uint8))
            reader.k_scale.copy_(self.cache.k_scale), reader.v_scale.copy_(self.cache.v_scale)
        k, v = (torch.full((count, *self.shape), float("nan"), dtype=DT[dtype], device="cuda") for _ in range(2))
        reader.read(k, v, first=first, nodes=nodes)
        return f64(k), f64(v)

    def check(self):
        blocks = -(-self.n // 32)
        for got, want, scale in zip(self.back(), (self.k, self.v), (self.cache.k_scale, self.cache.v_scale)):
            np.testing.assert_array_equal(scale[:, :blocks].cpu().numpy().astype(int) - 64, want.e.T)
            np.testing.assert_array_equal(got, want.read())


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n,heads,d", [(1, 1, 8), (32, 2, 64), (33, 3, 72), (100, 4, 128), (1000, 1, 40), (31, 2, 120), (4097, 2, 16)])
def test_whole(n, heads, d, dtype):
    rng = np.random.default_rng(n + d)
    b = Both(n, heads, d, dtype)
    b.check()                                     # a new cache holds zeros
    b.write(states(rng, dtype, n, heads, d), states(rng, dtype, n, heads, d))
    b.check()
    b.write(*(t * 2.0 ** -9 for t in (states(rng, dtype, n, heads, d), states(rng, dtype, n, heads, d))))
    b.check()                                     # scales of whole blocks shrink again


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_parts(dtype):
    """Runs of nodes that begin and end inside blocks, larger and smaller than what stays."""
    rng = np.random.default_rng(5)
    n, heads, d = 203, 2, 72
    b = Both(n, heads, d, dtype)
    for first, count, size in ((0, 5, 1), (5, 1, 30), (6, 40, 0.01), (200, 3, 5), (195, 5, 1e-3), (31, 2, 1e4), (0, 203, 1), (64, 32, 1e-4),
                               (70, 1, 1e-3), (96, 107, 2), (128, 70, 1), (202, 1, 100), (10, 0, 1), (203, 0, 1)):
        k, v = (dev(rng, dtype, count, heads, d, scale=s) for s in (size, 1 / size))
        b.write(k, v, first)
        b.check()


def test_one_node_at_a_time():
    rng = np.random.default_rng(6)
    b = Both(70, 1, 24, "bf16")
    for i in range(70):
        b.write(states(rng, "bf16", 1, 1, 24), states(rng, "bf16", 1, 1, 24), i)
    b.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_values(dtype):
    """Every rounding border, the ends of the range, zeros, infinities and NaN."""
    e4m3 = np.unique(np.abs(cache_ref.to_e4m3(np.concatenate([np.arange(0, 2, 2.0 ** -9), np.arange(2, 449, 2.0 ** -3)]))))
    border = (e4m3[1:] + e4m3[:-1]) / 2
    x = np.concatenate([e4m3, border, np.nextafter(border.astype(np.float32), np.float32(0)).astype(np.float64)])
    x = np.concatenate([x, -x, np.zeros(-2 * x.size % 64)]).reshape(-1, 1, 8)
    n = x.shape[0]
    x[:, 0, 0] = 448                                # every block at scale 1
    for up in (0, -3, 5):
        k = torch.from_numpy(x * 2.0 ** up).to(DT[dtype]).cuda()
        b = Both(n, 1, 8, dtype)
        b.write(k, -k)
        b.check()
    rng = np.random.default_rng(7)
    odd = states(rng, dtype, 96, 2, 32)
    odd[3, 0, 4], odd[4, 0, 5], odd[40, 1, 0] = float("inf"), float("nan"), -float("inf")
    odd[64:, 0] = 0
    odd[64:, 1] = float("nan")
    if dtype != "fp16":
        odd[33, 0] = 2.0 ** 75                      # above the largest scale's reach
        odd[34, 0, 1] = -(2.0 ** 100)
        odd[0, 1] = 2.0 ** -75
    b = Both(96, 2, 32, dtype)
    b.write(odd, odd)
    b.check()
    tiny = torch.full((32, 1, 8), 2.0 ** -74 if dtype != "fp16" else 2.0 ** -24, dtype=DT[dtype], device="cuda")
    tiny[0] *= 1.5
    b = Both(32, 1, 8, dtype)
    b.write(tiny, -tiny)
    b.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_read(dtype):
    rng = np.random.default_rng(8)
    n, heads, d = 300, 3, 40
    b = Both(n, heads, d, dtype)
    b.write(dev(rng, dtype, n, heads, d), dev(rng, dtype, n, heads, d))
    want = b.k.read(), b.v.read()
    for first, count in ((0, n), (7, 100), (299, 1), (300, 0)):
        for got, w in zip(b.back(dtype, first, count), want):
            np.testing.assert_array_equal(got, w[first:first + count])
    nodes = np.concatenate([rng.integers(0, n, size=50), [5, 5, -1, n, 2 ** 31 - 1, -2 ** 31, 299, 0]]).astype(np.int32)
    for got, w in zip(b.back(dtype, nodes=torch.from_numpy(nodes).cuda()), want):
        inside = (nodes >= 0) & (nodes < n)
        np.testing.assert_array_equal(got, np.where(inside[:, None, None], w[np.where(inside, nodes, 0)], 0.0))


def test_layouts():
    rng = np.random.default_rng(9)
    k, v = dev(rng, "bf16", 45, 2, 24), dev(rng, "bf16", 45, 2, 24)
    for lay in (lambda t: padded(t, 8), lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)):
        b = Both(50, 2, 24, "bf16")
        b.write(lay(k), lay(v), 3)
        b.check()
        out = lay(torch.full((45, 2, 24), float("nan"), device="cuda", dtype=torch.bfloat16)), lay(torch.zeros_like(k))
        b.cache.read(*out, first=3)
        np.testing.assert_array_equal(f64(out[0]), b.k.read()[3:48])
        np.testing.assert_array_equal(f64(out[1]), b.v.read()[3:48])
    b = Both(50, 2, 24, "bf16")
    b.write(k[:1].expand(50, 2, 24), v[:1, :1].expand(50, 2, 24))        # one state for all nodes
    b.check()


# ---- attention -------------------------------------------------------------------

def cached(p, dtype, capacity=None):
    """A cache of the problem's states, and the values that it holds in their place."""
    n, hkv, d = p["k"].shape
    b = Both(capacity or n, hkv, d, dtype)
    b.write(p["k"], p["v"])
    return b.cache, dict(p, k=b.k.read()[:n], v=b.v.read()[:n])


def ask(p, dtype, cache, scale=None, nodes=None, poison=True):
    T, hq, d = p["q"].shape
    op = pkg.CachedAttention(T, cache.n_nodes if p["hops"] is None else p["hops"].shape[0], hq, cache.n_kv_heads, d, DT[dtype],
                             sources=0 if p["hops"] is None else p["hops"].shape[1], edges=p["edges"], scale=scale)
    out = torch.full_like(p["q"].contiguous(), float("nan"))
    lse = torch.full((T, hq), float("nan"), device="cuda")
    if poison:
        op._work_of(0)
        op._work[0].fill_(0xff)
        op._work[0][:4].zero_()
    op.forward(p["q"], cache, out, lse, hops=p["hops"], bias=p["bias"], query_source=p["source"], nodes=nodes)
    torch.cuda.synchronize()
    assert op.status() == 0
    return out, lse


def check(p, dtype, got, scale=None):
    q, k, v = f64(p["q"]), p["k"], p["v"]
    d = q.shape[2]
    scale = d ** -0.5 if scale is None else scale
    if p["hops"] is not None:   # states that no query sees do not count
        hops = p["hops"].cpu().numpy()
        cols = list(range(q.shape[0])) if p["source"] is None else p["source"].cpu().tolist()
        used = [c for c in cols if 0 <= c < hops.shape[1]]
        if len(used) == len(cols):
            hidden = (hops[:, used] < 0).all(axis=1) if used else np.ones(k.shape[0], bool)
            k[hidden] = 0
            v[hidden] = 0
    want = ref.attention(q, k, v, scale, **ref_table(p, dtype))
    tol = ref.attention_tolerances(q, k, v, scale, dtype, bias=None if p["bias"] is None else f64(p["bias"]), ref=want)
    close("out", got[0], want[0], tol["out"])
    close("lse", got[1], want[1], tol["lse"])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,n,hq,hkv,d,sources,buckets,mapped", [
    (1, 1, 1, 1, 64, 1, 4, False), (1, 63, 8, 8, 64, 1, 16, False), (1, 1000, 16, 4, 128, 1, 32, False),
    (2, 64, 2, 1, 8, 2, 1, False), (5, 65, 3, 3, 40, 5, 2, False), (13, 777, 6, 2, 72, 13, 11, False),
    (32, 515, 4, 4, 128, 32, 64, False), (32, 300, 8, 2, 64, 32, 7, False), (17, 129, 4, 4, 96, 3, 5, True),
    (70, 200, 4, 1, 64, 32, 32, True), (131, 321, 2, 2, 128, 7, 3, True), (9, 200, 3, 1, 128, 9, 0, False),
    (8, 100, 4, 4, 32, 0, 0, False), (33, 130, 16, 1, 64, 0, 0, False), (300, 2, 4, 2, 40, 17, 15, True),
    (64, 1025, 2, 2, 128, 0, 0, False), (129, 640, 3, 1, 128, 30, 20, True), (260, 300, 1, 1, 24, 0, 0, False),
])
def test_attention_matches(T, n, hq, hkv, d, sources, buckets, mapped, dtype):
    p = problem(T, n, hq, hkv, d, sources, buckets, dtype, mapped, seed=T * 1000 + n)
    cache, held = cached(p, dtype)
    check(held, dtype, ask(p, dtype, cache))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,hq,hkv,d", [(1, 4, 4, 64), (20, 4, 1, 64), (4, 4, 1, 40), (7, 1, 1, 128), (30, 1, 1, 64), (2, 2, 2, 128), (32, 4, 2, 128), (150, 2, 1, 72)])
def test_many_nodes(T, hq, hkv, d, dtype):
    p = problem(T, 6001, hq, hkv, d, min(T, 32), 9, dtype, T > 32, seed=T + d)
    cache, held = cached(p, dtype)
    check(held, dtype, ask(p, dtype, cache))


@pytest.mark.parametrize("order", ["rising", "falling", "shuffled"])
@pytest.mark.parametrize("T,G", [(1, 3), (2, 4), (3, 5), (20, 1), (16, 4), (130, 1)])
def test_scores_that_rise(T, G, order):
    """A row's largest score grows by some 2^10 in the weights from tile to tile, in others it falls: each block has many tiles."""
    rng = np.random.default_rng(T)
    n, hkv, d = 2900, 40, 32
    p = problem(T, n, hkv * G, hkv, d, min(T, 32), 4, "fp16", T > 32, seed=T + G, reach=0.9)
    rise = np.arange(n) / 128.0 * 7.0
    rise = {"rising": rise, "falling": rise[::-1].copy(), "shuffled": rng.permutation(rise)}[order]
    p["q"] *= 0.1
    p["q"][:, :, 0] = torch.from_numpy(rng.choice([-1.0, 0.25, 1.0], size=(T, hkv * G))).cuda()
    p["k"][:, :, 0] = torch.from_numpy(rise)[:, None].cuda()
    cache, held = cached(p, "fp16")
    check(held, "fp16", ask(p, "fp16", cache, scale=1.0), scale=1.0)


@pytest.mark.parametrize("T,G,d,sources", [(1, 4, 16, 1), (2, 3, 72, 2), (5, 4, 16, 5), (16, 1, 16, 16), (33, 2, 16, 7), (5, 4, 72, 0), (70, 1, 72, 31)])
def test_many_tiles_a_block(T, G, d, sources):
    """Some 80 tiles for each block, so that every slot and buffer goes round many times, and calls of it at once."""
    hkv = 76 if T < 30 else 19
    n = 20000 if T < 30 else 60000 // G
    p = problem(T, n, hkv * G, hkv, d, sources, 6 if sources else 0, "bf16", sources not in (0, T), seed=T + d)
    cache, held = cached(p, "bf16")
    out = ask(p, "bf16", cache)
    check(held, "bf16", out)
    again = ask(p, "bf16", cache)
    assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T", [1, 20, 40, 140])
def test_blocks_of_very_different_size(T, dtype):
    """Keys and values whose blocks differ by 2^24 in size, and queries whose values do."""
    rng = np.random.default_rng(T)
    p = problem(T, 700, 2, 1, 64, 0, 0, dtype, False, seed=T)
    size = torch.from_numpy(2.0 ** rng.integers(-12, 3, size=(700 // 32 + 1, 1, 1))).repeat_interleave(32, 0)[:700].cuda()
    p["k"] = (p["k"].double() * size).to(DT[dtype])
    p["v"] = (p["v"].double() * size.flip(0)).to(DT[dtype])
    p["q"] = (p["q"].double() * torch.from_numpy(2.0 ** rng.integers(-10, 2, size=(T, 2, 64))).cuda()).to(DT[dtype])
    cache, held = cached(p, dtype)
    check(held, dtype, ask(p, dtype, cache))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T", [1, 40, 140])
def test_masks(T, dtype):
    """Nodes that nobody sees may hold anything; a query that sees nothing; buckets masked by the table."""
    p = problem(T, 300, 4, 2, 64, min(T, 32), 5, dtype, T > 32, seed=3 * T)
    p["hops"][50:90] = -1
    if T <= 32:
        p["hops"][:, 0] = -1
    else:
        p["source"][3] = 7
        p["hops"][:, 7] = -1
        p["source"][p["source"] < 0] = 0            # no query without hop information
    p["bias"][1, 2] = -float("inf")
    p["bias"][2, 1] = torch.finfo(DT[dtype]).min
    p["bias"][3] = -float("inf")
    p["k"][50:90] = float("nan")
    p["v"][50:90] = float("inf")
    cache, held = cached(p, dtype)
    held["k"][50:90] = held["v"][50:90] = 0
    out, lse = ask(p, dtype, cache)
    check(held, dtype, (out, lse))
    row = 0 if T <= 32 else 3
    assert not out[row].any() and torch.isneginf(lse[row]).all()


def test_a_filling_cache():
    """Fewer nodes than the cache has: what lies behind them (NaN here) is not used."""
    n, hkv, d = 500, 2, 64
    p = problem(3, n, 4, hkv, d, 3, 6, "bf16", False, seed=12)
    cache = Both(n, hkv, d, "bf16")
    cache.write(torch.full_like(p["k"], float("nan")), torch.full_like(p["v"], float("nan")))
    at = 0
    for count in (0, 1, 30, 2, 100, 250):
        if count:
            cache.write(p["k"][at:at + count], p["v"][at:at + count], at)
        at += count
        held = dict(p, k=cache.k.read()[:at], v=cache.v.read()[:at], hops=p["hops"][:at])
        check(held, "bf16", ask(p, "bf16", cache.cache, nodes=at))


def test_queries_without_nodes_and_nodes_without_queries():
    cache = pkg.NodeCache(0, 2, 64, torch.bfloat16)
    q, lse = torch.randn(3, 4, 64, device="cuda").bfloat16(), torch.empty(3, 4, device="cuda")
    out = torch.full_like(q, 7)
    pkg.CachedAttention(3, 0, 4, 2, 64, torch.bfloat16).forward(q, cache, out, lse)
    assert not out.any() and torch.isneginf(lse).all()
    cache = pkg.NodeCache(9, 2, 64, torch.bfloat16)
    pkg.CachedAttention(0, 9, 4, 2, 64, torch.bfloat16).forward(q[:0], cache, out[:0], lse[:0])
    cache.write(q[:0, :2], q[:0, :2])
    cache.read(out[:0, :2], out[:0, :2])
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,G,n", [(1, 2, 1), (3, 1, 1), (9, 1, 1), (40, 2, 1), (130, 1, 1), (1, 2, 40), (20, 2, 40), (20, 2, 2000), (2, 4, 2000)])
def test_one_node_alone_is_its_value(T, G, n, dtype):
    """A row that sees one node is that node's value to the last bit: 4 bits of it, of which rounding leaves all.

    The weight is off by 2^-9 (bf16) or 2^-12 (fp16) with few rows; that is less than half a step of a value of at most 1.875
    (2^-8 of 1.875, 2^-11 of 1.875).  With more rows it is off by 2^-11, and in fp16 the same again divides it.
    """
    rng = np.random.default_rng(T + n)
    p = problem(T, n, 3 * G, 3, 72, 1, 0, dtype, True, seed=T + n)
    p["source"][:] = 0
    p["hops"][:] = -1
    at = int(rng.integers(0, n))
    p["hops"][at] = 2
    cache, held = cached(p, dtype)
    out, _ = ask(p, dtype, cache)
    np.testing.assert_array_equal(f64(out), np.repeat(held["v"][at][None], T, 0).repeat(G, 1))


@pytest.mark.parametrize("value,at", [(float("nan"), "q"), (float("nan"), "v"), (float("nan"), "k")])
def test_what_is_no_number_shows(value, at):
    p = problem(2, 200, 2, 1, 64, 0, 0, "bf16", False, seed=4)
    p[at][1, 0, 3] = value
    cache, _ = cached(p, "bf16")
    out, lse = ask(p, "bf16", cache)
    if at == "q":
        assert torch.isnan(out[1, 0]).all() and torch.isnan(lse[1, 0]) and not torch.isnan(out[0]).any()
    elif at == "k":
        assert torch.isnan(out).all() and torch.isnan(lse).all()
    else:
        assert torch.isnan(out[:, :, 3]).all() and not torch.isnan(lse).any()


def test_concentrated_and_spread_weights():
    """One node of weight 1 beside very many of 2^-20 each, which make up half of the output."""
    n, d = 1 << 20, 64
    q = torch.zeros(1, 1, d, device="cuda", dtype=torch.float16)
    q[..., 0] = 1
    k = torch.zeros(n, 1, d, device="cuda", dtype=torch.float16)
    k[7, 0, 0] = 14.0                                # e4m3 holds it: weight e^14 = 2^20.2 times the others'
    v = torch.ones(n, 1, d, device="cuda", dtype=torch.float16)
    v[7] = -1
    cache = pkg.NodeCache(n, 1, d, torch.float16)
    cache.write(k, v)
    out, lse = torch.empty_like(q), torch.empty(1, 1, device="cuda")
    pkg.CachedAttention(1, n, 1, 1, d, torch.float16, scale=1.0).forward(q, cache, out, lse)
    total = np.exp(14.0) + n - 1
    assert np.all(np.abs(f64(out) - (n - 1 - np.exp(14.0)) / total) < 2.0 ** -10)
    assert abs(float(lse) - np.log(total)) < 2e-5


def test_norm_write_and_ask_together():
    """Keys normed and turned, kept in 8 bits in two runs, asked by normed queries: as a model would, captured and replayed."""
    rng = np.random.default_rng(22)
    T, n, hq, hkv, d = 4, 900, 8, 2, 64
    p = problem(T, n, hq, hkv, d, T, 8, "bf16", False, seed=21)
    w = (1 + dev(rng, "fp32", d, scale=0.1)).bfloat16()
    where = torch.arange(n, dtype=torch.int32, device="cuda") * 3
    norm_q, norm_k = pkg.HeadNorm(T, hq, d, torch.bfloat16), pkg.HeadNorm(n, hkv, d, torch.bfloat16)
    cache = pkg.NodeCache(n, hkv, d, torch.bfloat16)
    op = pkg.CachedAttention(T, n, hq, hkv, d, torch.bfloat16, sources=T, edges=p["edges"])
    q, k = torch.empty_like(p["q"]), torch.empty_like(p["k"])
    out, lse = torch.empty_like(q), torch.empty(T, hq, device="cuda")

    def step():
        norm_q.forward(p["q"], w, q, positions=where[:T])
        norm_k.forward(p["k"], w, k, positions=where)
        cache.write(k[:333], p["v"][:333])
        cache.write(k[333:], p["v"][333:], first=333)
        op.forward(q, cache, out, lse, hops=p["hops"], bias=p["bias"])
    step()
    torch.cuda.synchronize()
    once = out.clone(), lse.clone()
    # from the inputs on in 64 bits: the rounded queries and keys are the kernels' own (within a rounding of the reference's)
    a = cache_ref.angles(where.cpu().numpy(), d)
    for got, x, angle in ((q, p["q"], a[:T]), (k, p["k"], a)):
        xs, ws = f64(x), f64(w)
        tol = cache_ref.head_norm_tolerances("bf16", xs, xs, ws, angle, d, False, 1e-6)
        close("turned", got, cache_ref.head_norm(xs, ws, angle, d, False, 1e-6)[0], tol["y"])
    kc, vc = cache_ref.Cache(n, hkv, d), cache_ref.Cache(n, hkv, d)
    for c, x in ((kc, k), (vc, p["v"])):
        c.write(f64(x)[:333], 0)
        c.write(f64(x)[333:], 333)
    check(dict(p, q=q, k=kc.read(), v=vc.read()), "bf16", once)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    out.zero_(), lse.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, once[0]) and torch.equal(lse, once[1])
