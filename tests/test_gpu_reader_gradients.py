"""Gradients of the attention where it concentrates and where it spreads over
very many nodes, against 64-bit references on the GPU.

Bounds beside those of tests/reader_ref.py (u: unit roundoff of the element
type, w: relative error of a weight, p weights, dp = dout . v).  The sums by
bucket are sums in 32 bits of score gradients that keep 16 bits or more, and
delta is the mean of dp under the same weights, both in 32 bits.  A thread adds
32 nodes of each of its block's tiles one after another, and the at least
150 / (key/value heads) blocks of a head share its tiles: r terms in a row are
off by at most r 2^-24 of the absolute terms (r = 256 where it is less):
  delta <= sum p (w |dp - delta| + e_dp) + r 2^-24 sum p |dp|
  ds    <= p (w |dp - delta| + e_dp + tol(delta)) + 2^-15 |ds|
  dbias <= u |dbias| + sum (tol(ds) + r 2^-24 |ds|)
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

K = pytest.importorskip("compressed_graph_spmv_gb300.k2t")
import compressed_graph_spmv_gb300 as pkg  # noqa: E402

torch = pytest.importorskip("torch")
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    K.load()


def call(x, dtype, edges, scale=None):
    """Forward and backward of one problem: every output, as 64-bit tensors."""
    T, hq, d = x["q"].shape
    n, hkv, _ = x["k"].shape
    op = pkg.HopAttention(T, n, hq, hkv, d, DT[dtype], sources=0 if x["hops"] is None else x["hops"].shape[1], edges=edges,
                          scale=scale)
    out, lse = torch.full_like(x["q"], float("nan")), torch.full((T, hq), float("nan"), device="cuda")
    table = dict(hops=x["hops"], bias=x["bias"], query_source=x.get("source"))
    op.forward(x["q"], x["k"], x["v"], out, lse, **table)
    g = {"d" + y: torch.full(x[y].shape, float("nan"), dtype=DT[dtype], device="cuda") for y in ("q", "k", "v")}
    db = None if x["bias"] is None else torch.full_like(x["bias"], float("nan"))
    op.backward(x["dout"], x["q"], x["k"], x["v"], out, lse, g["dq"], g["dk"], g["dv"], dbias=db, **table)
    assert op.status() == 0
    return {a: b.double() for a, b in dict(g, out=out, lse=lse, dbias=db).items() if b is not None}


def reference(x, dtype, edges, scale=None):
    """The definitions in 64 bits on the GPU, one head at a time, and the sharp bounds of dbias."""
    u = U[dtype]
    q, k, v, dout = (x[y].double() for y in ("q", "k", "v", "dout"))
    T, hq, d = q.shape
    group, scale = hq // k.shape[1], d ** -0.5 if scale is None else scale
    bucket = hidden = None
    if x["hops"] is not None:
        first = torch.tensor(edges, device="cuda", dtype=torch.int32)
        column = torch.arange(T, device="cuda") if x.get("source") is None else x["source"].long()
        seen = x["hops"][:, column.clamp(min=0)].t()
        bucket = torch.searchsorted(first, seen.clamp(min=0).contiguous(), right=True) - 1
        hidden = (seen < 0) & (column >= 0)[:, None]
        bucket[column < 0] = -1
    r = {y: torch.zeros_like(t) for y, t in (("out", q), ("dq", q), ("dk", k), ("dv", v))}
    r["dbias"] = tol = None
    row = max(256, 32 * -(-(-(-k.shape[0] // 128)) // (150 // k.shape[1]))) * 2.0 ** -24
    if x["bias"] is not None:
        r["dbias"], tol = torch.zeros_like(x["bias"], dtype=torch.float64), torch.zeros_like(x["bias"], dtype=torch.float64)
    for h in range(hq):
        c = h // group
        s = scale * q[:, h] @ k[:, c].t()
        if x["bias"] is not None:
            s += torch.where(bucket >= 0, x["bias"][h].double()[bucket.clamp(min=0)], 0.0)
        if hidden is not None:
            s[hidden] = -float("inf")
        p = torch.softmax(s, 1)
        dp = dout[:, h] @ v[:, c].t()
        delta = (p * dp).sum(1, keepdim=True)
        ds = p * (dp - delta)
        r["out"][:, h] = p @ v[:, c]
        r["dq"][:, h] = scale * ds @ k[:, c]
        r["dk"][:, c] += scale * ds.t() @ q[:, h]
        r["dv"][:, c] += p.t() @ dout[:, h]
        if tol is None:
            continue
        size = (scale * q[:, h].abs() @ k[:, c].abs().t()).max() + x["bias"][h].double().abs().max()
        w = 2.5 * (d + 8) * 2.0 ** -24 * size + 2.0 ** -20
        e_dp = d * 2.0 ** -24 * dout[:, h].abs() @ v[:, c].abs().t()
        e_delta = (p * (w * (dp - delta).abs() + e_dp)).sum(1, keepdim=True) + row * (p * dp.abs()).sum(1, keepdim=True)
        e_ds = p * (w * (dp - delta).abs() + e_dp + e_delta) + (2.0 ** -15 + row) * ds.abs()
        for b in range(len(edges)):
            r["dbias"][h, b] = ds[bucket == b].sum()
            tol[h, b] = u * r["dbias"][h, b].abs() + e_ds[bucket == b].sum()
    return r, tol


def problem(T, n, hq, hkv, d, dtype, edges, seed, sources=None, mapped=False):
    """Each source at hop 0 of itself, the other nodes some hops away, a twentieth not reached."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(DT[dtype])  # noqa: E731
    sources = sources or T
    hops = torch.randint(1, edges[-1] + 2, (n, sources), generator=g, device="cuda", dtype=torch.int32)
    hops[torch.rand(n, generator=g, device="cuda") < 0.05] = -1
    at = torch.randperm(n, generator=g, device="cuda")[:sources]
    hops[at, torch.arange(sources, device="cuda")] = 0
    x = dict(q=rand(T, hq, d), k=rand(n, hkv, d), v=rand(n, hkv, d), dout=rand(T, hq, d), hops=hops, bias=rand(hq, len(edges)), at=at)
    if mapped:
        x["source"] = torch.randint(-1, sources, (T,), generator=g, device="cuda", dtype=torch.int32)
    return x


def within(name, got, want, tol):
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of its bound" % (
        name, int(bad.sum()), bad.numel(), float(((got - want).abs() / tol)[bad].max()))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,n,hq,hkv,d,mapped,peak", [
    (1, 65536, 2, 2, 64, False, 17.0), (8, 65536, 4, 2, 64, False, 17.0), (3, 65536, 2, 1, 128, False, 17.0),
    (40, 20000, 4, 2, 64, True, 16.0), (150, 20000, 3, 1, 96, True, 16.0), (8, 3001, 2, 2, 64, False, 0.0)])
def test_bias_gradient_where_attention_concentrates(T, n, hq, hkv, d, mapped, peak, dtype):
    """About 0.99 of a row's weight on the source's own node: every bucket within its own bound."""
    edges = list(range(9))
    x = problem(T, n, hq, hkv, d, dtype, edges, seed=T + n, sources=min(T, 32), mapped=mapped)
    if peak:
        x["bias"][:, 0] = peak
        x["q"] *= 0.25
    want, tol = reference(x, dtype, edges)
    within("dbias", call(x, dtype, edges)["dbias"], want["dbias"], tol)


def test_bias_gradient_of_queries_that_match_their_own_node():
    x = problem(32, 20000, 2, 2, 64, "bf16", list(range(9)), seed=5)
    x["q"] = (x["k"][x["at"]] * 1.75).contiguous()
    want, tol = reference(x, "bf16", list(range(9)))
    within("dbias", call(x, "bf16", list(range(9)))["dbias"], want["dbias"], tol)


def off(got, want):
    return float((got - want).norm() / want.norm())


@pytest.mark.parametrize("n,peak,buckets,spread", [(1 << 20, 0.0, 9, 1.0), (1 << 20, 18.5, 9, 1.0), (1 << 22, 0.0, 9, 1.0), (1 << 22, 20.0, 9, 1.0),
                                                   (1 << 21, 0.0, 0, 1.0), (1 << 20, 0.0, 9, 2.0 ** -9), (1 << 20, 0.0, 0, 2.0 ** 10)])
def test_half_gradients_over_very_many_nodes(n, peak, buckets, spread):
    """Weights of 2^-20 and less are not lost in fp16, whatever the size of dout (its second row's is `spread` times the
    first's).  Score gradients and results are rounded once each, 2^-11 of a value: a row's dq as a whole is off by no more
    than 2^-10 of its norm, the least value's step (2^-25 each) aside."""
    edges = list(range(9)) if buckets else None
    x = problem(2, n, 1, 1, 32, "fp16", list(range(9)), seed=n + buckets, sources=2)
    if buckets:
        x["bias"][:, 0] = peak
    else:
        x["hops"] = x["bias"] = None
    x["q"] *= 0.25
    x["dout"][1] *= spread
    # results of ordinary size: what fp16 cannot hold of them is not the question here
    x["dout"] *= 16
    x["k"] *= 16
    x["q"] /= 16
    want, tol = reference(x, "fp16", edges)
    got = call(x, "fp16", edges)
    for t in range(2):
        least = 2.0 ** -25 * 32 ** 0.5 / float(want["dq"][t].norm())
        assert off(got["dq"][t], want["dq"][t]) <= 2.0 ** -10 + least, (t, off(got["dq"][t], want["dq"][t]))
    if buckets:
        within("dbias", got["dbias"], want["dbias"], tol + 2.0 ** -25)


@pytest.mark.parametrize("scale", [2.0 ** -14, 2.0 ** -8, 256.0, 4096.0])
@pytest.mark.parametrize("T,d,mapped", [(5, 64, False), (40, 128, True), (150, 96, True)])
def test_half_gradients_of_any_size(T, d, mapped, scale):
    """dout over the whole range of the type: products of dout and v far above and below it."""
    edges = list(range(9))
    x = problem(T, 700, 2, 1, d, "fp16", edges, seed=T, sources=min(T, 5), mapped=mapped)
    x["dout"] *= scale
    x["v"] *= 4
    want, tol = reference(x, "fp16", edges)
    got = call(x, "fp16", edges)
    fits = want["dbias"].abs() < 65000
    within("dbias", got["dbias"][fits], want["dbias"][fits], tol[fits] + 2.0 ** -25)
    for name in ("dq", "dk", "dv"):
        # rounded operands of the products, weights or score gradients: 2^-10 of the norm; the result: 2^-11 and the least step
        least = 2.0 ** -25 * got[name].numel() ** 0.5 / float(want[name].norm())
        fits = want[name].abs() < 65000
        assert torch.isfinite(got[name][fits]).all() and off(got[name][fits], want[name][fits]) <= 2.0 ** -9 + least, name


@pytest.mark.parametrize("T,n,hq,hkv,d,mapped", [(2, 65536, 1, 1, 32, False), (8, 65536, 4, 2, 64, False), (100, 30000, 2, 2, 128, True)])
def test_half_gradients_beside_values_that_do_not_count(T, n, hq, hkv, d, mapped):
    """A thousand nodes with values 2^12 times as large as the others', in a bucket whose bias leaves them 2^-58 of a weight:
    they change nothing, nor what the others' gradients keep."""
    edges = list(range(9))
    x = problem(T, n, hq, hkv, d, "fp16", edges, seed=T, sources=min(T, 32), mapped=mapped)
    if mapped:
        x["source"].clamp_(min=0)
    far = torch.randperm(n, device="cuda")[:1000]
    x["hops"][far] = 8
    x["bias"][:, 8] = -40.0
    x["hops"][x["hops"] == 9] = 7
    near = torch.ones(n, dtype=torch.bool, device="cuda")
    near[far] = False
    x["hops"][near] = x["hops"][near].clamp(max=7)
    x["v"][far] *= 2.0 ** 12
    x["q"] /= 16
    x["k"] *= 16
    want, tol = reference(x, "fp16", edges)
    got = call(x, "fp16", edges)
    least = 2.0 ** -25 * got["dq"].numel() ** 0.5 / float(want["dq"].norm())
    assert off(got["dq"], want["dq"]) <= 2.0 ** -10 + least, off(got["dq"], want["dq"])
    within("dbias", got["dbias"], want["dbias"], tol + 2.0 ** -25)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,low", [(1, -8.0), (1, -6.0), (8, -8.0), (20, -10.0)])
def test_bias_gradient_of_a_bucket_of_little_weight(T, low, dtype):
    """A bucket whose nodes have 2^-33 to 2^-39 of the weight of a row's largest each: its sum does not lose them."""
    edges, n = list(range(9)), 65536
    x = problem(T, n, 2, 2, 8, dtype, edges, seed=T, sources=min(T, 32))
    x["bias"].zero_()
    x["bias"][:, 0], x["bias"][:, 8] = 17.0, low
    x["q"] *= 2.0 ** -4
    x["dout"] *= 2.0 ** 13
    want, tol = reference(x, dtype, edges)
    within("dbias", call(x, dtype, edges)["dbias"], want["dbias"], tol + 2.0 ** -25)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,hq,hkv,d,mapped,table", [(6, 4, 2, 64, False, True), (1, 2, 2, 128, False, True), (90, 4, 2, 64, True, True),
                                                     (150, 2, 1, 96, True, True), (6, 4, 2, 64, False, False)])
def test_nodes_in_parts(T, hq, hkv, d, mapped, table, dtype):
    """Forward calls of parts of the nodes, their out and lse joined, and backward calls of the parts with the joined ones:
    the gradients of all nodes at once, within a few roundings of the outputs (delta comes from a rounded out)."""
    edges, n = list(range(9)), 3000
    x = problem(T, n, hq, hkv, d, dtype, edges, seed=T, sources=min(T, 6), mapped=mapped)
    if not table:
        x["hops"] = x["bias"] = None
    want, _ = reference(x, dtype, edges)
    parts = [slice(0, 1000), slice(1000, 1100), slice(1100, n)]
    outs, lses, ops = [], [], []
    for s in parts:
        m = s.stop - s.start
        op = pkg.HopAttention(T, m, hq, hkv, d, DT[dtype], sources=x["hops"].shape[1] if table else 0, edges=edges if table else None)
        out, lse = torch.empty_like(x["q"]), torch.empty(T, hq, device="cuda")
        hops = x["hops"][s].contiguous() if table else None
        op.forward(x["q"], x["k"][s], x["v"][s], out, lse, hops=hops, bias=x["bias"], query_source=x.get("source"))
        outs.append(out.double()), lses.append(lse.double()), ops.append((op, hops))
    lse = torch.logsumexp(torch.stack(lses), 0)
    out = sum(o * torch.exp(l - lse)[..., None] for o, l in zip(outs, lses)).to(DT[dtype])
    lse, dq, db = lse.float(), 0, 0
    dk, dv = torch.empty_like(x["k"]), torch.empty_like(x["v"])
    for s, (op, hops) in zip(parts, ops):
        dqp, dbp = torch.empty_like(x["q"]), torch.empty_like(x["bias"]) if table else None
        op.backward(x["dout"], x["q"], x["k"][s], x["v"][s], out, lse, dqp, dk[s], dv[s], dbias=dbp, hops=hops, bias=x["bias"],
                    query_source=x.get("source"))
        dq = dq + dqp.double()
        db = db + dbp.double() if table else 0
    got = dict(dq=dq, dk=dk.double(), dv=dv.double())
    if table:
        got["dbias"] = db
    for name, g in got.items():
        assert off(g, want[name]) <= 8 * U[dtype], (name, off(g, want[name]))
