"""Calls of the 8-bit cache, attention over it and the head norm as programs make them: hop tables at their ends, sources
given twice, part of a cache, other layouts, streams, threads, graphs, offsets past 32 bits, tensors in place."""
import threading

import numpy as np
import pytest

from test_gpu_cache import Both, ask, cached, check
from test_gpu_reader import DT, dev, f64, padded, problem

pytestmark = pytest.mark.gpu

K = pytest.importorskip("compressed_graph_spmv_gb300.k2t")
import compressed_graph_spmv_gb300 as pkg  # noqa: E402

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    K.load()


FEW_AND_MANY = [(8, 1), (4, 2), (1, 8), (9, 1), (20, 2), (70, 2)]


@pytest.mark.parametrize("T,G", FEW_AND_MANY)
@pytest.mark.parametrize("sources", [1, 3, 32])
def test_sources(T, G, sources):
    """Queries that share a source or have none, hops of any int32, a table on a 4-byte boundary."""
    p = problem(T, 5003, 2 * G, 2, 64, sources, 6, "bf16", True, seed=T + sources)
    rng = np.random.default_rng(T * sources)
    p["source"][0] = sources - 1
    p["source"][-1] = [-1, sources, 2 ** 31 - 1, -2 ** 31][T % 4]
    ends = torch.tensor([-2 ** 31, -2, -1, 0, 255, 256, 257, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    at = torch.from_numpy(rng.integers(0, 5003 * sources, size=4000)).cuda()
    p["hops"].view(-1)[at] = ends[torch.from_numpy(rng.integers(0, 8, size=4000)).cuda()]
    room = torch.empty(5003 * sources + 1, dtype=torch.int32, device="cuda")
    room[1:] = p["hops"].view(-1)
    p["hops"] = room[1:].view(5003, sources)
    cache, held = cached(p, "bf16")
    check(held, "bf16", ask(p, "bf16", cache))


@pytest.mark.parametrize("T,G", FEW_AND_MANY)
def test_part_of_a_cache(T, G):
    """What lies behind the nodes of the call, NaN here, is not used; ends inside a tile and a block."""
    n, d = 1000, 72
    p = problem(T, n, 2 * G, 2, d, min(T, 32), 6, "fp16", T > 32, seed=T)
    b = Both(n, 2, d, "fp16")
    b.write(torch.full_like(p["k"], float("nan")), torch.full_like(p["v"], float("nan")))
    at = 0
    for count in (1, 126, 1, 1, 31, 555):
        b.write(p["k"][at:at + count], p["v"][at:at + count], at)
        at += count
        check(dict(p, k=b.k.read()[:at], v=b.v.read()[:at], hops=p["hops"][:at]), "fp16", ask(p, "fp16", b.cache, nodes=at))


@pytest.mark.parametrize("T,G", FEW_AND_MANY)
def test_query_layouts(T, G):
    p = problem(T, 700, 2 * G, 2, 64, min(T, 32), 4, "bf16", T > 32, seed=T)
    cache, held = cached(p, "bf16")
    want = ask(p, "bf16", cache)
    op = pkg.CachedAttention(T, 700, 2 * G, 2, 64, torch.bfloat16, sources=p["hops"].shape[1], edges=p["edges"])
    for lay in (lambda t: padded(t, 8), lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)):
        out, lse = lay(torch.full_like(p["q"], 7)), torch.empty(T, 2 * G, device="cuda")
        op.forward(lay(p["q"]), cache, out, lse, hops=p["hops"], bias=p["bias"], query_source=p["source"])
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    one = p["q"][:1, :1].expand_as(p["q"])               # one query for all
    out, lse = torch.empty_like(p["q"]), torch.empty(T, 2 * G, device="cuda")
    op.forward(one, cache, out, lse, hops=p["hops"], bias=p["bias"], query_source=p["source"])
    check(dict(held, q=one), "bf16", (out, lse))


@pytest.mark.parametrize("T,G", [(2, 2), (1, 8), (33, 2)])
def test_graphs_streams_and_threads(T, G):
    """Two graphs of one object replayed in turn with calls between them; its calls on streams ordered one after another; then
    host threads with a stream and an object each (an object's calls share its work buffer) that ask one cache."""
    n = 30000
    a, b = (problem(T, n, 2 * G, 2, 64, min(T, 32), 6, "bf16", T > 32, seed=s) for s in (1, 2))
    cache, _ = cached(a, "bf16")
    op = pkg.CachedAttention(T, n, 2 * G, 2, 64, torch.bfloat16, sources=a["hops"].shape[1], edges=a["edges"])

    def call(p, out, lse, op=op):
        op.forward(p["q"], cache, out, lse, hops=p["hops"], bias=p["bias"], query_source=p["source"])

    def fresh():
        return torch.zeros_like(a["q"]), torch.zeros(T, 2 * G, device="cuda")
    want = []
    for p in (a, b):
        want.append(fresh())
        call(p, *want[-1])
    torch.cuda.synchronize()
    got, graphs = [fresh(), fresh()], [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for g, p, to in zip(graphs, (a, b), got):
        with torch.cuda.graph(g):
            call(p, *to)
    between = fresh()
    for _ in range(3):
        for g in graphs:
            g.replay()
            call(a, *between)
    torch.cuda.synchronize()
    for g, w in zip(got + [between], want + [want[0]]):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])

    streams, shared = [torch.cuda.Stream() for _ in range(3)], [fresh() for _ in range(6)]
    before = torch.cuda.current_stream()
    for i, to in enumerate(shared):
        streams[i % 3].wait_stream(before)
        before = streams[i % 3]
        with torch.cuda.stream(before):
            call((a, b)[i % 2], *to)
    torch.cuda.synchronize()
    for i, to in enumerate(shared):
        assert torch.equal(to[0], want[i % 2][0]) and torch.equal(to[1], want[i % 2][1])

    results, errors, ops = {}, [], []

    def work(i):
        try:
            own = pkg.CachedAttention(T, n, 2 * G, 2, 64, torch.bfloat16, sources=a["hops"].shape[1], edges=a["edges"])
            ops.append(own)
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                to = fresh()
                for _ in range(20):
                    call((a, b)[i % 2], *to, op=own)
            stream.synchronize()
            results[i] = to
        except Exception as e:      # noqa: BLE001 - shown below
            errors.append(e)
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for i, to in results.items():
        assert torch.equal(to[0], want[i % 2][0]) and torch.equal(to[1], want[i % 2][1])
    assert op.status() == 0 and len(ops) == 4 and all(o.status() == 0 for o in ops)


@pytest.mark.parametrize("T", [1, 40])
def test_offsets_past_32_bits(T):
    """Heads that begin more than 2^32 bytes into the cache; the last hundred nodes and the first two are seen."""
    n, heads, d, last = 1100001, 32, 128, 100
    rng = np.random.default_rng(T)
    cache = pkg.NodeCache(n, heads, d, torch.bfloat16)
    k, v = dev(rng, "bf16", last, heads, d), dev(rng, "bf16", last, heads, d)
    cache.write(k, v, first=n - last)
    back = torch.empty_like(k), torch.empty_like(v)
    cache.read(*back, first=n - last)
    nodes = torch.arange(n - last, n, dtype=torch.int32, device="cuda")
    again = torch.empty_like(k), torch.empty_like(v)
    cache.read(*again, nodes=nodes)
    for x, held, other in zip((k, v), back, again):
        assert torch.equal(held, other)
        # half a step of a normal e4m3 is 2^-4 of a value; below, 2^-10 of the scale, which is under 1/224 of the largest value
        xs = f64(x)
        assert np.all(np.abs(f64(held) - xs) <= np.maximum(np.abs(xs) * 2.0 ** -4, np.abs(xs).max() * 2.0 ** -17))
    hops = torch.full((n, 1), -1, dtype=torch.int32, device="cuda")
    hops[-last:, 0] = torch.from_numpy(rng.integers(0, 9, size=last).astype(np.int32)).cuda()
    hops[:2] = 3
    p = dict(q=dev(rng, "bf16", T, heads, d), hops=hops, bias=dev(rng, "bf16", heads, 5), edges=pkg.hop_edges(5, 12),
             source=torch.zeros(T, dtype=torch.int32, device="cuda"))
    out = ask(p, "bf16", cache)
    zero = np.zeros((2, heads, d))
    seen = dict(p, hops=torch.cat([hops[:2], hops[-last:]]), k=np.concatenate([zero, f64(back[0])]), v=np.concatenate([zero, f64(back[1])]))
    check(seen, "bf16", out)


@pytest.mark.parametrize("T,G", [(2, 2), (40, 2)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("at,value", [("q", "nan"), ("q", "inf"), ("bias", "nan"), ("bias", "inf"), ("bias", "-inf"), ("bias", "max"), ("bias", "min")])
def test_what_is_no_number_shows_where_it_does_over_16_bits(T, G, dtype, at, value):
    p = problem(T, 300, 2 * G, 2, 64, min(T, 32), 3, dtype, T > 32, seed=T)
    x = {"max": torch.finfo(DT[dtype]).max, "min": torch.finfo(DT[dtype]).min}.get(value)
    x = float(value) if x is None else x
    if at == "q":
        p["q"][1, 0, 3] = x
    else:
        p["bias"][1, 1] = x
    cache, held = cached(p, dtype)
    out, lse = ask(p, dtype, cache)
    k, v = (torch.from_numpy(held[s]).to(DT[dtype]).cuda() for s in "kv")
    op = pkg.HopAttention(T, 300, 2 * G, 2, 64, DT[dtype], sources=p["hops"].shape[1], edges=p["edges"])
    w, l = torch.empty_like(out), torch.empty_like(lse)
    op.forward(p["q"], k, v, w, l, hops=p["hops"], bias=p["bias"], query_source=p["source"])
    assert torch.equal(torch.isnan(out), torch.isnan(w)) and torch.equal(torch.isnan(lse), torch.isnan(l))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("heads,d,rotary", [(4, 128, 128), (5, 72, 40), (1, 8, 8)])
def test_head_norm_in_place(heads, d, rotary, dtype):
    rng = np.random.default_rng(d)
    n = 60013
    x, dy, w = dev(rng, dtype, n, heads, d), dev(rng, dtype, n, heads, d), dev(rng, dtype, d)
    op = pkg.HeadNorm(n, heads, d, DT[dtype], rotary_dim=rotary)
    y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)
    op.forward(x, w, y)
    op.backward(dy, x, w, dx, dw)
    a = x.clone()
    op.forward(a, w, a)
    assert torch.equal(a, y)
    for over in ("dy", "x"):
        a, b, dw2 = x.clone(), dy.clone(), torch.empty_like(w)
        to = b if over == "dy" else a
        op.backward(b, a, w, to, dw2)
        assert torch.equal(to, dx) and torch.equal(dw2, dw)
    row = x[:1].expand(n, heads, d)                      # one row at every position
    op.forward(row, w, y)
    op.forward(row.contiguous(), w, a)
    assert torch.equal(a, y)
