"""Graph-reading operators on the GPU against 64-bit references: outputs and
gradients element by element within the bounds of tests/reader_ref.py."""
import numpy as np
import pytest

import reader_ref as ref
import synth

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


def f64(t):
    return t.detach().double().cpu().numpy()


def dev(rng, dtype, *shape, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale).to(DT[dtype]).cuda()


def padded(t, extra):
    """The same values with `extra` unused values after every head and row."""
    n, h, d = t.shape
    wide = torch.full((n, h + 1, d + extra), float("nan"), dtype=t.dtype, device=t.device)
    wide[:, :h, :d] = t
    return wide[:, :h, :d]


def close(name, got, want, tol):
    got = f64(got)
    assert got.shape == want.shape, name
    same = np.isneginf(want) & np.isneginf(got)
    bad = ~(same | (np.abs(got - want) <= tol))
    assert not bad.any(), "%s: %d of %d off, worst %.3g of its bound" % (
        name, int(bad.sum()), bad.size, float(np.nanmax(np.abs(got - want)[bad] / tol[bad])))


def problem(T, n, hq, hkv, d, sources, buckets, dtype, mapped, seed, reach=0.7):
    rng = np.random.default_rng(seed)
    p = dict(q=dev(rng, dtype, T, hq, d), k=dev(rng, dtype, n, hkv, d), v=dev(rng, dtype, n, hkv, d),
             dout=dev(rng, dtype, T, hq, d), hops=None, bias=None, source=None, edges=None)
    if sources:
        depth = rng.integers(0, 9, size=(n, 1)) + rng.integers(0, 3, size=(n, sources))
        depth[rng.random(n) > reach] = -1
        depth[rng.random((n, sources)) > 0.95] = -1
        if n > 2:
            depth[1] = 300   # past the last bucket's first hop and past a byte
        p["hops"] = torch.from_numpy(depth.astype(np.int32)).cuda()
        if buckets:
            p["bias"] = dev(rng, dtype, hq, buckets)
            p["edges"] = pkg.hop_edges(buckets, max(buckets - 1, 12))
        if mapped:
            p["source"] = torch.from_numpy(rng.integers(-1, sources, size=T).astype(np.int32)).cuda()
    return p


def table_of(p):
    return dict(hops=p["hops"], bias=p["bias"], query_source=p["source"])


def ref_table(p, dtype):
    return dict(dtype=dtype, hops=None if p["hops"] is None else p["hops"].cpu().numpy(),
                bias=None if p["bias"] is None else f64(p["bias"]), edges=p["edges"],
                source=None if p["source"] is None else p["source"].cpu().numpy())


def run(p, dtype, scale=None, backward=True, poison=True):
    T, hq, d = p["q"].shape
    n, hkv, _ = p["k"].shape
    op = pkg.HopAttention(T, n, hq, hkv, d, DT[dtype], sources=0 if p["hops"] is None else p["hops"].shape[1],
                          edges=p["edges"], scale=scale)
    out = torch.full_like(p["q"].contiguous(), float("nan"))
    lse = torch.full((T, hq), float("nan"), device="cuda")
    if poison:   # nothing in the work buffers may be relied on
        for b in (0, 1):
            op._work_of(b)
            op._work[b].fill_(0xff)
            op._work[b][:4].zero_()   # the status word is the caller's to clear
    op.forward(p["q"], p["k"], p["v"], out, lse, **table_of(p))
    got = dict(out=out, lse=lse)
    if backward:
        g = {x: torch.full(p[x[1:]].shape, float("nan"), dtype=DT[dtype], device="cuda") for x in ("dq", "dk", "dv")}
        db = None if p["bias"] is None else torch.full_like(p["bias"], float("nan"))
        op.backward(p["dout"], p["q"], p["k"], p["v"], out, lse, g["dq"], g["dk"], g["dv"], dbias=db, **table_of(p))
        got |= g | dict(dbias=db)
    torch.cuda.synchronize()
    assert op.status() == 0
    return got


def check(p, dtype, got, scale=None):
    q, k, v, dout = (f64(p[x]) for x in ("q", "k", "v", "dout"))
    d = q.shape[2]
    scale = d ** -0.5 if scale is None else scale
    nb = 0 if p["bias"] is None else p["bias"].shape[1]
    if p["hops"] is not None:   # states that no query sees do not count
        hops = p["hops"].cpu().numpy()
        T = q.shape[0]
        cols = list(range(T)) if p["source"] is None else p["source"].cpu().tolist()
        used = [c for c in cols if 0 <= c < hops.shape[1]]
        if len(used) == len(cols):
            hidden = (hops[:, used] < 0).all(axis=1) if used else np.ones(k.shape[0], bool)
            k[hidden] = 0
            v[hidden] = 0
    want = ref.gradients(q, k, v, dout, scale, n_buckets=nb, **ref_table(p, dtype))
    tol = ref.attention_tolerances(q, k, v, scale, dtype, bias=None if p["bias"] is None else f64(p["bias"]), dout=dout,
                                   ref=want)
    for name, x in got.items():
        if x is not None:
            close(name, x, want[name], tol[name])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,n,hq,hkv,d,sources,buckets,mapped", [
    (1, 1, 1, 1, 64, 1, 4, False), (1, 63, 8, 8, 64, 1, 16, False), (1, 1000, 16, 4, 128, 1, 32, False),
    (2, 64, 2, 1, 8, 2, 1, False), (5, 65, 3, 3, 40, 5, 2, False), (13, 777, 6, 2, 72, 13, 11, False),
    (32, 515, 4, 4, 128, 32, 64, False), (32, 300, 8, 2, 64, 32, 7, False), (17, 129, 4, 4, 96, 3, 5, True),
    (70, 200, 4, 1, 64, 32, 32, True), (131, 321, 2, 2, 128, 7, 3, True), (9, 200, 3, 1, 128, 9, 0, False),
    (8, 100, 4, 4, 32, 0, 0, False), (33, 130, 16, 1, 64, 0, 0, False), (300, 2, 4, 2, 40, 17, 15, True),
    (64, 1025, 2, 2, 128, 0, 0, False), (129, 640, 3, 1, 128, 30, 20, True),
])
def test_attention_matches(T, n, hq, hkv, d, sources, buckets, mapped, dtype):
    p = problem(T, n, hq, hkv, d, sources, buckets, dtype, mapped, seed=T * 1000 + n)
    check(p, dtype, run(p, dtype))


@pytest.mark.parametrize("T,hq,hkv,d", [(1, 4, 4, 64), (20, 4, 1, 64), (32, 8, 4, 64), (2, 2, 2, 128), (32, 4, 2, 128),
                                        (32, 3, 1, 128), (150, 2, 1, 128), (140, 2, 1, 64), (300, 1, 1, 72)])
def test_attention_many_nodes(T, hq, hkv, d):
    """Enough nodes that every block of the split takes many tiles."""
    p = problem(T, 40000 if T <= 32 else 20000, hq, hkv, d, min(T, 32), 16, "bf16", T > 32, seed=7)
    check(p, "bf16", run(p, "bf16"))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T", [6, 90])
def test_attention_strides(dtype, T):
    p = problem(T, 150, 4, 2, 72, 6, 5, dtype, T > 6, seed=3)
    plain = run(p, dtype)
    for x in ("q", "k", "v", "dout"):
        p[x] = padded(p[x], 8)
    strided = run(p, dtype)
    for name in plain:
        assert torch.equal(plain[name], strided[name]), name
    # outputs with strides of their own, nothing written between them
    T, hq, d = p["q"].shape
    op = pkg.HopAttention(T, 150, 4, 2, 72, DT[dtype], sources=6, edges=p["edges"])
    wide = {x: torch.full((s[0], s[1] + 1, s[2] + 8), 7.0, dtype=DT[dtype], device="cuda")
            for x, s in (("out", (T, 4, 72)), ("dq", (T, 4, 72)), ("dk", (150, 2, 72)), ("dv", (150, 2, 72)))}
    view = {x: t[:, :-1, :72] for x, t in wide.items()}
    lse, db = torch.empty(T, 4, device="cuda"), torch.empty_like(p["bias"])
    op.forward(p["q"], p["k"], p["v"], view["out"], lse, **table_of(p))
    op.backward(p["dout"], p["q"], p["k"], p["v"], view["out"], lse, view["dq"], view["dk"], view["dv"], dbias=db,
                **table_of(p))
    for x, t in wide.items():
        assert torch.equal(view[x], plain[x]), x
        assert (t[:, -1] == 7).all() and (t[:, :, 72:] == 7).all(), x


@pytest.mark.parametrize("T", [5, 80])
def test_rows_with_nothing_left(T):
    """A query whose column is all masked gives zeros and no gradient; all masked gives zeros everywhere."""
    p = problem(T, 100, 4, 2, 64, 5, 4, "bf16", T > 5, seed=11)
    p["hops"][:, 2] = -1
    got = run(p, "bf16")
    check(p, "bf16", got)
    dead = [2] if p["source"] is None else (p["source"] == 2).nonzero().flatten().tolist()
    assert dead
    assert (got["out"][dead] == 0).all() and (got["dq"][dead] == 0).all() and torch.isneginf(got["lse"][dead]).all()
    p["hops"].fill_(-1)
    if p["source"] is not None:
        p["source"].clamp_(min=0)
    got = run(p, "bf16")
    for x in ("out", "dq", "dk", "dv", "dbias"):
        assert (got[x] == 0).all(), x
    assert torch.isneginf(got["lse"]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T", [4, 70])
@pytest.mark.parametrize("value", ["-inf", "lowest"])
def test_masked_buckets(dtype, T, value):
    p = problem(T, 200, 4, 2, 64, 4, 6, dtype, T > 4, seed=13)
    low = float("-inf") if value == "-inf" else torch.finfo(DT[dtype]).min
    p["bias"][:, 2] = low
    p["bias"][1] = low   # one head sees nothing at all, except through queries without hop information
    got = run(p, dtype)
    check(p, dtype, got)
    assert (got["dbias"][:, 2] == 0).all() and (got["dbias"][1] == 0).all()


@pytest.mark.parametrize("T,n,hq,hkv,d,sources,buckets,mapped", [
    (3, 41, 1, 1, 128, 3, 6, False), (121, 66, 4, 4, 128, 18, 2, True), (387, 1498, 8, 8, 64, 13, 2, True),
    (8, 3, 2, 1, 64, 8, 32, False), (40, 9000, 8, 2, 72, 5, 64, True), (1, 1, 2, 2, 64, 1, 3, False), (2, 300000, 3, 3, 40, 2, 1, False)])
def test_bias_gradients_add_up_to_zero(T, n, hq, hkv, d, sources, buckets, mapped):
    """A row's weights always sum to 1, so shifting all buckets of a head changes nothing."""
    p = problem(T, n, hq, hkv, d, sources, buckets, "bf16", mapped, seed=T + n)
    got = run(p, "bf16")
    db = f64(got["dbias"])
    # each value is rounded once (2^-9 of it); the sums before it have 32 bits, and no value exceeds the largest of dout . v
    most = np.abs(f64(p["dout"])).sum(axis=2).max() * np.abs(f64(p["v"])).max()
    assert (np.abs(db.sum(axis=1)) <= 2.0 ** -9 * np.abs(db).sum(axis=1) + 2.0 ** -20 * T * most).all()
    check(p, "bf16", got)


@pytest.mark.parametrize("T", [6, 100])
def test_unseen_nodes_may_hold_anything(T):
    p = problem(T, 333, 4, 2, 128, 6, 5, "bf16", False, seed=17) if T <= 6 else problem(T, 333, 4, 2, 128, 6, 5, "bf16", True, seed=17)
    if p["source"] is not None:
        p["source"].clamp_(min=0)
    clean = run(p, "bf16")
    hidden = (p["hops"] < 0).all(dim=1)
    assert hidden.any()
    p["k"][hidden] = float("nan")
    p["v"][hidden] = float("inf")
    got = run(p, "bf16")
    for x in clean:
        assert torch.equal(clean[x], got[x]), x
    assert (got["dk"][hidden] == 0).all() and (got["dv"][hidden] == 0).all()


@pytest.mark.parametrize("T,sources", [(5, 5), (8, 8), (32, 32), (40, 20)])
def test_hops_of_any_value(T, sources):
    """Every negative number masks, every large one falls into the last bucket."""
    p = problem(T, 700, 2, 1, 64, sources, 6, "bf16", T > 32, seed=43)
    odd = torch.tensor([-(1 << 31), -(1 << 31) + 1, -1000, -257, -256, -2, (1 << 31) - 1, (1 << 31) - 2, 65536, 257, 256, 255, 254],
                       dtype=torch.int32, device="cuda")
    where = torch.rand(p["hops"].shape, device="cuda") < 0.5
    pick = odd[torch.randint(0, odd.numel(), p["hops"].shape, device="cuda")]
    p["hops"] = torch.where(where, pick, p["hops"]).contiguous()
    check(p, "bf16", run(p, "bf16"))


def test_lengths_of_zero():
    p = problem(3, 0, 4, 2, 64, 3, 4, "bf16", False, seed=1)
    got = run(p, "bf16")
    assert (got["out"] == 0).all() and torch.isneginf(got["lse"]).all()
    assert (got["dq"] == 0).all() and (got["dbias"] == 0).all() and got["dk"].numel() == 0
    p = problem(0, 70, 4, 2, 64, 3, 4, "bf16", False, seed=1)
    got = run(p, "bf16")
    assert (got["dk"] == 0).all() and (got["dv"] == 0).all() and (got["dbias"] == 0).all()
    p = problem(100, 0, 4, 2, 64, 3, 4, "bf16", True, seed=1)
    got = run(p, "bf16")
    assert (got["out"] == 0).all() and (got["dq"] == 0).all() and (got["dbias"] == 0).all()


def test_large_scores_and_scale():
    """Scores of several hundred: the running maximum carries them."""
    for T in (7, 90):
        p = problem(T, 400, 2, 2, 64, 0, 0, "fp16", False, seed=19)
        p["q"] *= 8
        p["k"] *= 8
        check(p, "fp16", run(p, "fp16", scale=0.5, backward=False), scale=0.5)


def test_offsets_past_32_bits():
    """Node rows 2^26 elements apart: element offsets pass 2^32."""
    n, pitch = 70, 1 << 26
    p = problem(3, n, 2, 2, 64, 3, 4, "bf16", False, seed=23)
    plain = run(p, "bf16")
    store = torch.empty((n - 1) * pitch + 2 * 64 + 1024, dtype=torch.bfloat16, device="cuda")
    for x, off in (("k", 0), ("v", 512)):
        far = store[off:].as_strided((n, 2, 64), (pitch, 64, 1))
        far.copy_(p[x])
        p[x] = far
    got = run(p, "bf16")
    for x in plain:
        assert torch.equal(plain[x], got[x]), x


@pytest.mark.parametrize("T", [9, 77])
def test_repeatable_and_on_another_stream(T):
    p = problem(T, 5000, 8, 2, 64, 9, 16, "bf16", T > 9, seed=29)
    first, again = run(p, "bf16"), run(p, "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        third = run(p, "bf16")
    for x in first:
        assert torch.equal(first[x], again[x]) and torch.equal(first[x], third[x]), x


def test_graph_capture():
    """The calls can be recorded: they allocate nothing and never wait."""
    p = problem(12, 3000, 4, 2, 64, 12, 8, "bf16", False, seed=31)
    op = pkg.HopAttention(12, 3000, 4, 2, 64, torch.bfloat16, sources=12, edges=p["edges"])
    out, lse = torch.empty_like(p["q"]), torch.empty(12, 4, device="cuda")
    g = {x: torch.empty_like(p[x[1:]]) for x in ("dq", "dk", "dv")}
    db = torch.empty_like(p["bias"])

    def step():
        op.forward(p["q"], p["k"], p["v"], out, lse, **table_of(p))
        op.backward(p["dout"], p["q"], p["k"], p["v"], out, lse, g["dq"], g["dk"], g["dv"], dbias=db, **table_of(p))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (out, lse, db, *g.values()):
        t.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    check(p, "bf16", dict(out=out, lse=lse, dbias=db, **g))


def test_hops_of_a_search():
    """The table k2t_msbfs leaves is the one the attention reads."""
    n = 1 << 10
    rows, cols = synth.rmat(10, 0.57, 0.19, 0.19, 3000, 5)
    tree = K.Tree(rows, cols, n, n).upload()
    dist = torch.empty(n, 32, dtype=torch.int32, device="cuda")
    work = torch.empty(tree.msbfs_work_bytes(), dtype=torch.uint8, device="cuda")
    tree.msbfs(K.RIGHT, np.random.default_rng(5).choice(n, size=32), dist, work)
    p = problem(32, n, 4, 2, 64, 0, 0, "bf16", False, seed=37)
    p["hops"], p["edges"] = dist, pkg.hop_edges(8)
    p["bias"] = dev(np.random.default_rng(6), "bf16", 4, 8)
    assert (dist < 0).any() and (dist > 1).any()
    check(p, "bf16", run(p, "bf16"))


# ---- layer norm ------------------------------------------------------------
def norm_tolerances(dtype, x, z, xh, rstd, w, b, dy, dz, y, dx, dw, db):
    """fp32 statistics: the mean of dim values is off by at most 2^-20 mean|z| (trees of short runs), so xh by
    e = 2^-20 (rstd mean|z| + |xh| + 1); then the formulas' terms, and u of the result."""
    u = ref.U[dtype]
    e = 2.0 ** -20 * (rstd * np.abs(z).mean(axis=1, keepdims=True) + np.abs(xh) + 1)
    tol = dict(y=u * np.abs(y) + np.abs(w) * e + 2.0 ** -22 * (np.abs(w * xh) + np.abs(b)) + 1e-30)
    a = np.abs(dy * w)
    c2 = (a * np.abs(xh)).mean(axis=1, keepdims=True)
    ec2 = (a * e).mean(axis=1, keepdims=True) + 2.0 ** -20 * c2
    tol["dx"] = u * np.abs(dx) + rstd * (2.0 ** -20 * (a + a.mean(axis=1, keepdims=True) + c2 * np.abs(xh)) +
                                         e * c2 + ec2 * np.abs(xh)) + 2.0 ** -22 * (0 if dz is None else np.abs(dz))
    tol["dw"] = u * np.abs(dw) + (np.abs(dy) * (e + 2.0 ** -18 * np.abs(xh))).sum(axis=0)
    tol["db"] = u * np.abs(db) + 2.0 ** -18 * np.abs(dy).sum(axis=0)
    if dtype == "fp16":
        tol = {k: v + 2.0 ** -25 for k, v in tol.items()}
    return tol


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n,dim", [(1, 1), (3, 2), (1, 8), (7, 33), (1000, 200), (257, 256), (65, 333), (300, 512),
                                   (4000, 1024), (33, 1000), (9, 2049), (21, 4096), (5, 8200), (3, 16384), (2, 9001)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_matches(n, dim, dtype, residual):
    check_norm(n, dim, dtype, residual)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,dim", [(40001, 64), (39999, 200), (20001, 512), (9800, 1000), (5001, 2048), (4990, 4096),
                                   (40001, 63), (30011, 201), (20011, 333), (10007, 777), (6011, 1999), (3001, 4095)])
def test_norm_of_many_rows(n, dim, dtype):
    """Enough rows that blocks stay for several and load ahead."""
    check_norm(n, dim, dtype, True)


def check_norm(n, dim, dtype, residual):
    rng = np.random.default_rng(n * 7 + dim)
    mk = lambda *s, scale=1.0, shift=0.0: torch.from_numpy(rng.standard_normal(s) * scale + shift).to(DT[dtype]).cuda()  # noqa: E731
    x, w, b, dy = mk(n, dim, shift=3.0), mk(dim, shift=1.0), mk(dim), mk(n, dim)
    r, dz = (mk(n, dim), mk(n, dim)) if residual else (None, None)
    op = pkg.LayerNorm(n, dim, DT[dtype], residual=residual, eps=1e-5)
    y, dx = torch.full_like(x, float("nan")), torch.full_like(x, float("nan"))
    z = torch.full_like(x, float("nan")) if residual else None
    dw, db = torch.full_like(w, float("nan")), torch.full_like(w, float("nan"))
    op.forward(x, w, b, y, residual=r, z=z)
    op.backward(dy, x if z is None else z, w, dx, dw, db, dz=dz)
    torch.cuda.synchronize()
    if residual:
        assert torch.equal(z, (x.float() + r.float()).to(DT[dtype]))
    zz = f64(x if z is None else z)
    ny, _, mean, rstd, xh = ref.norm(zz, f64(w), f64(b), 1e-5)
    ndx, ndw, ndb = ref.norm_gradients(f64(dy), xh, rstd, f64(w), None if dz is None else f64(dz))
    tol = norm_tolerances(dtype, f64(x), zz, xh, rstd, f64(w), f64(b), f64(dy), None if dz is None else f64(dz), ny, ndx,
                          ndw, ndb)
    for name, got, want in (("y", y, ny), ("dx", dx, ndx), ("dw", dw, ndw), ("db", db, ndb)):
        close(name, got, want, tol[name])


def test_norm_unaligned_in_place_and_empty():
    rng = np.random.default_rng(3)
    flat = torch.from_numpy(rng.standard_normal(40 * 64 + 3)).to(torch.bfloat16).cuda()
    x = flat[3:].view(40, 64)          # rows of whole vectors, but a base that is not aligned to one
    w, b = torch.ones(64, dtype=torch.bfloat16, device="cuda"), torch.zeros(64, dtype=torch.bfloat16, device="cuda")
    op = pkg.LayerNorm(40, 64, torch.bfloat16)
    y = torch.empty(40, 64, dtype=torch.bfloat16, device="cuda")
    op.forward(x, w, b, y)
    want = op.forward(x.clone(), w, b, torch.empty_like(y))
    assert torch.allclose(y.float(), want.float(), atol=2.0 ** -6)
    op.forward(x, w, b, x)             # in place
    assert torch.equal(x, y)
    dx, dw, db = torch.empty_like(y), torch.full_like(w, float("nan")), torch.full_like(w, float("nan"))
    none = pkg.LayerNorm(0, 64, torch.bfloat16)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    none.forward(e, w, b, e)
    none.backward(e, e, w, e, dw, db)
    assert (dw == 0).all() and (db == 0).all()
    for dim in (63, 2049, 5000, 5001):
        none = pkg.LayerNorm(0, dim, torch.bfloat16, residual=True)
        e, one = torch.empty(0, dim, dtype=torch.bfloat16, device="cuda"), torch.ones(dim, dtype=torch.bfloat16, device="cuda")
        dw0, db0 = torch.full_like(one, float("nan")), torch.full_like(one, float("nan"))
        none.forward(e, one, one, e.clone(), residual=e, z=e.clone())
        none.backward(e, e, one, e.clone(), dw0, db0)
        assert (dw0 == 0).all() and (db0 == 0).all()
    first = [t.clone() for t in op.backward(y, want, w, dx, dw, db)]
    again = op.backward(y, want, w, dx, dw, db)
    assert all(torch.equal(a, c) for a, c in zip(first, again))


@pytest.mark.parametrize("offsets", [(1, 1, 1, 1), (3, 3, 3, 3), (1, 2, 0, 5)])
@pytest.mark.parametrize("dim", [63, 1001, 2500])
def test_norm_of_many_unaligned_rows(dim, offsets):
    """Tensors that start anywhere: alike modulo 16 bytes, and not."""
    n = 20001
    rng = np.random.default_rng(dim)
    w, b = (torch.from_numpy(rng.standard_normal(dim)).to(torch.float16).cuda() for _ in range(2))

    def tensor(off, values=None):
        flat = torch.full((n * dim + off + 8,), float("nan"), dtype=torch.float16, device="cuda")
        t = flat[off:off + n * dim].view(n, dim)
        if values is not None:
            t.copy_(values)
        return flat, t
    values = torch.randn(n, dim, device="cuda")
    _, x = tensor(offsets[0], values)
    _, dy = tensor(offsets[1], values.flip(0))
    fy, y = tensor(offsets[2])
    fdx, dx = tensor(offsets[3])
    op = pkg.LayerNorm(n, dim, torch.float16)
    dw, db = torch.empty_like(w), torch.empty_like(w)
    op.forward(x, w, b, y)
    op.backward(dy, x, w, dx, dw, db)
    al = {k: t.contiguous().clone() for k, t in (("x", x), ("dy", dy))}
    y2, dx2, dw2, db2 = torch.empty_like(al["x"]), torch.empty_like(al["x"]), torch.empty_like(w), torch.empty_like(w)
    pick = slice(0, 300)                       # few rows go another way: the same values up to rounding
    few = pkg.LayerNorm(300, dim, torch.float16)
    few.forward(al["x"][pick], w, b, y2[pick])
    few.backward(al["dy"][pick], al["x"][pick], w, dx2[pick], dw2, db2)
    assert torch.allclose(y[pick].float(), y2[pick].float(), atol=2.0 ** -8, rtol=2.0 ** -9)
    assert torch.allclose(dx[pick].float(), dx2[pick].float(), atol=2.0 ** -8, rtol=2.0 ** -9)
    for flat, off in ((fy, offsets[2]), (fdx, offsets[3])):   # nothing around them was written
        assert torch.isnan(flat[:off]).all() and torch.isnan(flat[off + n * dim:]).all() and not torch.isnan(flat[off:off + n * dim]).any()
    zz, g = f64(x), f64(dy)
    ny, _, _, rstd, xh = ref.norm(zz, f64(w), f64(b), 1e-5)
    ndx, ndw, ndb = ref.norm_gradients(g, xh, rstd, f64(w))
    tol = norm_tolerances("fp16", zz, zz, xh, rstd, f64(w), f64(b), g, None, ny, ndx, ndw, ndb)
    for name, got, want in (("y", y, ny), ("dx", dx, ndx), ("dw", dw, ndw), ("db", db, ndb)):
        close(name, got, want, tol[name])


@pytest.mark.parametrize("n,dim,dtype,residual", [(16390, 1031, "bf16", False), (16387, 1466, "fp16", True), (16391, 517, "fp32", True),
                                                  (25, 2051, "bf16", True), (1, 2055, "fp16", False), (2500, 3999, "fp16", True),
                                                  (70, 7001, "bf16", False), (33, 2049, "fp32", False), (3, 4086, "fp32", True)])
def test_norm_of_shifted_rows(n, dim, dtype, residual):
    """Rows whose pitch is no multiple of 16 bytes, long enough to be read in aligned pieces all the same."""
    check_norm(n, dim, dtype, residual)


def test_norm_of_shifted_rows_stays_in_them():
    """In place, between guards, and beside a row of NaN: the neighbours' values are read with a row but not used."""
    n, dim = 203, 2053
    t = lambda: torch.randn(n, dim, device="cuda").to(torch.float16)  # noqa: E731
    x, r, dy, dz = t(), t(), t(), t()
    x[77] = float("nan")
    dy[101, 0] = float("inf")
    w, b = torch.randn(2, dim, device="cuda").to(torch.float16)
    op = pkg.LayerNorm(n, dim, torch.float16, residual=True)
    z, y, dx, dw, db = t(), t(), t(), torch.empty_like(w), torch.empty_like(w)
    op.forward(x, w, b, y, residual=r, z=z)
    op.backward(dy, z, w, dx, dw, db, dz=dz)
    good = torch.ones(n, dtype=torch.bool, device="cuda")
    good[77] = False
    assert not torch.isnan(y[good]).any() and torch.isnan(y[77]).all()
    good[101] = False
    assert torch.isfinite(dx[good]).all()
    guarded = []
    for v in (x, dy):
        flat = torch.full((8 + n * dim + 9,), 7.0, dtype=torch.float16, device="cuda")
        flat[8:8 + n * dim].copy_(v.flatten())
        guarded.append((flat, flat[8:8 + n * dim].view(n, dim)))
    (fx, gx), (fdy, gdy) = guarded
    op.forward(gx, w, b, gx, residual=r, z=r)              # y over x, z over the residual
    assert torch.equal(gx.nan_to_num(), y.nan_to_num()) and torch.equal(r.nan_to_num(), z.nan_to_num())
    op.backward(gdy, z, w, gdy, dw, db, dz=dz)             # dx over dy
    assert torch.equal(gdy.nan_to_num(), dx.nan_to_num())
    for flat in (fx, fdy):
        assert (flat[:8] == 7).all() and (flat[8 + n * dim:] == 7).all()


def test_norm_rows_that_hold_no_number():
    """A row with an infinity or NaN spoils itself and the weight's gradient, no other row."""
    x = torch.randn(10, 96, device="cuda")
    x[3, 5] = float("nan")
    x[7, 1] = float("inf")
    w, b = torch.ones(96, device="cuda"), torch.zeros(96, device="cuda")
    y = torch.empty_like(x)
    pkg.LayerNorm(10, 96, torch.float32).forward(x, w, b, y)
    fine = [i for i in range(10) if i not in (3, 7)]
    assert torch.isfinite(y[fine]).all() and torch.isnan(y[3]).all()


def test_example_runs_them_together():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "read_graph.py")
    spec = importlib.util.spec_from_file_location("read_graph", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses, dx = m.read_graph(scale=10, edges=6000, steps=20, say=lambda *_: None)
    assert losses[-1] < 0.9 * losses[0] and torch.isfinite(dx.float()).all()
