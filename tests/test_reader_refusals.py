"""Graph-reading operators on the host: what the calls refuse, what they need
of memory, and the reference gradients against differences (no GPU)."""
import ctypes

import numpy as np
import pytest

import reader_ref as ref

K = pytest.importorskip("compressed_graph_spmv_gb300.k2t")
import compressed_graph_spmv_gb300 as pkg  # noqa: E402

EINVAL, ERANGE, ENOMEM = -1, -2, -3
P = 1 << 20   # an aligned address that no refused call reads


def attn(**kw):
    a = K.Attn()
    base = dict(dtype=K.BF16, n_queries=4, n_heads=4, n_kv_heads=2, head_dim=64, n_sources=4, n_buckets=3, n_nodes=100,
                scale=0.125, q=P, k=P, v=P, hops=P, bias=P, out=P, lse=P, q_row=256, q_head=64, k_row=128, k_head=64,
                v_row=128, v_head=64, out_row=256, out_head=64, dout=P, dout_row=256, dout_head=64, dq=P, dk=P, dv=P,
                dq_row=256, dq_head=64, dk_row=128, dk_head=64, dv_row=128, dv_head=64, dbias=P)
    edges = kw.pop("edges", (0, 1, 2))
    base.update(kw)
    for k, v in base.items():
        setattr(a, k, v)
    for i, e in enumerate(edges):
        a.edges[i] = e
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=K.FP32), EINVAL), (dict(dtype=7), EINVAL), (dict(n_heads=0), EINVAL), (dict(n_kv_heads=0), EINVAL),
    (dict(n_heads=5), EINVAL), (dict(head_dim=0), EINVAL), (dict(head_dim=60), EINVAL), (dict(head_dim=136), ERANGE),
    (dict(n_heads=34), ERANGE), (dict(n_sources=33), ERANGE), (dict(n_buckets=65), ERANGE),
    (dict(n_nodes=(1 << 31)), ERANGE), (dict(n_queries=1 << 31), ERANGE), (dict(n_sources=0, hops=None), EINVAL),
    (dict(edges=(1, 2, 3)), EINVAL), (dict(edges=(0, 2, 2)), EINVAL), (dict(scale=float("nan")), EINVAL),
    (dict(q=None), EINVAL), (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(out=None), EINVAL),
    (dict(lse=None), EINVAL), (dict(hops=None), EINVAL), (dict(bias=None), EINVAL), (dict(n_buckets=0), EINVAL),
    (dict(q=P + 8), EINVAL), (dict(k_row=132), EINVAL), (dict(v_head=60), EINVAL), (dict(out_row=250), EINVAL), (dict(k_row=-128), EINVAL),
    (dict(n_queries=5), ERANGE),
])
def test_attention_refuses(kw, status):
    lib = K.load()
    a = attn(**kw)
    for call in (lib.k2t_attn_forward, lib.k2t_attn_backward):
        assert call(ctypes.byref(a), P, 1 << 40, None) == status


@pytest.mark.parametrize("kw", [dict(dout=None), dict(dq=None), dict(dk=None), dict(dv=None), dict(dbias=None),
                                dict(dout=P + 2), dict(dq_row=4), dict(dk_head=3), dict(dv=P + 4)])
def test_attention_backward_refuses(kw):
    a = attn(**kw)
    assert K.load().k2t_attn_backward(ctypes.byref(a), P, 1 << 40, None) == EINVAL


def test_attention_work():
    lib = K.load()
    a = attn()
    need = lib.k2t_attn_work_bytes(ctypes.byref(a), 1)
    assert need > 0 and lib.k2t_attn_work_bytes(ctypes.byref(attn(head_dim=60)), 1) == 0
    assert lib.k2t_attn_backward(ctypes.byref(a), P, need - 1, None) == ENOMEM
    assert lib.k2t_attn_backward(ctypes.byref(a), None, need, None) == EINVAL
    assert lib.k2t_attn_backward(ctypes.byref(a), P + 4, need, None) == EINVAL
    assert lib.k2t_attn_forward(None, None, 0, None) == EINVAL
    # no query: nothing to do, whatever the pointers
    assert lib.k2t_attn_forward(ctypes.byref(attn(n_queries=0, q=None, out=None, lse=None)), P, 1 << 40, None) == 0


def norm(**kw):
    a = K.Norm()
    base = dict(dtype=K.BF16, dim=64, n_rows=10, eps=1e-5, x=P, weight=P, bias=P, y=P, z=P + 4096, mean=P, rstd=P, dy=P,
                dx=P, dweight=P, dbias=P)
    base.update(kw)
    for k, v in base.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), EINVAL), (dict(dim=0), ERANGE), (dict(dim=16385), ERANGE), (dict(eps=0.0), EINVAL),
    (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(n_rows=(1 << 32) + 1), ERANGE),
    (dict(weight=None), EINVAL), (dict(mean=None), EINVAL), (dict(rstd=None), EINVAL), (dict(weight=P + 1), EINVAL),
])
def test_norm_refuses(kw, status):
    lib = K.load()
    a = norm(**kw)
    assert lib.k2t_norm_forward(ctypes.byref(a), None) == status
    assert lib.k2t_norm_backward(ctypes.byref(a), P, 1 << 40, None) == status


def test_norm_refuses_tensors():
    lib = K.load()
    for kw in (dict(x=None), dict(y=None), dict(x=P + 1), dict(residual=P, z=None), dict(residual=P, y=P, z=P)):
        assert lib.k2t_norm_forward(ctypes.byref(norm(**kw)), None) == EINVAL
    for kw in (dict(z=None), dict(dy=None), dict(dx=None), dict(dweight=None), dict(dy=P + 1)):
        assert lib.k2t_norm_backward(ctypes.byref(norm(**kw)), P, 1 << 40, None) == EINVAL
    need = lib.k2t_norm_work_bytes(ctypes.byref(norm()))
    assert need >= 2 * 64 * 4
    assert lib.k2t_norm_backward(ctypes.byref(norm()), P, need - 1, None) == ENOMEM
    assert lib.k2t_norm_backward(ctypes.byref(norm()), None, need, None) == EINVAL
    assert lib.k2t_norm_forward(ctypes.byref(norm(n_rows=0, x=None, y=None, mean=None, rstd=None)), None) == 0


def test_struct_sizes_match_the_header():
    assert ctypes.sizeof(K.Attn) == 336 and ctypes.sizeof(K.Norm) == 128


def test_python_refusals():
    torch = pytest.importorskip("torch")
    with pytest.raises(TypeError):
        pkg.HopAttention(1, 1, 1, 1, 64, torch.float32)
    with pytest.raises(ValueError):
        pkg.HopAttention(1, 1, 1, 1, 64, torch.bfloat16, sources=1, edges=[0, 256])
    with pytest.raises(ValueError):
        pkg.hop_edges(0)
    with pytest.raises(ValueError):
        pkg.hop_edges(40, 20)
    op = pkg.HopAttention(2, 3, 2, 1, 64, torch.bfloat16)
    q, kv = torch.zeros(2, 2, 64, dtype=torch.bfloat16), torch.zeros(3, 1, 64, dtype=torch.bfloat16)
    lse = torch.zeros(2, 2)
    with pytest.raises(ValueError):   # host tensors
        op.forward(q, kv, kv, q, lse)
    with pytest.raises(ValueError):   # a shape
        op.forward(q[:1], kv, kv, q, lse)
    with pytest.raises(TypeError):
        op.forward(q.half(), kv, kv, q, lse)
    n = pkg.LayerNorm(4, 8, torch.float32, residual=True, device="cpu")
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        n.forward(x, x[0], x[0], x)


def test_hop_edges():
    for n in (1, 2, 3, 16, 33, 64):
        for top in (n - 1, 64, 255):
            if top < n - 1:
                continue
            e = pkg.hop_edges(n, top)
            assert len(e) == n and e[0] == 0 and all(a < b for a, b in zip(e, e[1:])) and e[-1] <= max(top, 0)


def _numeric(f, x, step=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + step
        up = f()
        x[i] = keep - step
        g[i] = (up - f()) / (2 * step)
        x[i] = keep
    return g


def test_reference_gradients_against_differences():
    """Central differences with step 1e-6 of sums of about 1: error about 1e-10 from the step, 1e-10 from rounding."""
    rng = np.random.default_rng(1)
    T, n, hq, hkv, d, edges = 3, 7, 4, 2, 8, [0, 1, 3]
    q, k, v = (rng.standard_normal(s) for s in ((T, hq, d), (n, hkv, d), (n, hkv, d)))
    bias, dout = rng.standard_normal((hq, 3)), rng.standard_normal((T, hq, d))
    bias[1, 2] = -np.inf
    hops = rng.integers(-1, 5, size=(n, 2))
    hops[:, 1] = -1
    source = np.array([0, -1, 1])
    table = dict(hops=hops, bias=bias, edges=edges, source=source)
    g = ref.gradients(q, k, v, dout, 0.4, n_buckets=3, **table)
    f = lambda: float((ref.attention(q, k, v, 0.4, **table)[0] * dout).sum())  # noqa: E731
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        assert np.allclose(g[name], _numeric(f, x), atol=1e-7, rtol=0), name
    bias[1, 2] = 0.3
    g = ref.gradients(q, k, v, dout, 0.4, n_buckets=3, **table)
    assert np.allclose(g["dbias"], _numeric(f, bias), atol=1e-7, rtol=0)


def test_reference_norm_gradients_against_differences():
    rng = np.random.default_rng(2)
    x, r, dy, dz = (rng.standard_normal((4, 6)) for _ in range(4))
    w, b = rng.standard_normal(6), rng.standard_normal(6)
    y, z, mean, rstd, xh = ref.norm(x, w, b, 1e-3, r)
    dx, dw, db = ref.norm_gradients(dy, xh, rstd, w, dz)

    def f():
        y, z = ref.norm(x, w, b, 1e-3, r)[:2]
        return float((y * dy).sum() + (z * dz).sum())
    for g, at in ((dx, x), (dx, r), (dw, w), (db, b)):
        assert np.allclose(g, _numeric(f, at), atol=1e-7, rtol=0)
