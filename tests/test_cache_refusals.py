"""The 8-bit node cache, attention over it and the head norm on the host: what
the calls refuse, and the references they are tested against (no GPU)."""
import ctypes
from decimal import Decimal, localcontext

import numpy as np
import pytest

import cache_ref as ref
from test_reader_host import Card
from test_reader_refusals import EINVAL, ENOMEM, ERANGE, P, _numeric, attn

K = pytest.importorskip("compressed_graph_spmv_gb300.k2t")
torch = pytest.importorskip("torch")
import compressed_graph_spmv_gb300 as pkg  # noqa: E402


def struct(cls, base, kw):
    a = cls()
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return a


def cache(**kw):
    return struct(K.Cache, dict(dtype=K.BF16, n_kv_heads=2, head_dim=64, n_nodes=100, k=P, v=P, k_scale=P, v_scale=P, first=3, count=20,
                                x_k=P, x_v=P, xk_row=128, xk_head=64, xv_row=128, xv_head=64), kw)


def head(**kw):
    return struct(K.HeadNormArgs, dict(dtype=K.BF16, n_heads=4, head_dim=64, rotary_dim=64, n_rows=10, eps=1e-6, x=P, weight=P, positions=P,
                                       y=P, x_row=256, x_head=64, y_row=256, y_head=64, dy=P, dx=P, dweight=P, dy_row=256, dy_head=64,
                                       dx_row=256, dx_head=64), kw)


CACHE = [(dict(n_kv_heads=0), EINVAL), (dict(head_dim=0), EINVAL), (dict(head_dim=60), EINVAL), (dict(head_dim=136), ERANGE),
         (dict(n_kv_heads=65536), ERANGE), (dict(n_nodes=1 << 31), ERANGE), (dict(k=None), EINVAL), (dict(v=None), EINVAL),
         (dict(k_scale=None), EINVAL), (dict(v_scale=None), EINVAL), (dict(k=P + 8), EINVAL), (dict(v=P + 4), EINVAL),
         (dict(k_scale=P + 1), EINVAL), (dict(v_scale=P + 2), EINVAL), (dict(reserved=1), EINVAL)]


@pytest.mark.parametrize("kw,status", CACHE + [
    (dict(dtype=3), EINVAL), (dict(x_k=None), EINVAL), (dict(x_v=None), EINVAL), (dict(x_k=P + 8), EINVAL), (dict(xk_row=132), EINVAL),
    (dict(xv_head=60), EINVAL), (dict(xv_row=-128), EINVAL), (dict(xk_head=1 << 38), EINVAL), (dict(first=81), ERANGE),
    (dict(first=101, count=0), ERANGE), (dict(count=101), ERANGE), (dict(first=1 << 63, count=1 << 63), ERANGE), (dict(nodes=P + 2), EINVAL),
])
def test_cache_refuses(kw, status):
    lib = K.load()
    for call in (lib.k2t_cache_write, lib.k2t_cache_read):
        assert call(ctypes.byref(cache(**kw)), None) == status
        assert call(None, None) == EINVAL


def test_cache_refuses_of_one_call():
    lib = K.load()
    assert lib.k2t_cache_write(ctypes.byref(cache(nodes=P)), None) == EINVAL
    assert lib.k2t_cache_read(ctypes.byref(cache(nodes=P)), None) == ERANGE               # first is 3
    assert lib.k2t_cache_read(ctypes.byref(cache(nodes=P, first=0, count=K.ATTN_MAX_NODES + 1)), None) == ERANGE
    for kw in (dict(xk_row=0), dict(xv_head=0), dict(xk_row=56, xk_head=8)):              # rows that overlap
        assert lib.k2t_cache_read(ctypes.byref(cache(**kw)), None) == EINVAL
    # nothing to do, whatever the pointers
    for call in (lib.k2t_cache_write, lib.k2t_cache_read):
        assert call(ctypes.byref(cache(count=0, x_k=None, x_v=None)), None) == 0
        assert call(ctypes.byref(cache(n_nodes=0, first=0, count=0, k=None, v=None, k_scale=None, v_scale=None)), None) == 0


@pytest.mark.parametrize("kw,status", CACHE + [(dict(n_kv_heads=4), EINVAL), (dict(head_dim=72), EINVAL), (dict(n_nodes=99), ERANGE)])
def test_cached_attention_refuses_caches(kw, status):
    a, c = attn(k=None, v=None), cache(**kw)
    assert K.load().k2t_cached_attn_forward(ctypes.byref(a), ctypes.byref(c), P, 1 << 40, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=K.FP32), EINVAL), (dict(n_heads=5), EINVAL), (dict(head_dim=60), EINVAL), (dict(n_heads=34), ERANGE),
    (dict(n_sources=33), ERANGE), (dict(edges=(1, 2, 3)), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(q=None), EINVAL),
    (dict(out=None), EINVAL), (dict(lse=None), EINVAL), (dict(hops=None), EINVAL), (dict(bias=None), EINVAL), (dict(q=P + 8), EINVAL),
    (dict(out_row=250), EINVAL), (dict(out_row=0), EINVAL), (dict(n_queries=5), ERANGE),
])
def test_cached_attention_refuses(kw, status):
    a, c = attn(**kw), cache()
    assert K.load().k2t_cached_attn_forward(ctypes.byref(a), ctypes.byref(c), P, 1 << 40, None) == status


def test_cached_attention_work():
    lib = K.load()
    c = cache()
    need = lib.k2t_cached_attn_work_bytes(ctypes.byref(attn()))
    assert need > 0 and lib.k2t_cached_attn_work_bytes(ctypes.byref(attn(head_dim=60))) == 0
    assert lib.k2t_cached_attn_forward(ctypes.byref(attn()), ctypes.byref(c), P, 0, None) == ENOMEM
    assert lib.k2t_cached_attn_forward(ctypes.byref(attn()), ctypes.byref(c), None, need, None) == EINVAL
    assert lib.k2t_cached_attn_forward(ctypes.byref(attn()), ctypes.byref(c), P + 4, need, None) == EINVAL
    assert lib.k2t_cached_attn_forward(ctypes.byref(attn()), None, P, need, None) == EINVAL
    assert lib.k2t_cached_attn_forward(None, ctypes.byref(c), P, need, None) == EINVAL
    assert lib.k2t_cached_attn_forward(ctypes.byref(attn(n_queries=0, q=None, out=None, lse=None)), ctypes.byref(c), P, need, None) == 0


def test_cached_attention_work_is_enough_for_fewer_nodes():
    """What the call with n nodes needs (it says ENOMEM before it launches) is never more than what was asked for n_nodes."""
    lib = K.load()
    for T, hq, hkv, most in ((1, 4, 4, 100000), (32, 16, 4, 50000), (900, 8, 8, 20000), (300, 4, 1, 5000), (7, 2, 1, 1)):
        size = dict(n_queries=T, n_heads=hq, n_kv_heads=hkv, n_sources=0, n_buckets=0, bias=None, edges=(), out_row=hq * 64)
        need = lib.k2t_cached_attn_work_bytes(ctypes.byref(attn(n_nodes=most, **size)))
        for n in {0, 1, 127, 128, 129, 1000, 5000, 19456, 19457, 38912, 49999, most} & set(range(most + 1)):
            assert lib.k2t_attn_work_bytes(ctypes.byref(attn(n_nodes=n, **size)), 0) <= need


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), EINVAL), (dict(n_heads=0), EINVAL), (dict(head_dim=0), EINVAL), (dict(head_dim=60), EINVAL), (dict(head_dim=264), ERANGE),
    (dict(rotary_dim=3), EINVAL), (dict(rotary_dim=66), EINVAL), (dict(n_heads=65536), ERANGE), (dict(n_rows=(1 << 32) + 1), ERANGE),
    (dict(eps=0.0), EINVAL), (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(flags=2), EINVAL), (dict(x=None), EINVAL),
    (dict(x=P + 8), EINVAL), (dict(x_row=252), EINVAL), (dict(x_head=-64), EINVAL), (dict(weight=P + 8), EINVAL), (dict(positions=P + 2), EINVAL),
])
def test_head_norm_refuses(kw, status):
    lib = K.load()
    assert lib.k2t_head_norm_forward(ctypes.byref(head(**kw)), None) == status
    assert lib.k2t_head_norm_backward(ctypes.byref(head(**kw)), P, 1 << 40, None) == status


def test_head_norm_refuses_of_one_call():
    lib = K.load()
    for kw in (dict(y=None), dict(y=P + 8), dict(y_row=4), dict(y_row=0), dict(y_head=56)):
        assert lib.k2t_head_norm_forward(ctypes.byref(head(**kw)), None) == EINVAL
    for kw in (dict(dy=None), dict(dx=None), dict(dx=P + 8), dict(dy_head=4), dict(dx_row=0), dict(dx_head=56), dict(dweight=None),
               dict(weight=None), dict(dweight=P + 8)):
        assert lib.k2t_head_norm_backward(ctypes.byref(head(**kw)), P, 1 << 40, None) == EINVAL
    need = lib.k2t_head_norm_work_bytes(ctypes.byref(head()))
    assert need > 0 and lib.k2t_head_norm_work_bytes(ctypes.byref(head(head_dim=60))) == 0
    assert lib.k2t_head_norm_backward(ctypes.byref(head()), P, need - 1, None) == ENOMEM
    assert lib.k2t_head_norm_backward(ctypes.byref(head()), None, need, None) == EINVAL
    assert lib.k2t_head_norm_backward(ctypes.byref(head()), P + 4, need, None) == EINVAL
    assert lib.k2t_head_norm_forward(ctypes.byref(head(n_rows=0, x=None, y=None)), None) == 0
    assert lib.k2t_head_norm_backward(ctypes.byref(head(n_rows=0, x=None, dy=None, dx=None, weight=None, dweight=None)), None, 0, None) == 0


def test_rates():
    lib = K.load()
    rates = (ctypes.c_uint64 * 128)()
    for base in (1.0, 10000.0, 5e5, 1e30):
        for rotary in (2, 10, 64, 256):
            assert lib.k2t_head_rates(base, rotary, rates) == 0
            for m in range(rotary // 2):
                want = base ** (-2 * m / rotary) / (2 * np.pi) * 2.0 ** 64
                assert abs(rates[m] - want) <= 2 + want * 2.0 ** -50
    for base, rotary in ((0.5, 64), (float("nan"), 64), (float("inf"), 64), (1e4, 3), (1e4, 258)):
        assert lib.k2t_head_rates(base, rotary, rates) == EINVAL
    assert lib.k2t_head_rates(1e4, 64, None) == EINVAL


def test_struct_sizes_match_the_header():
    assert ctypes.sizeof(K.Cache) == 128 and ctypes.sizeof(K.HeadNormArgs) == 1176


def test_python_refusals():
    bf16 = torch.bfloat16
    for size in ((-1, 1, 64), (4, 0, 64), (4, 1, 60), (4, 1, 136), (4, 1, 0), (1 << 31, 1, 8)):
        with pytest.raises(ValueError):
            pkg.NodeCache(*size, bf16, device="cpu")
    with pytest.raises(TypeError):
        pkg.NodeCache(4, 1, 64, torch.float64, device="cpu")
    c = pkg.NodeCache(100, 2, 72, bf16, device="cpu")
    assert c.k.shape == (2, 100, 80) and c.k.dtype is torch.float8_e4m3fn and c.v_scale.shape == (2, 16) and not c.v_scale.any()
    x = torch.zeros(5, 2, 72, dtype=bf16)
    with pytest.raises(ValueError):                      # host tensors
        c.write(x, x)
    # a cache as it would be on a card, which no refused call reads
    c._here, c._current, c.k = (lambda: 0), (lambda d: 0), Card(2, 100, 80)
    c._streams = {0}
    calls = []
    c._write = c._read = lambda ref, st: calls.append((c._a.first, c._a.count, c._a.nodes)) or 0
    k = Card(5, 2, 72)
    c.write(k, k, first=7)
    c.read(k, k, nodes=Card(5, dtype=torch.int32))
    assert calls == [(7, 5, None), (0, 5, P)]
    for bad, error in ((dict(v=Card(4, 2, 72)), ValueError), (dict(v=Card(5, 2, 64)), ValueError), (dict(v=Card(5, 2, 72, dtype=torch.float16)), TypeError),
                       (dict(v=Card(5, 2, 72, device=1)), ValueError), (dict(k=Card(5, 2, 72, device=1)), ValueError), (dict(first=-1), ValueError)):
        with pytest.raises(error):
            c.write(**{**dict(k=k, v=k), **bad})
    for nodes in (Card(4, dtype=torch.int32), Card(5, dtype=torch.int64), Card(5, dtype=torch.int32, device=1)):
        with pytest.raises((ValueError, TypeError)):
            c.read(k, k, nodes=nodes)
    op = pkg.CachedAttention(3, 100, 4, 2, 72, bf16, sources=3, edges=[0, 1])
    op._here = op._current = lambda *a: 0
    op._forward = lambda *a: calls.append(op._a.n_nodes) or 0
    op._buffers[0].at, op._buffers[0].last = P, 0
    q, lse, hops, bias = Card(3, 4, 72), Card(3, 4, dtype=torch.float32), Card(100, 3, dtype=torch.int32), Card(4, 2)
    op.forward(q, c, q, lse, hops=hops, bias=bias, nodes=17)
    op.forward(q, c, q, lse, hops=hops, bias=bias)
    assert calls[2:] == [17, 100]
    good = dict(q=q, cache=c, out=q, lse=lse, hops=hops, bias=bias)
    for bad in (dict(nodes=101), dict(nodes=-1), dict(hops=None), dict(hops=Card(99, 3, dtype=torch.int32)), dict(bias=Card(4, 3)),
                dict(q=Card(3, 4, 72, device=1)), dict(lse=Card(3, 4, dtype=torch.float32, device=1)), dict(out=Card(3, 2, 72))):
        with pytest.raises(ValueError):
            op.forward(**{**good, **bad})
    with pytest.raises(TypeError):
        pkg.CachedAttention(1, 1, 1, 1, 64, torch.float32)
    for kw in (dict(rotary_dim=3), dict(rotary_dim=300), dict(base=0.0), dict(base=float("nan"))):
        with pytest.raises(ValueError):
            pkg.HeadNorm(4, 2, 64, bf16, **kw)
    n = pkg.HeadNorm(4, 2, 64, bf16)
    x, w = torch.zeros(4, 2, 64, dtype=bf16), torch.zeros(64, dtype=bf16)
    with pytest.raises(ValueError):
        n.forward(x, w, x)
    n._here = n._current = lambda *a: 0
    n._forward = n._backward = lambda *a: 0
    n._work.at, n._work.last = P, 0
    x, w, at = Card(4, 2, 64), Card(64), Card(4, dtype=torch.int32)
    n.forward(x, w, x, positions=at)
    n.backward(x, x, w, x, w)
    for bad in (dict(weight=Card(32)), dict(positions=Card(3, dtype=torch.int32)), dict(y=Card(4, 2, 64, device=1)), dict(x=Card(4, 2, 64, device=1)),
                dict(weight=Card(64, device=1))):
        with pytest.raises(ValueError):
            n.forward(**{**dict(x=x, weight=w, y=x), **bad})


def test_reference_rounding():
    """All 256 bytes stand for themselves, and values between two go to the nearer, or the even one."""
    held = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(ref.to_e4m3(held), held)
    x = np.random.default_rng(1).uniform(-448, 448, size=20000) * 2.0 ** np.random.default_rng(2).integers(-20, 1, size=20000)
    fine = np.unique(held[np.isfinite(held)])
    near = np.abs(x[:, None] - fine[None]).min(axis=1)
    assert np.array_equal(np.abs(ref.to_e4m3(x) - x), near)
    border = (fine[1:] + fine[:-1]) / 2
    even = torch.from_numpy(border).to(torch.float32).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(ref.to_e4m3(border), even)
    assert [ref.exponent_for(t) for t in (0.0, 448.0, 449.0, 224.0, 225.0, 1e30)] == [-64, 0, 1, -1, 0, 63]


@pytest.mark.parametrize("paired", [False, True])
def test_reference_head_gradients_against_differences(paired):
    """Central differences with step 1e-6 of sums of about 1: error about 1e-10 from the step, 1e-10 from rounding."""
    rng = np.random.default_rng(3)
    x, dy, w = rng.standard_normal((3, 2, 8)), rng.standard_normal((3, 2, 8)), rng.standard_normal(8)
    angle = ref.angles([0, 5, -3], 6)
    f = lambda: float((ref.head_norm(x, w, angle, 6, paired, 1e-3)[0] * dy).sum())  # noqa: E731
    dx, dw, _, _ = ref.head_norm_gradients(dy, x, w, angle, 6, paired, 1e-3)
    assert np.allclose(dx, _numeric(f, x), atol=1e-7, rtol=0) and np.allclose(dw, _numeric(f, w), atol=1e-7, rtol=0)


@pytest.mark.parametrize("base", [1e4, 5e5, 1e6])
@pytest.mark.parametrize("rotary", [2, 64, 96, 256])
def test_rates_hold_at_far_positions(base, rotary):
    """A rate is right to its last bits, so that a far position turns by what it should.

    A rate is rounded to a step of 2 units of 2^-64 turns: at most 1.  The power and the product
    before it are held in 64 bits: 4.4 steps of 2^-64 relative to at most 0.16 * 2^64, 0.7 units.
    """
    lib = K.load()
    rates = (ctypes.c_uint64 * 128)()
    assert lib.k2t_head_rates(base, rotary, rates) == 0
    with localcontext() as c:
        c.prec = 60
        for m in range(rotary // 2):
            exact = Decimal(base) ** (Decimal(-2 * m) / rotary) * 2 ** 64 / (2 * Decimal("3.14159265358979323846264338327950288419716939937510582"))
            assert abs(rates[m] - exact) <= 2
