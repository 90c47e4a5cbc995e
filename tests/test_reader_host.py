"""Graph-reading calls on the host: flags, layouts of outputs, threads, devices (no GPU)."""
import ctypes
import threading
import time

import pytest

from test_reader_refusals import ENOMEM, EINVAL, P, attn, norm

K = pytest.importorskip("compressed_graph_spmv_gb300.k2t")
torch = pytest.importorskip("torch")
import compressed_graph_spmv_gb300 as pkg  # noqa: E402
from compressed_graph_spmv_gb300 import reader  # noqa: E402


def test_norm_flags():
    lib = K.load()
    for flags in (2, 3, 1 << 31):
        a = norm(flags=flags)
        assert lib.k2t_norm_work_bytes(ctypes.byref(a)) == 0
        assert lib.k2t_norm_forward(ctypes.byref(a), None) == EINVAL
        assert lib.k2t_norm_backward(ctypes.byref(a), P, 1 << 40, None) == EINVAL
    # statistics formed again: neither is needed, so that the work buffer is what is refused
    a = norm(flags=K.NORM_FORM_STATS, mean=None, rstd=None)
    assert lib.k2t_norm_backward(ctypes.byref(a), P, 0, None) == ENOMEM
    assert lib.k2t_norm_forward(ctypes.byref(a), None) == EINVAL


class Card:
    """A tensor as the calls see one, on a card that is not there."""

    def __init__(self, *shape, dtype=torch.bfloat16, at=P, device=0, strides=None):
        self.shape, self.dtype, self.ndim, self.at, self.device_index = torch.Size(shape), dtype, len(shape), at, device
        self.is_cuda, self.strides = True, strides or torch.empty(shape, device="meta").stride()

    def get_device(self):
        return self.device_index

    def is_contiguous(self):
        return True

    def stride(self):
        return self.strides

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return self.at


def attention(monkeypatch, call):
    """An attention object whose C calls are `call(struct)`, and its tensors at addresses from `at` on."""
    op = pkg.HopAttention(2, 3, 2, 1, 64, torch.bfloat16, sources=2, edges=[0, 1])
    fake = lambda ref, work, size, stream: call(op._a)  # noqa: E731
    op._forward = op._backward = fake
    for b in op._buffers:
        b.at, b.last = P, 0
    op._current, op._here = (lambda device: 0), (lambda: 0)

    def tensors(at, device=0):
        shapes = dict(q=(2, 2, 64), k=(3, 1, 64), v=(3, 1, 64), out=(2, 2, 64), lse=(2, 2), hops=(3, 2), bias=(2, 2), dout=(2, 2, 64),
                      dq=(2, 2, 64), dk=(3, 1, 64), dv=(3, 1, 64), dbias=(2, 2))
        types = dict(lse=torch.float32, hops=torch.int32)
        return {x: Card(*s, dtype=types.get(x, torch.bfloat16), at=at + i * 4096, device=device) for i, (x, s) in enumerate(shapes.items())}
    return op, tensors


def forward(op, t):
    op.forward(t["q"], t["k"], t["v"], t["out"], t["lse"], hops=t["hops"], bias=t["bias"])


def backward(op, t):
    op.backward(t["dout"], t["q"], t["k"], t["v"], t["out"], t["lse"], t["dq"], t["dk"], t["dv"], dbias=t["dbias"], hops=t["hops"],
                bias=t["bias"])


def in_threads(jobs):
    errors = []

    def body(job):
        try:
            job()
        except Exception as e:   # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=body, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


@pytest.mark.parametrize("call", [forward, backward])
def test_threads_share_an_attention_object(monkeypatch, call):
    """What a C call reads does not change while it runs, and no two run at once."""
    inside, seen = [], []

    def c_call(a):
        inside.append(1)
        before = bytes(a)
        time.sleep(0.02)
        seen.append((len(inside), bytes(a) == before, a.q, a.k))
        inside.pop()
        return 0
    op, tensors = attention(monkeypatch, c_call)
    sets = [tensors(P * (i + 1)) for i in range(4)]
    in_threads([lambda t=t: call(op, t) for t in sets])
    assert all(n == 1 and same for n, same, _, _ in seen)
    assert sorted((q, k) for _, _, q, k in seen) == sorted((t["q"].at, t["k"].at) for t in sets)


def test_threads_share_a_norm_object():
    op = pkg.LayerNorm(4, 8, torch.float32, device="cpu")        # where its buffers are
    seen = []

    def c_call(*_):
        before = bytes(op._a)
        time.sleep(0.02)
        seen.append((bytes(op._a) == before, op._a.x if op._a.flags == 0 else op._a.dy, op._a.weight))
        return 0
    op._forward = op._backward = c_call
    op._current = op._own._current = op._work._current = lambda device: 0
    op._here = lambda: 0

    def job(i):
        x, w = Card(4, 8, dtype=torch.float32, at=P * i), Card(8, dtype=torch.float32, at=P * i + 64)
        return (lambda: op.forward(x, w, None, x)) if i % 2 else (lambda: op.backward(x, x, w, x, w))
    in_threads([job(i) for i in range(1, 7)])
    assert all(same for same, _, _ in seen) and sorted((x, w) for _, x, w in seen) == [(P * i, P * i + 64) for i in range(1, 7)]


@pytest.mark.parametrize("call,names", [(forward, "q k v out lse hops bias"), (backward, "q k v out lse hops bias dout dq dk dv dbias")])
def test_attention_refuses_tensors_of_several_devices(monkeypatch, call, names):
    calls = []
    op, tensors = attention(monkeypatch, lambda a: calls.append(1) or 0)
    call(op, tensors(P))
    for name in names.split():
        t = tensors(P)
        t[name].device_index = 1
        with pytest.raises(ValueError, match="device"):
            call(op, t)
    with pytest.raises(ValueError, match="the object is on device 0"):
        call(op, tensors(P, device=1))
    op._here = lambda: 1
    with pytest.raises(ValueError, match="current"):
        call(op, tensors(P))
    assert len(calls) == 1
    op, tensors = attention(monkeypatch, lambda a: calls.append(1) or 0)
    op.device = "cuda:1"
    with pytest.raises(ValueError, match="the object is on device 1"):
        call(op, tensors(P))


def test_norm_refuses_tensors_of_several_devices():
    op = pkg.LayerNorm(4, 8, torch.float32, residual=True)
    op._forward = op._backward = lambda *a: 0
    op._here = op._current = lambda *a: 0
    for b in (op._own, op._work):
        b.at, b.last, b._streams = P, 0, {0}
        b.tensor, op._own_at = Card(1), (P, P)
    shapes = dict(x=(4, 8), residual=(4, 8), weight=(8,), bias=(8,), y=(4, 8), z=(4, 8), mean=(4,), rstd=(4,))
    back = dict(dy=(4, 8), z=(4, 8), weight=(8,), dx=(4, 8), dweight=(8,), dbias=(8,), dz=(4, 8), mean=(4,), rstd=(4,))
    for call, wants in ((op.forward, shapes), (op.backward, back)):
        for odd in (None, *wants):
            t = {x: Card(*s, dtype=torch.float32, device=int(x == odd)) for x, s in wants.items()}
            if odd is None:
                call(**t)
                continue
            with pytest.raises(ValueError, match="device"):
                call(**t)


def test_rows_of_outputs_that_overlap():
    """Checked for every pair of pitches against the definition; a layout that is taken fails for its work buffer, next."""
    lib = K.load()
    calls = dict(out=lib.k2t_attn_forward, dq=lib.k2t_attn_backward, dk=lib.k2t_attn_backward, dv=lib.k2t_attn_backward)
    refused = taken = 0
    for name, call in calls.items():
        nodes = name in ("dk", "dv")
        for rows, heads in ((4, 4), (1, 4), (3, 2), (4, 2)) if not nodes else ((5, 2), (1, 2), (3, 2)):
            for row in (0, 8, 16, 24, 40, 48, 56, 64, 80):
                for head in (0, 8, 16, 24, 40, 56, 64, 72, 96):
                    kw = {name + "_row": row, name + "_head": head}
                    a = attn(head_dim=16, n_sources=0, n_buckets=0, bias=None, edges=(), n_heads=2 if nodes else heads,
                             n_kv_heads=heads if nodes else 1, n_queries=4 if nodes else rows, n_nodes=rows if nodes else 5, **kw)
                    starts = sorted(i * row + j * head for i in range(rows) for j in range(heads))
                    free = all(b - c >= 16 for c, b in zip(starts, starts[1:]))
                    assert call(ctypes.byref(a), P, 0, None) == (ENOMEM if free else EINVAL), (name, rows, heads, row, head)
                    taken, refused = taken + free, refused + (not free)
    assert taken > 300 and refused > 300
    # very long pitches and very many nodes
    far = dict(n_nodes=K.ATTN_MAX_NODES, n_sources=0, n_buckets=0, bias=None, edges=())
    for kw, status in ((dict(dk_row=(1 << 38) - 8, dk_head=64), ENOMEM), (dict(dk_row=64, dk_head=(1 << 38) - 8), ENOMEM),
                       (dict(dk_row=64, dk_head=1 << 20), EINVAL), (dict(dv_row=0), EINVAL)):
        assert lib.k2t_attn_backward(ctypes.byref(attn(**far, **kw)), P, 0, None) == status, kw
    # inputs may be broadcast
    for kw in (dict(k_row=0, v_head=0), dict(q_row=0, q_head=0), dict(dout_row=0)):
        assert lib.k2t_attn_backward(ctypes.byref(attn(**kw)), P, 0, None) == ENOMEM
