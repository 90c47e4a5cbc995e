"""The layers of a model that reads a graph, on device tensors: attention of
queries to node states biased by hop distance, layer norm of node states, and
the norm and rotation of each head of queries and keys (``k2t_attn_*``,
``k2t_norm_*`` and ``k2t_head_*`` of ``include/k2t.h``).

As in ``k2t.py``, argument marshalling only.  An object holds the sizes and
the work buffer of one layer; its calls take tensors that the caller owns,
write the output tensors they are given and return them.  Calls of one
object share its buffers: order them on the GPU (one stream, or events).  The
buffers are made on the stream of the call that first needs them; a stream
that a call was given has to outlive the object.
Host threads may call one object; each call queues its kernels together.
"""
from __future__ import annotations

import ctypes
import math
import struct
import threading

from .k2t import (ATTN_MAX_BUCKETS, ATTN_MAX_HOP, BF16, FP16, FP32, HEAD_PAIRED, NORM_FORM_STATS, Attn, HeadNormArgs, Norm, _check,
                  _stream_ptr, load)


def hop_edges(n_buckets: int, max_hop: int = 64) -> list:
    """First hop of each of ``n_buckets`` buckets: one bucket a hop for the
    first half, then growing ones; hops of ``max_hop`` or more share the last."""
    if not 1 <= n_buckets <= ATTN_MAX_BUCKETS:
        raise ValueError("n_buckets must be 1..%d" % ATTN_MAX_BUCKETS)
    if not n_buckets - 1 <= max_hop <= ATTN_MAX_HOP:
        raise ValueError("max_hop must be n_buckets - 1..%d" % ATTN_MAX_HOP)
    half = (n_buckets + 1) // 2
    grown = n_buckets - half
    edges = list(range(half))
    for i in range(1, grown + 1):
        geometric = round(half * (max_hop / half) ** (i / grown))
        edges.append(min(max(edges[-1] + 1, geometric), max_hop - (grown - i)))
    return edges


def _dtype_code(dtype, allowed):
    import torch
    code = {torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32}.get(dtype)
    if code not in allowed:
        raise TypeError("unsupported dtype %s" % dtype)
    return code


def _stream_getter(torch):
    """How a call learns the current stream's address: torch's own short way where it has one (a few hundred
    nanoseconds less than building a stream object, of calls that take microseconds)."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:
        return raw
    return lambda device: torch.cuda.current_stream(device).cuda_stream


def _device_getter(torch):
    """The current device's number, torch's own short way where it has one."""
    return getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _refuse(name, t, shape, dtype, device, last_only):
    """Say what is wrong with a tensor that a call does not take."""
    if t.shape != shape:
        raise ValueError("%s: expected shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.dtype is not dtype:
        raise TypeError("%s: expected %s, got %s" % (name, dtype, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s: expected a CUDA tensor" % name)
    if t.get_device() != device:
        raise ValueError("%s: on device %d, the call is on device %d" % (name, t.get_device(), device))
    raise ValueError("%s: expected a contiguous %s" % (name, "last dimension" if last_only else "tensor"))


def _flat(name, t, shape, dtype, device):
    """Address of a contiguous tensor of this shape and type on this device."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
        _refuse(name, t, shape, dtype, device, False)
    return t.data_ptr()


def _rows(name, t, shape, dtype, device):
    """(address, row pitch, head pitch) of a tensor [rows, heads, dim] on this device whose last dimension is contiguous;
    a dimension of one value has no pitch, whatever its stride says."""
    row, head, last = t.stride()
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device or last != 1 and t.numel():
        _refuse(name, t, shape, dtype, device, True)
    return t.data_ptr(), row if shape[0] > 1 else 0, head if shape[1] > 1 else 0


class _Buffer:
    """Device memory of an object, made by the first call that needs it on that call's stream, so that what the allocator's
    memory was used for before has ended there, and given back only when the work of every stream it served has ended."""

    def __init__(self, torch, device, current):
        self._torch, self._device, self._current = torch, device, current
        self.tensor, self.at, self._streams, self.last = None, 0, None, None     # last: stream of the latest call

    def _stream(self, ptr, device):
        cuda = self._torch.cuda
        return cuda.ExternalStream(ptr, device=device) if ptr else cuda.default_stream(device)

    def get(self, size, ptr, device, zeroed=0):
        """Address of `size` bytes for a call on stream `ptr`; the first `zeroed` ones are zero when they are made."""
        if self.tensor is None:
            torch = self._torch
            if ptr == self._current(device):
                made = torch.empty(size, dtype=torch.uint8, device=self._device)
                made[:zeroed].zero_()
            else:
                with torch.cuda.stream(self._stream(ptr, device)):
                    made = torch.empty(size, dtype=torch.uint8, device=self._device)
                    made[:zeroed].zero_()
            self.tensor, self.at, self._streams, self.last = made, made.data_ptr(), {ptr}, ptr
        elif ptr != self.last:
            if ptr not in self._streams:
                self.tensor.record_stream(self._stream(ptr, device))
                self._streams.add(ptr)
            self.last = ptr
        return self.at


class _Placed:
    """The device of an object: of its first call's tensors, or the one it was made for."""
    _on = None

    def _device_of(self, name, t):
        """Device of a call whose first tensor is t (-2, which no tensor is on, for a host tensor)."""
        device = t.get_device()
        if device != self._on:
            if device < 0:
                return -2
            if self._on is None:
                self._on = self._torch.device(self.device).index
            if self._on is None:
                self._on = device
            if device != self._on:
                raise ValueError("%s: on device %d, the object is on device %d" % (name, device, self._on))
        if device != self._here():
            raise ValueError("%s: on device %d, which is not the current one" % (name, device))
        return device


class _Attention(_Placed):
    """Sizes and work buffers of an attention; ``PASSES`` of them."""
    PASSES = 2

    def __init__(self, n_queries: int, n_nodes: int, n_heads: int, n_kv_heads: int, head_dim: int, dtype,
                 sources: int = 0, edges=None, scale: float | None = None, device="cuda"):
        import torch
        self._torch = torch
        self.dtype, self.device = dtype, device
        edges = list(edges) if edges is not None else []
        if len(edges) > ATTN_MAX_BUCKETS or any(not 0 <= e <= ATTN_MAX_HOP for e in edges):
            raise ValueError("edges: at most %d first hops of 0..%d" % (ATTN_MAX_BUCKETS, ATTN_MAX_HOP))
        a = self._a = Attn()
        a.dtype = _dtype_code(dtype, (BF16, FP16))
        a.n_queries, a.n_heads, a.n_kv_heads, a.head_dim = n_queries, n_heads, n_kv_heads, head_dim
        a.n_sources, a.n_buckets, a.n_nodes = sources, len(edges), n_nodes
        a.scale = 1.0 / math.sqrt(head_dim) if scale is None else scale
        for i, e in enumerate(edges):
            a.edges[i] = e
        self._ref = ctypes.byref(a)
        self._buf = memoryview(a).cast("B")
        self._int, self._float = torch.int32, torch.float32
        self._rows = torch.Size((n_queries, n_heads, head_dim))
        self._nodes = torch.Size((n_nodes, n_kv_heads, head_dim))
        self._lse = torch.Size((n_queries, n_heads))
        self._hops, self._hops_flat = torch.Size((n_nodes, sources)), torch.Size((n_nodes * sources,))
        self._source = torch.Size((n_queries,))
        self._table = torch.Size((n_heads, len(edges)))
        self._lib = load()
        self._current, self._here = _stream_getter(torch), _device_getter(torch)
        self._buffers, self._bytes = [_Buffer(torch, device, self._current) for _ in range(self.PASSES)], [0] * self.PASSES
        self._lock = threading.Lock()      # of the struct and the buffers: ctypes lets other threads run during a call

    @property
    def _work(self):
        return [b.tensor for b in self._buffers]

    def _work_of(self, backward: int, stream=None, device=None):
        if device is None:
            device = self._torch.cuda.current_device()
        if not self._bytes[backward]:
            self._bytes[backward] = self.work_bytes(bool(backward))
        size = self._bytes[backward]
        return self._buffers[backward].get(size, self._current(device) if stream is None else stream, device, zeroed=4), size

    def status(self) -> int:
        """The device status words of the passes, joined: waits for the device; 0, or
        ``k2t.STATUS_WAIT_TIMEOUT`` once a bounded wait ran out in a call of this object."""
        word = 0
        for work in self._work:
            if work is not None:
                self._torch.cuda.synchronize()
                word |= int(work[:4].view(self._torch.int32).item())
        return word


class HopAttention(_Attention):
    """Attention of ``n_queries`` queries to the states of ``n_nodes`` nodes.

    ``sources`` columns of a hop table (int32 [n_nodes, sources], as
    ``Tree.msbfs`` leaves it: -1 masks a node) and ``edges``, the first hop of
    each bucket of the bias table [n_heads, len(edges)]; ``sources`` 0 is plain
    attention, no ``edges`` masks without a bias.  See ``k2t_attn``.

    A call returns before its kernels have run: should a bounded wait in one of
    them run out, the outputs are undefined and only ``status`` tells.
    """

    def __init__(self, n_queries: int, n_nodes: int, n_heads: int, n_kv_heads: int, head_dim: int, dtype,
                 sources: int = 0, edges=None, scale: float | None = None, device="cuda"):
        super().__init__(n_queries, n_nodes, n_heads, n_kv_heads, head_dim, dtype, sources, edges, scale, device)
        self._forward, self._backward = self._lib.k2t_attn_forward, self._lib.k2t_attn_backward

    def work_bytes(self, backward: bool = False) -> int:
        """Device bytes of the work buffer of a pass (k2t_attn_work_bytes)."""
        return int(self._lib.k2t_attn_work_bytes(self._ref, int(backward)))

    def _inputs(self, q, k, v, out, lse, hops, bias, query_source):
        a, dt, device = self._a, self.dtype, q.get_device()
        if device != self._on or device != self._here():
            device = self._device_of("q", q)
        if (hops is None) != (a.n_sources == 0):
            raise ValueError("hops: given %s, sources %d" % (hops is not None, a.n_sources))
        qp, qr, qh = _rows("q", q, self._rows, dt, device)
        kp, kr, kh = _rows("k", k, self._nodes, dt, device)
        vp, vr, vh = _rows("v", v, self._nodes, dt, device)
        op, orow, oh = _rows("out", out, self._rows, dt, device)
        _INPUTS.pack_into(self._buf, _AT_INPUTS, qp, kp, vp, qr, qh, kr, kh, vr, vh,
                          0 if hops is None else _flat("hops", hops, self._hops if hops.ndim == 2 else self._hops_flat, self._int, device),
                          0 if query_source is None else _flat("query_source", query_source, self._source, self._int, device),
                          0 if bias is None else _flat("bias", bias, self._table, dt, device),
                          op, _flat("lse", lse, self._lse, self._float, device), orow, oh)
        return device

    def forward(self, q, k, v, out, lse, hops=None, bias=None, query_source=None, stream=None):
        """out [T, n_heads, head_dim] and lse (fp32 [T, n_heads]) of q, k, v."""
        with self._lock:
            device = self._inputs(q, k, v, out, lse, hops, bias, query_source)
            st = self._current(device) if stream is None else _stream_ptr(stream)
            work = self._buffers[0]
            if work.last != st:
                self._work_of(0, st, device)
            rc = self._forward(self._ref, work.at, self._bytes[0], st)
        if rc:
            _check("k2t_attn_forward", rc)
        return out, lse

    def backward(self, dout, q, k, v, out, lse, dq, dk, dv, dbias=None, hops=None, bias=None, query_source=None,
                 stream=None):
        """Gradients of q, k, v and the bias table from dout, the inputs and the forward's out and lse."""
        dt = self.dtype
        with self._lock:
            device = self._inputs(q, k, v, out, lse, hops, bias, query_source)
            dqp, dqr, dqh = _rows("dq", dq, self._rows, dt, device)
            dkp, dkr, dkh = _rows("dk", dk, self._nodes, dt, device)
            dvp, dvr, dvh = _rows("dv", dv, self._nodes, dt, device)
            _GRADIENTS.pack_into(self._buf, _AT_GRADIENTS, *_rows("dout", dout, self._rows, dt, device), dqp, dkp, dvp, dqr, dqh,
                                 dkr, dkh, dvr, dvh, 0 if dbias is None else _flat("dbias", dbias, self._table, dt, device))
            st = self._current(device) if stream is None else _stream_ptr(stream)
            work = self._buffers[1]
            if work.last != st:
                self._work_of(1, st, device)
            rc = self._backward(self._ref, work.at, self._bytes[1], st)
        if rc:
            _check("k2t_attn_backward", rc)
        return dq, dk, dv, dbias


# the pointers and pitches of k2t_attn, in the header's order: q .. out_head, dout .. dbias
_INPUTS, _AT_INPUTS = struct.Struct("=3Q6q5Q2q"), Attn.q.offset
_GRADIENTS, _AT_GRADIENTS = struct.Struct("=Q2q3Q6qQ"), Attn.dout.offset
assert _AT_INPUTS + _INPUTS.size == _AT_GRADIENTS and _AT_GRADIENTS + _GRADIENTS.size == ctypes.sizeof(Attn)


class LayerNorm(_Placed):
    """Layer norm of ``n_rows`` states of ``dim`` values, with the residual sum before it (``k2t_norm``).

    A backward call takes the mean and rstd (fp32 [n_rows] each) that its
    forward call wrote, or forms them again from the states it is given.
    ``mean`` and ``rstd`` of the object are of its latest forward call that was
    not given tensors for them.
    """

    def __init__(self, n_rows: int, dim: int, dtype, residual: bool = False, eps: float = 1e-5, device="cuda"):
        import torch
        self._torch = torch
        self.dtype, self.device, self.residual = dtype, device, residual
        a = self._a = Norm()
        a.dtype = _dtype_code(dtype, (BF16, FP16, FP32))
        a.dim, a.n_rows, a.eps = dim, n_rows, eps
        self._ref = ctypes.byref(a)
        self._buf = memoryview(a).cast("B")
        self._rows, self._cols, self._one = torch.Size((n_rows, dim)), torch.Size((dim,)), torch.Size((n_rows,))
        self._float = torch.float32
        self._lib = load()
        self._forward, self._backward = self._lib.k2t_norm_forward, self._lib.k2t_norm_backward
        self._current, self._here = _stream_getter(torch), _device_getter(torch)
        self._n = n_rows
        self._work, self._own = (_Buffer(torch, device, self._current) for _ in range(2))     # backward's; mean and rstd
        a.flags = NORM_FORM_STATS           # the more of the two
        self._bytes = int(self._lib.k2t_norm_work_bytes(self._ref))
        self._lock = threading.Lock()

    def work_bytes(self) -> int:
        """Device bytes of the backward pass's work buffer (k2t_norm_work_bytes), statistics formed again or not."""
        return self._bytes

    def _own_stats(self, stream, device):
        at = self._own.get(max(8 * self._n, 16), stream, device)
        self._own_at = at, at + 4 * self._n
        return self._own_at

    def _stat(self, which):
        with self._lock:
            device = self._torch.cuda.current_device()
            self._own_stats(self._current(device), device)
            return self._own.tensor.view(self._float)[which * self._n:(which + 1) * self._n]

    mean = property(lambda self: self._stat(0), doc="Means of the latest forward call that was not given a tensor for them.")
    rstd = property(lambda self: self._stat(1), doc="Likewise 1 / sqrt(var + eps).")

    def _stats(self, mean, rstd, device):
        if mean is None or rstd is None:
            raise ValueError("mean and rstd are given together")
        return _flat("mean", mean, self._one, self._float, device), _flat("rstd", rstd, self._one, self._float, device)

    def forward(self, x, weight, bias, y, residual=None, z=None, stream=None, mean=None, rstd=None):
        """y = norm(z) and, with a residual, z = x + residual; writes the rows' mean and rstd."""
        if (residual is not None) != self.residual or (z is not None) != self.residual:
            raise ValueError("residual and z are given exactly when the layer has a residual")
        dt, rows, cols = self.dtype, self._rows, self._cols
        with self._lock:
            device = x.get_device()
            if device != self._on or device != self._here():
                device = self._device_of("x", x)
            at = _flat("x", x, rows, dt, device)
            st = self._current(device) if stream is None else _stream_ptr(stream)
            if mean is not None or rstd is not None:
                stats = self._stats(mean, rstd, device)
            else:
                stats = self._own_at if self._own.last == st else self._own_stats(st, device)
            _FORWARD.pack_into(self._buf, _AT_FORWARD, 0, at,
                               0 if residual is None else _flat("residual", residual, rows, dt, device),
                               _flat("weight", weight, cols, dt, device), 0 if bias is None else _flat("bias", bias, cols, dt, device),
                               _flat("y", y, rows, dt, device), 0 if z is None else _flat("z", z, rows, dt, device), *stats)
            rc = self._forward(self._ref, st)
        if rc:
            _check("k2t_norm_forward", rc)
        return y if z is None else (y, z)

    def backward(self, dy, z, weight, dx, dweight, dbias=None, dz=None, stream=None, mean=None, rstd=None):
        """dx (of x and of the residual alike), dweight and dbias from dy and the forward's z (its x without a
        residual); dz, the gradient that reaches z from elsewhere, is added to dx.  mean and rstd: what the forward call
        of this z wrote; without them they are formed again from z."""
        dt, rows, cols = self.dtype, self._rows, self._cols
        with self._lock:
            device = dy.get_device()
            if device != self._on or device != self._here():
                device = self._device_of("dy", dy)
            form = mean is None and rstd is None
            _BACKWARD.pack_into(self._buf, _AT_FORWARD, NORM_FORM_STATS if form else 0, 0, 0,
                                _flat("weight", weight, cols, dt, device), 0, 0, _flat("z", z, rows, dt, device),
                                *(_NONE if form else self._stats(mean, rstd, device)), _flat("dy", dy, rows, dt, device),
                                0 if dz is None else _flat("dz", dz, rows, dt, device), _flat("dx", dx, rows, dt, device),
                                _flat("dweight", dweight, cols, dt, device), 0 if dbias is None else _flat("dbias", dbias, cols, dt, device))
            st = self._current(device) if stream is None else _stream_ptr(stream)
            work = self._work
            if work.last != st:
                work.get(max(16, self._bytes), st, device)
            rc = self._backward(self._ref, work.at, self._bytes, st)
        if rc:
            _check("k2t_norm_backward", rc)
        return dx, dweight, dbias


_NONE = (0, 0)
# flags and pointers of k2t_norm: up to rstd, and all
_FORWARD, _BACKWARD, _AT_FORWARD = struct.Struct("=I8Q"), struct.Struct("=I13Q"), Norm.flags.offset
assert _AT_FORWARD + _FORWARD.size == Norm.dy.offset and _AT_FORWARD + _BACKWARD.size == ctypes.sizeof(Norm)


class HeadNorm(_Placed):
    """RMS norm of each of ``n_heads`` heads of ``head_dim`` values of ``n_rows`` queries or keys, and their rotation by
    position in the same pass (``k2t_head_norm``).

    The first ``rotary_dim`` values of a head (all of them by default; 0: norm alone) turn in pairs, value i with
    i + rotary_dim / 2 or, ``paired``, neighbours, by position times base^(-2 m / rotary_dim).  A backward call needs
    the forward's input and nothing else of it.
    """

    def __init__(self, n_rows: int, n_heads: int, head_dim: int, dtype, rotary_dim: int | None = None, paired: bool = False,
                 base: float = 10000.0, eps: float = 1e-6, device="cuda"):
        import torch
        self._torch = torch
        self.dtype, self.device = dtype, device
        a = self._a = HeadNormArgs()
        a.dtype = _dtype_code(dtype, (BF16, FP16, FP32))
        a.n_heads, a.head_dim, a.n_rows, a.eps, a.flags = n_heads, head_dim, n_rows, eps, HEAD_PAIRED if paired else 0
        a.rotary_dim = head_dim if rotary_dim is None else rotary_dim
        self._lib = load()
        if self._lib.k2t_head_rates(base, a.rotary_dim, ctypes.cast(a.rates, ctypes.c_void_p)):
            raise ValueError("rotary_dim must be even and at most 256, base at least 1 and finite")
        self._ref = ctypes.byref(a)
        self._buf = memoryview(a).cast("B")
        self._shape, self._cols, self._one = torch.Size((n_rows, n_heads, head_dim)), torch.Size((head_dim,)), torch.Size((n_rows,))
        self._int = torch.int32
        self._forward, self._backward = self._lib.k2t_head_norm_forward, self._lib.k2t_head_norm_backward
        self._current, self._here = _stream_getter(torch), _device_getter(torch)
        self._work, self._bytes = _Buffer(torch, device, self._current), self.work_bytes()
        self._lock = threading.Lock()

    def work_bytes(self) -> int:
        """Device bytes of the backward pass's work buffer (k2t_head_norm_work_bytes)."""
        return int(self._lib.k2t_head_norm_work_bytes(self._ref))

    def _inputs(self, x, weight, positions, device):
        at, row, head = _rows("x", x, self._shape, self.dtype, device)
        return (at, 0 if weight is None else _flat("weight", weight, self._cols, self.dtype, device),
                0 if positions is None else _flat("positions", positions, self._one, self._int, device)), (row, head)

    def forward(self, x, weight, y, positions=None, stream=None):
        """y [n_rows, n_heads, head_dim] of x; weight [head_dim] or None, positions int32 [n_rows] (None: a row's number)."""
        with self._lock:
            device = x.get_device()
            if device != self._on or device != self._here():
                device = self._device_of("x", x)
            (xp, wp, pp), (xr, xh) = self._inputs(x, weight, positions, device)
            yp, yr, yh = _rows("y", y, self._shape, self.dtype, device)
            _HEAD.pack_into(self._buf, _AT_HEAD, xp, wp, pp, yp, xr, xh, yr, yh, 0, 0, 0, 0, 0, 0, 0)
            rc = self._forward(self._ref, self._current(device) if stream is None else _stream_ptr(stream))
        if rc:
            _check("k2t_head_norm_forward", rc)
        return y

    def backward(self, dy, x, weight, dx, dweight, positions=None, stream=None):
        """dx and dweight from dy and the forward call's x and positions; weight and dweight are given together or are both None."""
        with self._lock:
            device = dy.get_device()
            if device != self._on or device != self._here():
                device = self._device_of("dy", dy)
            (xp, wp, pp), (xr, xh) = self._inputs(x, weight, positions, device)
            gp, gr, gh = _rows("dy", dy, self._shape, self.dtype, device)
            dp, dr, dh = _rows("dx", dx, self._shape, self.dtype, device)
            _HEAD.pack_into(self._buf, _AT_HEAD, xp, wp, pp, 0, xr, xh, 0, 0, gp, dp,
                            0 if dweight is None else _flat("dweight", dweight, self._cols, self.dtype, device), gr, gh, dr, dh)
            st = self._current(device) if stream is None else _stream_ptr(stream)
            work = self._work
            if wp and work.last != st:
                work.get(max(16, self._bytes), st, device)
            rc = self._backward(self._ref, work.at, self._bytes, st)
        if rc:
            _check("k2t_head_norm_backward", rc)
        return dx, dweight


# pointers and pitches of k2t_head_norm
_HEAD, _AT_HEAD = struct.Struct("=4Q4q3Q4q"), HeadNormArgs.x.offset
assert _AT_HEAD + _HEAD.size == ctypes.sizeof(HeadNormArgs)
