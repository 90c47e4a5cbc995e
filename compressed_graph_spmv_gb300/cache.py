"""Node states kept in 8 bits, and attention over them (``k2t_cache_*`` and
``k2t_cached_attn_*`` of ``include/k2t.h``), on device tensors.

As in ``reader.py``: argument marshalling only, outputs are the caller's, an
object's calls are ordered on the GPU by the caller, and host threads may share
an object.
"""
from __future__ import annotations

import ctypes
import threading

from .k2t import BF16, CACHE_BLOCK, FP16, FP32, Cache, _check, _stream_ptr, load
from .reader import (_AT_INPUTS, _Attention, _device_getter, _dtype_code, _flat, _INPUTS, _Placed, _rows, _stream_getter)


class NodeCache(_Placed):
    """Keys and values of ``n_nodes`` nodes in 8 bits (``k2t_cache``): e4m3, with a power of two for each block of 32
    nodes and head.

    ``k`` and ``v`` (float8_e4m3fn [n_kv_heads, n_nodes, head_dim rounded up to 16]) and ``k_scale`` and ``v_scale``
    (uint8 s [n_kv_heads, blocks rounded up to 16], for 2^(s - 64)) are made, all zero, on the stream that is current
    when the object is made; a stream that uses them before that is done has to wait for it.  Between calls another tensor of
    the same type and layout may be assigned in the place of one (a cache that was saved); graphs captured before go on with
    the old one, which they do not keep.
    """

    def __init__(self, n_nodes: int, n_kv_heads: int, head_dim: int, dtype, device="cuda"):
        import torch
        self._torch = torch
        self.n_nodes, self.n_kv_heads, self.head_dim, self.dtype, self.device = n_nodes, n_kv_heads, head_dim, dtype, device
        if not (0 <= n_nodes < 1 << 31 and 1 <= n_kv_heads <= 65535 and 8 <= head_dim <= 128 and head_dim % 8 == 0):
            raise ValueError("a cache of %s nodes, %s heads of %s" % (n_nodes, n_kv_heads, head_dim))
        if torch.device(device).type == "cuda" and torch.cuda.is_available() and torch.cuda.is_current_stream_capturing():
            raise RuntimeError("a cache made during a capture would be emptied by every replay")
        self._lib = load()
        self._write, self._read = self._lib.k2t_cache_write, self._lib.k2t_cache_read
        self._current, self._here = _stream_getter(torch), _device_getter(torch)
        pitch, blocks = (head_dim + 15) // 16 * 16, -(-n_nodes // CACHE_BLOCK)
        rows, scales = (n_kv_heads, n_nodes, pitch), (n_kv_heads, (blocks + 15) // 16 * 16)
        k, v = (torch.zeros(rows, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(2))
        k_scale, v_scale = (torch.zeros(scales, dtype=torch.uint8, device=device) for _ in range(2))
        self._tensors = dict(k=k, v=v, k_scale=k_scale, v_scale=v_scale)
        self._streams = {self._current(k.get_device())} if k.is_cuda else set()
        self._a, self._held = Cache(), Cache()         # of a write or read; of an attention, which does not change
        for a in (self._a, self._held):
            a.dtype, a.n_kv_heads, a.head_dim, a.n_nodes = _dtype_code(dtype, (BF16, FP16, FP32)), n_kv_heads, head_dim, n_nodes
            a.k, a.v, a.k_scale, a.v_scale = (t.data_ptr() for t in (k, v, k_scale, v_scale))
        self._ref, self._held_ref = ctypes.byref(self._a), ctypes.byref(self._held)
        self._int = torch.int32
        self._lock = threading.Lock()

    def _assign(self, name, t):
        """Another tensor in the place of one: the calls take its address from here on."""
        with self._lock:
            old = self._tensors[name]
            if t.shape != old.shape or not t.is_contiguous():
                raise ValueError("%s: expected a contiguous tensor of shape %s, got %s" % (name, tuple(old.shape), tuple(t.shape)))
            if isinstance(t, self._torch.Tensor):
                if t.dtype is not old.dtype:
                    raise TypeError("%s: expected %s, got %s" % (name, old.dtype, t.dtype))
                if t.device != old.device or t.data_ptr() % 16:
                    raise ValueError("%s: expected a tensor on %s that begins on 16 bytes" % (name, old.device))
            self._tensors[name] = t
            for a in (self._a, self._held):
                setattr(a, name, t.data_ptr())
            self._streams = set()          # no stream is known to have used it

    k, v, k_scale, v_scale = (property(lambda self, name=name: self._tensors[name], lambda self, t, name=name: self._assign(name, t))
                              for name in ("k", "v", "k_scale", "v_scale"))

    def _used_on(self, ptr, device):
        """The tensors are not given back before the work of every stream that used them has ended."""
        if ptr not in self._streams:
            cuda = self._torch.cuda
            stream = cuda.ExternalStream(ptr, device=device) if ptr else cuda.default_stream(device)
            for t in self._tensors.values():
                t.record_stream(stream)
            self._streams.add(ptr)

    def _call(self, name, call, k, v, first, count, nodes, stream):
        a, shape = self._a, self._torch.Size((count, self.n_kv_heads, self.head_dim))
        if first < 0:
            raise ValueError("first: %d" % first)
        with self._lock:
            device = k.get_device()
            if device != self._on or device != self._here():
                device = self._device_of("k", k)
            own = self._tensors["k"].get_device()
            if own != device:
                raise ValueError("k: on device %d, the cache is on device %d" % (device, own))
            a.x_k, a.xk_row, a.xk_head = _rows("k", k, shape, self.dtype, device)
            a.x_v, a.xv_row, a.xv_head = _rows("v", v, shape, self.dtype, device)
            a.nodes = 0 if nodes is None else _flat("nodes", nodes, shape[:1], self._int, device)
            a.first, a.count = first, count
            st = self._current(device) if stream is None else _stream_ptr(stream)
            self._used_on(st, device)
            rc = call(self._ref, st)
        if rc:
            _check(name, rc)

    def write(self, k, v, first: int = 0, stream=None):
        """Nodes first, first + 1, .. get the states k and v ([count, n_kv_heads, head_dim] each)."""
        self._call("k2t_cache_write", self._write, k, v, first, k.shape[0], None, stream)

    def read(self, k, v, first: int = 0, nodes=None, stream=None):
        """k and v become the states of nodes first, first + 1, .., or of ``nodes`` (int32 [count])."""
        self._call("k2t_cache_read", self._read, k, v, first, k.shape[0], nodes, stream)
        return k, v


class CachedAttention(_Attention):
    """``HopAttention``'s forward pass over the first ``n_nodes`` nodes of a ``NodeCache`` (``k2t_cached_attn_forward``).

    A call may take fewer of them (``nodes``), as a cache that is still being filled has; the hop table stays
    [n_nodes, sources].  A call returns before its kernels have run: should a bounded wait in one of them run out, the
    outputs are undefined and only ``status`` tells.
    """
    PASSES = 1

    def __init__(self, n_queries: int, n_nodes: int, n_heads: int, n_kv_heads: int, head_dim: int, dtype,
                 sources: int = 0, edges=None, scale: float | None = None, device="cuda"):
        super().__init__(n_queries, n_nodes, n_heads, n_kv_heads, head_dim, dtype, sources, edges, scale, device)
        self.n_nodes = n_nodes
        self._forward = self._lib.k2t_cached_attn_forward

    def work_bytes(self, backward: bool = False) -> int:
        """Device bytes of the work buffer (k2t_cached_attn_work_bytes), for any number of nodes up to n_nodes."""
        with self._lock:
            return self._most_bytes()

    def _most_bytes(self):
        at = self._a.n_nodes
        self._a.n_nodes = self.n_nodes
        size = int(self._lib.k2t_cached_attn_work_bytes(self._ref))
        self._a.n_nodes = at
        return size

    def forward(self, q, cache, out, lse, hops=None, bias=None, query_source=None, nodes=None, stream=None):
        """out [T, n_heads, head_dim] and lse (fp32 [T, n_heads]) of q and the cache's first ``nodes`` nodes."""
        a, dt = self._a, self.dtype
        nodes = self.n_nodes if nodes is None else nodes
        if not 0 <= nodes <= self.n_nodes:
            raise ValueError("nodes: %d of %d" % (nodes, self.n_nodes))
        with self._lock:
            device = q.get_device()
            if device != self._on or device != self._here():
                device = self._device_of("q", q)
            if cache.k.get_device() != device:
                raise ValueError("cache: on device %d, the call is on device %d" % (cache.k.get_device(), device))
            if (hops is None) != (a.n_sources == 0):
                raise ValueError("hops: given %s, sources %d" % (hops is not None, a.n_sources))
            qp, qr, qh = _rows("q", q, self._rows, dt, device)
            op, orow, oh = _rows("out", out, self._rows, dt, device)
            _INPUTS.pack_into(self._buf, _AT_INPUTS, qp, 0, 0, qr, qh, 0, 0, 0, 0,
                              0 if hops is None else _flat("hops", hops, self._hops if hops.ndim == 2 else self._hops_flat, self._int, device),
                              0 if query_source is None else _flat("query_source", query_source, self._source, self._int, device),
                              0 if bias is None else _flat("bias", bias, self._table, dt, device),
                              op, _flat("lse", lse, self._lse, self._float, device), orow, oh)
            st = self._current(device) if stream is None else _stream_ptr(stream)
            work = self._buffers[0]
            if work.last != st:
                if not self._bytes[0]:
                    self._bytes[0] = self._most_bytes()
                work.get(max(16, self._bytes[0]), st, device, zeroed=4)
            cache._used_on(st, device)
            a.n_nodes = nodes
            rc = self._forward(self._ref, cache._held_ref, work.at, self._bytes[0], st)
        if rc:
            _check("k2t_cached_attn_forward", rc)
        return out, lse
