"""Graph-reading calls on the host: flags, layouts of outputs, threads, devices (no GPU)."""
import ctypes

import pytest

from test_reader_refusals import ENOMEM, EINVAL, P, norm

K = pytest.importorskip("compressed_graph_spmv_gb300.k2t")


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
