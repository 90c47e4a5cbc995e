"""The work buffer of the attention over the 8-bit cache is enough for any part of the cache (no GPU: whether it is, the call
itself tells by ENOMEM, which it says before it launches; no address here is real)."""
import ctypes

import pytest

from test_cache_refusals import cache
from test_reader_refusals import ENOMEM, P, attn

K = pytest.importorskip("compressed_graph_spmv_gb300.k2t")
torch = pytest.importorskip("torch")

if torch.cuda.is_available():
    pytest.skip("with a GPU a call that has enough would launch", allow_module_level=True)

SIZES = [  # queries, heads, key/value heads, head_dim, sources, nodes
    (1, 4, 4, 64, 0, 100000), (1, 16, 4, 128, 1, 1 << 20), (32, 16, 4, 128, 32, 1 << 20), (1024, 8, 8, 128, 32, 16384),
    (13, 6, 2, 72, 13, 100003), (300, 4, 1, 64, 7, 5000), (7, 2, 1, 64, 0, 1), (9, 3, 3, 40, 9, 0), (64, 115, 115, 64, 0, 40000),
    (900, 24, 12, 64, 3, 30000), (5, 59, 59, 32, 5, 9000), (129, 7, 7, 96, 30, 77777),
]


def calls(T, hq, hkv, d, sources, n):
    size = dict(n_queries=T, n_heads=hq, n_kv_heads=hkv, head_dim=d, n_sources=sources, n_buckets=0, bias=None, edges=(), hops=P if sources else None,
                query_source=P if sources else None, q_row=hq * d, q_head=d, out_row=hq * d, out_head=d, k=None, v=None)
    c = cache(n_kv_heads=hkv, head_dim=d, n_nodes=n)
    lib = K.load()

    def enough(nodes, work):
        return lib.k2t_cached_attn_forward(ctypes.byref(attn(n_nodes=nodes, **size)), ctypes.byref(c), P, work, None) != ENOMEM
    return enough, lambda nodes: lib.k2t_cached_attn_work_bytes(ctypes.byref(attn(n_nodes=nodes, **size)))


def part_sizes(n):
    return sorted({min(n, x) for x in (0, 1, 127, 128, 129, 1000, 4864, 4865, 5000, 19456, 19457, 38912, 38913, n - 1 if n else 0, n)} |
                  {min(n, 128 * t) for t in range(1, 160)} | {n * i // 97 for i in range(98)})


@pytest.mark.parametrize("size", SIZES)
def test_work_is_enough_for_any_part_of_the_cache(size):
    enough, asked = calls(*size)
    work = asked(size[-1])
    for nodes in part_sizes(size[-1]):
        assert enough(nodes, work) and asked(nodes) <= work
    assert not enough(size[-1], 0)
