"""k^2-tree semiring SpMV on GB300 (sm_103a): thin Python binding of libk2t.so.

The C ABI is declared in ``include/k2t.h``; ``k2t.Tree`` wraps it, and
``reader.HopAttention`` and ``reader.LayerNorm`` the layers of a model that
reads a graph (attention biased by hop distances, layer norm), with
``reader.HeadNorm`` (norm and rotation of each head of queries and keys).
``cache.NodeCache`` keeps node states in 8 bits and ``cache.CachedAttention``
attends to them.  Build the shared library with ``compressed_graph_spmv_gb300._build.build()`` (or
``__graft_entry__.build()``).
"""
from .k2t import (BOOLEAN, ENGINE_AUTO, ENGINE_BANDED, ENGINE_CACHED, ENGINE_FUSED, ENGINE_LEVELSYNC, LEFT,
                  MIN_PLUS, OFFSETS_DIRECTORY, OFFSETS_SCAN, PLUS_TIMES, RIGHT, K2TError, Tree,
                  default_opts, load)
from .reader import HeadNorm, HopAttention, LayerNorm, hop_edges
from .cache import CachedAttention, NodeCache

__all__ = ["Tree", "default_opts", "load", "K2TError", "RIGHT", "LEFT", "PLUS_TIMES", "BOOLEAN",
           "MIN_PLUS", "ENGINE_AUTO", "ENGINE_BANDED", "ENGINE_FUSED", "ENGINE_LEVELSYNC", "ENGINE_CACHED",
           "OFFSETS_DIRECTORY", "OFFSETS_SCAN", "HopAttention", "LayerNorm", "HeadNorm", "NodeCache",
           "CachedAttention", "hop_edges"]
