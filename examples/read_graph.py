"""Read a graph with a model: search, aggregation, norm, attention, one training loop.

A multi-source search gives the hop distance of every node from up to 32
entities; a plus-times product aggregates node features along the edges; the
sum of a node's own and aggregated features is normalised; each entity then
attends to the states of all nodes that its search reached, with a learned
bias by hop bucket.  The loop trains queries and bias table so that each
entity's answer matches a target, through the operators' backward passes.

    python examples/read_graph.py [--scale 12] [--edges 60000] [--steps 30]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import numpy as np
import torch

import compressed_graph_spmv_gb300 as k2t
import synth


def read_graph(scale=12, edges=60000, steps=30, heads=8, kv_heads=4, head_dim=64, buckets=8, seed=1, say=print):
    n, sources, width = 1 << scale, 32, kv_heads * head_dim
    rng = np.random.default_rng(seed)
    torch.manual_seed(seed)
    bf16 = torch.bfloat16

    # the graph, and how far every node is from each of the entities
    rows, cols = synth.rmat(scale, 0.57, 0.19, 0.19, edges, seed)
    tree = k2t.Tree(rows, cols, n, n).upload()
    entities = rng.choice(np.unique(cols), size=sources)
    hops = torch.empty(n, sources, dtype=torch.int32, device="cuda")
    work = torch.empty(tree.msbfs_work_bytes(), dtype=torch.uint8, device="cuda")
    tree.msbfs(k2t.LEFT, entities, hops, work)

    # node states: features aggregated along the edges, projected, added to the node's own and normalised
    features = torch.randn(n, 32, device="cuda")
    gathered = torch.empty_like(features)
    tree.spmv(k2t.RIGHT, k2t.PLUS_TIMES, features, gathered, B=32)
    project = torch.randn(32, 2 * width, device="cuda") / 32 ** 0.5
    own, aggregated = (features @ project).to(bf16), (gathered @ project).to(bf16)
    weight, bias = (torch.full((2 * width,), v, dtype=bf16, device="cuda") for v in (1.0, 0.0))
    norm = k2t.LayerNorm(n, 2 * width, bf16, residual=True)
    states, summed = torch.empty_like(own), torch.empty_like(own)
    norm.forward(aggregated, weight, bias, states, residual=own, z=summed)
    halves = states.view(n, 2, kv_heads, head_dim)
    k, v = halves[:, 0], halves[:, 1]          # views: the attention takes strides

    # the reader: queries of the entities, a bias by hop bucket
    edges_of = k2t.hop_edges(buckets, 16)
    attention = k2t.HopAttention(sources, n, heads, kv_heads, head_dim, bf16, sources=sources, edges=edges_of)
    q = torch.randn(sources, heads, head_dim, device="cuda")
    table = torch.zeros(heads, buckets, device="cuda")
    out, dq = (torch.empty(sources, heads, head_dim, dtype=bf16, device="cuda") for _ in range(2))
    lse = torch.empty(sources, heads, device="cuda")
    dstates = torch.empty_like(states)
    dhalves = dstates.view(n, 2, kv_heads, head_dim)
    dtable = torch.empty(heads, buckets, dtype=bf16, device="cuda")
    target = v[torch.from_numpy(entities.astype(np.int64)).cuda()].repeat_interleave(heads // kv_heads, 1).float()

    losses = []
    for step in range(steps):
        qh, th = q.to(bf16), table.to(bf16)
        attention.forward(qh, k, v, out, lse, hops=hops, bias=th)
        error = out.float() - target
        losses.append(error.square().mean().item())
        dout = (2.0 / error.numel() * error * 256).to(bf16)     # scaled, so that bf16 holds small gradients
        attention.backward(dout, qh, k, v, out, lse, dq, dhalves[:, 0], dhalves[:, 1], dbias=dtable, hops=hops, bias=th)
        q -= 4.0 * dq.float()
        table -= 4.0 * dtable.float()
        if step % 10 == 0 or step == steps - 1:
            say("step %3d  loss %.4f" % (step, losses[-1]))
    # the gradient goes on through the norm to the features
    dsummed, dweight, dbias = torch.empty_like(states), torch.empty_like(weight), torch.empty_like(bias)
    norm.backward(dstates, summed, weight, dsummed, dweight, dbias)
    reached = (hops >= 0).float().mean().item()
    say("%d nodes, %.0f%% reached; bias of head 0 by first hop %s: %s" % (
        n, 100 * reached, edges_of, [round(x, 2) for x in table[0].tolist()]))
    return losses, dsummed


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--scale", type=int, default=12)
    ap.add_argument("--edges", type=int, default=60000)
    ap.add_argument("--steps", type=int, default=30)
    a = ap.parse_args()
    read_graph(a.scale, a.edges, a.steps)
