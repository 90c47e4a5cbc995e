"""The operators that read a graph with a model, as measured work.

Two families, each forward and as a training pass:
* attention of queries to the states of a graph's nodes, with a learned bias
  by bucket of the hop distance (the table k2t_msbfs writes: n x B int32,
  -1 where a source does not reach a node, which masks it);
* layer norm of node states, with the residual sum before it.

``own`` false computes the plain form (elementary torch operations in 32
bits), true calls this package.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one entity asks about a graph of the smallest configuration (1024 nodes): a latency-bound call
        dict(name="read 1 of 1024", op="read", T=1, n=1024, hq=8, hkv=8, d=64, sources=1, seen=0.9, buckets=16,
             dtype="bf16"),
        # one entity asks about a graph of 2^20 nodes, grouped heads: the serving form at full size
        dict(name="read 1 of 2^20", op="read", T=1, n=1 << 20, hq=16, hkv=4, d=128, sources=1, seen=1.0, buckets=32,
             dtype="bf16"),
        # a full search batch (32 sources) against 2^20 nodes of which the search reaches a part, as on power-law graphs
        dict(name="read 32 of 2^20", op="read", T=32, n=1 << 20, hq=16, hkv=4, d=128, sources=32, seen=0.7,
             buckets=32, dtype="bf16"),
        # odd everything: 13 sources, a prime number of nodes, a head size that is no power of two
        dict(name="read 13 of 100003", op="read", T=13, n=100003, hq=6, hkv=2, d=72, sources=13, seen=0.8, buckets=11,
             dtype="fp16"),
        # text tokens, each of which mentions one of 32 entities or none, against a retrieved subgraph
        dict(name="read 1024 tokens", op="read", T=1024, n=16384, hq=8, hkv=8, d=128, sources=32, seen=0.95,
             buckets=32, dtype="bf16"),
        # training over a full search batch, the framework's 2^18-node size
        dict(name="train 32 of 2^18", op="train", T=32, n=1 << 18, hq=8, hkv=8, d=64, sources=32, seen=0.8,
             buckets=32, dtype="bf16"),
        # training over ragged token and node counts with grouped heads
        dict(name="train 257 tokens", op="train", T=257, n=8191, hq=8, hkv=2, d=128, sources=32, seen=0.95,
             buckets=32, dtype="bf16"),
        # plain cross attention (no hop table), small: latency of a training step's calls
        dict(name="train 8 of 1000", op="train", T=8, n=1000, hq=4, hkv=4, d=32, sources=0, seen=1.0, buckets=0,
             dtype="fp16"),
        # node states of 2^20 nodes after aggregation: residual sum and norm
        dict(name="norm 2^20 x 512", op="norm", n=1 << 20, d=512, residual=True, dtype="bf16"),
        # a few states of an odd width in the products' own type: a latency-bound call
        dict(name="norm 1000 x 200", op="norm", n=1000, d=200, residual=False, dtype="fp32"),
        # training over 2^18 node states
        dict(name="norm train 2^18 x 1024", op="norm_train", n=1 << 18, d=1024, residual=True, dtype="bf16"),
        # training over an odd number of states of an odd width
        dict(name="norm train 4999 x 333", op="norm_train", n=4999, d=333, residual=False, dtype="fp32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["read", "read", "train", "train", "norm", "norm_train"])
    if op in ("norm", "norm_train"):
        d = _log_int(rng, 32, 4096)
        n = min(_log_int(rng, 1, 1 << 20), (1 << (29 if op == "norm" else 28)) // d)
        return dict(op=op, n=n, d=d, residual=rng.random() < 0.5, dtype=rng.choice(["bf16", "fp16", "fp32"]))
    T = _log_int(rng, 1, 1024)
    hkv = rng.choice([1, 2, 3, 4, 8])
    hq = hkv * rng.choice([1, 1, 2, 4])
    d = rng.choice([32, 40, 64, 64, 72, 96, 128, 128])
    n = _log_int(rng, 1, 1 << 20)
    products = 2 if op == "read" else 6
    while n > 1 and (2 * products * T * hq * n * d > (2 if op == "read" else 1) * 10 ** 11
                     or n * hkv * d > (1 << 29 if op == "read" else 1 << 27)):
        n = n * 3 // 4
    hops = rng.random() < 0.85
    sources = 0 if not hops else T if T <= 32 else rng.randint(1, 32)
    return dict(op=op, T=T, n=n, hq=hq, hkv=hkv, d=d, sources=sources,
                seen=round(rng.uniform(0.4, 1.0), 2) if hops else 1.0, buckets=rng.randint(2, 32) if hops else 0,
                dtype=rng.choice(["bf16", "bf16", "fp16"]))


def _edges(buckets):
    """First hop of each bucket: one bucket a hop for the first half, then growing ones up to 64 hops."""
    half = (buckets + 1) // 2
    edges = list(range(half))
    for b in range(half, buckets):
        grown = int(half * (64.0 / half) ** ((b - half + 1) / (buckets - half + 1)))
        edges.append(max(edges[-1] + 1, grown))
    return edges


def _rand(g, *shape, dtype, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _hops(g, n, sources, seen):
    """Hop distances as a search leaves them: some nodes no source reaches, the others a few hops away, with a long
    tail, nearly the same for every source; the last of several sources reaches nothing it was asked for."""
    depth = 2.0 + torch.rand(n, 1, generator=g, device="cuda").pow(3).mul(12)
    hops = (depth + torch.rand(n, sources, generator=g, device="cuda").mul(2.5)).to(torch.int32)
    hops[torch.rand(n, generator=g, device="cuda") >= seen] = -1
    hops.masked_fill_(torch.rand(n, sources, generator=g, device="cuda") < 0.01, -1)
    if sources > 4:
        hops[:, -1] = -1
    return hops


def _inputs(case, seed):
    """The inputs of a case, as a dict of tensors: the same for the plain form, the kernels and exact()."""
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    n, d = case["n"], case["d"]
    s = {}
    if case["op"] in ("norm", "norm_train"):
        s["x"] = _rand(g, n, d, dtype=dt, scale=1.5)
        s["x"] += 0.25
        s["residual"] = _rand(g, n, d, dtype=dt) if case["residual"] else None
        s["weight"] = (1 + _rand(g, d, dtype=torch.float32, scale=0.1)).to(dt)
        s["bias"] = _rand(g, d, dtype=dt, scale=0.1)
        if case["op"] == "norm_train":
            s["dy"] = _rand(g, n, d, dtype=dt)
            s["dz"] = _rand(g, n, d, dtype=dt) if case["residual"] else None
        return s
    T, hq, hkv = case["T"], case["hq"], case["hkv"]
    s["q"] = _rand(g, T, hq, d, dtype=dt)
    s["k"] = _rand(g, n, hkv, d, dtype=dt)
    s["v"] = _rand(g, n, hkv, d, dtype=dt)
    s["hops"] = s["bias"] = s["source"] = None
    if case["sources"]:
        s["hops"] = _hops(g, n, case["sources"], case["seen"])
        s["bias"] = _rand(g, hq, case["buckets"], dtype=dt, scale=0.7)
        if case["sources"] != T:
            s["source"] = torch.randint(-1, case["sources"], (T,), generator=g, device="cuda", dtype=torch.int32)
    if case["op"] == "train":
        s["dout"] = _rand(g, T, hq, d, dtype=dt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if not own:
        if case.get("buckets"):
            s["edges"] = torch.tensor(_edges(case["buckets"]), dtype=torch.int32, device="cuda")
        return s
    import compressed_graph_spmv_gb300 as k2t
    dt = DTYPES[case["dtype"]]
    if case["op"] in ("norm", "norm_train"):
        s["op"] = k2t.LayerNorm(case["n"], case["d"], dt, residual=case["residual"], eps=1e-5)
        s["y"] = torch.empty_like(s["x"])
        s["z"] = torch.empty_like(s["x"]) if case["residual"] else None
        if case["op"] == "norm_train":
            s["dx"], s["dw"], s["db"] = (torch.empty_like(s[k]) for k in ("x", "weight", "bias"))
        return s
    s["op"] = k2t.HopAttention(case["T"], case["n"], case["hq"], case["hkv"], case["d"], dt, sources=case["sources"],
                               edges=_edges(case["buckets"]) if case["buckets"] else None)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(case["T"], case["hq"], dtype=torch.float32, device="cuda")
    if case["op"] == "train":
        s["dq"], s["dk"], s["dv"] = (torch.empty_like(s[k]) for k in ("q", "k", "v"))
        s["dbias"] = torch.empty_like(s["bias"]) if s["bias"] is not None else None
    return s


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    op, kind = s["op"], s["case"]["op"]
    if kind in ("norm", "norm_train"):
        op.forward(s["x"], s["weight"], s["bias"], s["y"], residual=s["residual"], z=s["z"])
        if kind == "norm":
            return {"y": s["y"], "z": s["z"]}
        z = s["x"] if s["z"] is None else s["z"]
        op.backward(s["dy"], z, s["weight"], s["dx"], s["dw"], s["db"], dz=s["dz"])
        return {"y": s["y"], "z": s["z"], "dx": s["dx"], "dweight": s["dw"], "dbias": s["db"]}
    table = dict(hops=s["hops"], bias=s["bias"], query_source=s["source"])
    op.forward(s["q"], s["k"], s["v"], s["out"], s["lse"], **table)
    if kind == "read":
        return {"out": s["out"], "lse": s["lse"]}
    op.backward(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], s["dq"], s["dk"], s["dv"], dbias=s["dbias"],
                **table)
    return {"out": s["out"], "dq": s["dq"], "dk": s["dk"], "dv": s["dv"], "dbias": s["dbias"]}


def _plain_bias(s, hq):
    """(index [T, n] of each query's bucket with the last one for a masked node, bias [hq, T, n])."""
    hops, source = s["hops"], s["source"]
    n, table = hops.shape[0], s["bias"].float()
    buckets = table.shape[1]
    index = torch.searchsorted(s["edges"], hops.clamp(min=0), right=True, out_int32=True) - 1
    index = torch.where(hops < 0, buckets + 1, index).t()
    if source is not None:
        index = torch.cat([index, torch.full((1, n), buckets, dtype=index.dtype, device=index.device)])
        index = index[source.long()]
    wide = torch.cat([table, table.new_zeros(hq, 1), table.new_full((hq, 1), -math.inf)], 1)
    return index, wide[:, index]


def _run_plain(s):
    case = s["case"]
    dt = DTYPES[case["dtype"]]
    if case["op"] in ("norm", "norm_train"):
        z = s["x"].float()
        if s["residual"] is not None:
            z = z + s["residual"].float()
        kept = z.to(dt)
        z = kept.float()
        w = s["weight"].float()
        centred = z - z.mean(1, keepdim=True)
        rstd = (centred.square().mean(1, keepdim=True) + 1e-5).rsqrt()
        xh = centred * rstd
        out = {"y": (xh * w + s["bias"].float()).to(dt), "z": kept if case["residual"] else None}
        if case["op"] == "norm_train":
            dy = s["dy"].float()
            wdy = dy * w
            dx = (wdy - wdy.mean(1, keepdim=True) - xh * (wdy * xh).mean(1, keepdim=True)) * rstd
            if s["dz"] is not None:
                dx = dx + s["dz"].float()
            out |= {"dx": dx.to(dt), "dweight": (dy * xh).sum(0).to(dt), "dbias": dy.sum(0).to(dt)}
        return out
    T, n, hq, hkv, d = (case[k] for k in ("T", "n", "hq", "hkv", "d"))
    group, scale = hq // hkv, 1.0 / math.sqrt(d)
    q = s["q"].float().permute(1, 0, 2).reshape(hkv, group * T, d)
    k, v = (s[x].float().permute(1, 0, 2) for x in ("k", "v"))
    scores = (q @ k.transpose(1, 2)).mul_(scale).view(hq, T, n)
    if s["hops"] is not None:
        index, bias = _plain_bias(s, hq)
        scores += bias
    top = scores.amax(2, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = scores.sub_(top).exp_()
    total = p.sum(2, keepdim=True)
    p /= torch.where(total == 0, 1.0, total)
    o = (p.view(hkv, group * T, n) @ v).view(hq, T, d)
    out = {"out": o.permute(1, 0, 2).to(dt).contiguous()}
    if case["op"] == "read":
        return out | {"lse": (top + total.log()).squeeze(2).t().contiguous()}
    do = s["dout"].float().permute(1, 0, 2)
    grouped = do.reshape(hkv, group * T, d)
    ds = (grouped @ v.transpose(1, 2)).view(hq, T, n)
    dv = p.view(hkv, group * T, n).transpose(1, 2) @ grouped
    ds -= (do * o).sum(2, keepdim=True)
    ds *= p
    flat = ds.view(hkv, group * T, n)
    dq = (flat @ k).mul_(scale).view(hq, T, d)
    dk = (flat.transpose(1, 2) @ q).mul_(scale)
    out |= {"dq": dq.permute(1, 0, 2).to(dt).contiguous(), "dk": dk.permute(1, 0, 2).to(dt).contiguous(),
            "dv": dv.permute(1, 0, 2).to(dt).contiguous(), "dbias": None}
    if s["hops"] is not None:
        one = torch.arange(case["buckets"], device="cuda", dtype=index.dtype)
        sums = torch.stack([torch.where(index == b, ds, 0.0).sum((1, 2)) for b in one], 1)
        out["dbias"] = sums.to(dt)
    return out


def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    n, d = case["n"], case["d"]
    if case["op"] == "norm":
        return {"bytes": n * d * e * (4 if case["residual"] else 2), "flops": 8 * n * d}
    if case["op"] == "norm_train":  # x (residual) and dy (dz) in, y (z) and dx out
        return {"bytes": n * d * e * (7 if case["residual"] else 4), "flops": 18 * n * d}
    T, hq, hkv = case["T"], case["hq"], case["hkv"]
    seen = case["seen"] * n  # a node that no query sees need not be read
    product = 2 * T * hq * seen * d
    reads = 2 * seen * hkv * d * e + 4 * n * case["sources"] + 4 * T * (hq if case["op"] == "read" else 0)
    if case["op"] == "read":
        return {"bytes": reads + 2 * T * hq * d * e, "flops": 2 * product}
    return {"bytes": reads + 2 * n * hkv * d * e + 4 * T * hq * d * e, "flops": 6 * product}


def exact(case, seed):
    """The definitions in 64 bits, one head (or the whole norm) at a time."""
    s = _inputs(case, seed)
    f = {k: v.double() for k, v in s.items() if v is not None and v.is_floating_point()}
    dt = DTYPES[case["dtype"]]
    if case["op"] in ("norm", "norm_train"):
        z = f["x"]
        if case["residual"]:
            z = (z + f["residual"]).to(dt).double()  # the sum is kept, and normalised, in the states' type
        var, mean = torch.var_mean(z, dim=1, correction=0, keepdim=True)
        xh = (z - mean) / torch.sqrt(var + 1e-5)
        out = {"y": f["weight"] * xh + f["bias"], "z": z if case["residual"] else None}
        if case["op"] == "norm_train":
            a = f["dy"] * f["weight"]
            c1, c2 = a.sum(1, keepdim=True) / case["d"], (a * xh).sum(1, keepdim=True) / case["d"]
            dx = (a - c1 - xh * c2) / torch.sqrt(var + 1e-5)
            if case["residual"]:
                dx = dx + f["dz"]
            out |= {"dx": dx, "dweight": torch.einsum("nd,nd->d", f["dy"], xh), "dbias": f["dy"].sum(0)}
        return out
    T, n, hq, hkv, d = (case[k] for k in ("T", "n", "hq", "hkv", "d"))
    if s["hops"] is not None:
        edges = _edges(case["buckets"])
        bucket = torch.zeros_like(s["hops"])
        for first in edges[1:]:
            bucket += s["hops"] >= first
        column = s["source"].long() if s["source"] is not None else torch.arange(T, device="cuda")
        informed = column >= 0
        bucket = bucket[:, column.clamp(min=0)].t().long()
        hidden = (s["hops"] < 0)[:, column.clamp(min=0)].t() & informed[:, None]
    out, lse = torch.zeros(T, hq, d, dtype=torch.float64, device="cuda"), torch.zeros(T, hq, dtype=torch.float64, device="cuda")
    train = case["op"] == "train"
    if train:
        dq, dk, dv = torch.zeros_like(f["q"]), torch.zeros_like(f["k"]), torch.zeros_like(f["v"])
        dbias = torch.zeros_like(f["bias"]) if "bias" in f else None
    for h in range(hq):
        kv = h * hkv // hq
        a = torch.einsum("td,nd->tn", f["q"][:, h], f["k"][:, kv]) / math.sqrt(d)
        if s["hops"] is not None:
            a += torch.where(informed[:, None], f["bias"][h][bucket], 0.0)
            a[hidden] = -math.inf
        lse[:, h] = torch.logsumexp(a, 1)
        p = torch.exp(a - lse[:, h, None])
        p[lse[:, h] == -math.inf] = 0
        out[:, h] = p @ f["v"][:, kv]
        if train:
            do = f["dout"][:, h]
            dp = do @ f["v"][:, kv].t()
            ds = p * (dp - (p * dp).sum(1, keepdim=True))
            dq[:, h] = ds @ f["k"][:, kv] / math.sqrt(d)
            dk[:, kv] += ds.t() @ f["q"][:, h] / math.sqrt(d)
            dv[:, kv] += p.t() @ do
            if dbias is not None:
                kept = ds * informed[:, None]
                dbias[h] = torch.stack([kept[bucket == b].sum() for b in range(len(edges))])
    if not train:
        return {"out": out, "lse": lse}
    return {"out": out, "dq": dq, "dk": dk, "dv": dv, "dbias": dbias}
