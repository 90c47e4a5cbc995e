"""The operators with which a model asks a graph whose node states are kept in 8 bits, as measured work.

Three families:
* turn, turn_train: RMS norm of each head of queries or keys, with the rotation by position in the same pass, forward
  and as a training pass;
* store: keys and values of nodes written into a cache of 8-bit values (e4m3) with a power-of-two scale for each block
  of 32 nodes and head, and read back, in their order or by index;
* ask: attention of queries to the nodes of such a cache, with the learned bias by bucket of the hop distance (the
  table k2t_msbfs writes: n x B int32, -1 where a source does not reach a node, which masks it).

``own`` false computes the plain form (elementary torch operations in 32 bits, angles in 64), true calls this package.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK = 32                       # nodes that share a scale
LEAST, MOST = -64, 63            # exponents of a scale
LARGEST = 448.0                  # of e4m3
EPS = 1e-6


def listed():
    return [
        # one entity asks about a graph of the smallest configuration (1024 nodes): a latency-bound call
        dict(name="ask 1 of 1024", op="ask", T=1, n=1024, hq=8, hkv=8, d=64, sources=1, seen=0.9, buckets=16, dtype="bf16"),
        # one entity asks about a graph of 2^20 nodes, grouped heads: the serving form at full size
        dict(name="ask 1 of 2^20", op="ask", T=1, n=1 << 20, hq=16, hkv=4, d=128, sources=1, seen=1.0, buckets=32,
             dtype="bf16"),
        # a full search batch (32 sources) against 2^20 nodes of which the search reaches a part, as on power-law graphs
        dict(name="ask 32 of 2^20", op="ask", T=32, n=1 << 20, hq=16, hkv=4, d=128, sources=32, seen=0.7, buckets=32,
             dtype="bf16"),
        # odd everything: 13 sources, a prime number of nodes, a head size that is no power of two
        dict(name="ask 13 of 100003", op="ask", T=13, n=100003, hq=6, hkv=2, d=72, sources=13, seen=0.8, buckets=11,
             dtype="fp16"),
        # text tokens, each of which mentions one of 32 entities or none, against a retrieved subgraph
        dict(name="ask 1024 tokens", op="ask", T=1024, n=16384, hq=8, hkv=8, d=128, sources=32, seen=0.95, buckets=32,
             dtype="bf16"),
        # one node's states change and are looked at again: a latency-bound update inside a block
        dict(name="store 1 node", op="store", n=1 << 16, first=12345, count=1, fetch=0, hkv=4, d=128, dtype="bf16"),
        # the states of a graph of 2^20 nodes as they are first kept, and brought back to 16 bits
        dict(name="store 2^20 nodes", op="store", n=1 << 20, first=0, count=1 << 20, fetch=0, hkv=4, d=128, dtype="bf16"),
        # a part of a graph is kept again from the products' own type, then a subgraph is fetched by its nodes' numbers
        dict(name="store 99991, fetch 16384", op="store", n=100003, first=12, count=99991, fetch=16384, hkv=2, d=72,
             dtype="fp32"),
        # the queries of one token: a latency-bound call
        dict(name="turn 1 token", op="turn", n=1, heads=16, d=128, rotary=128, paired=False, span=1 << 20, dtype="bf16"),
        # the keys of 2^20 nodes, before they are kept
        dict(name="turn 2^20 nodes", op="turn", n=1 << 20, heads=4, d=128, rotary=128, paired=False, span=1 << 20,
             dtype="bf16"),
        # training over the keys of 2^18 nodes, half of each head turned
        dict(name="turn train 2^18 nodes", op="turn_train", n=1 << 18, heads=8, d=64, rotary=32, paired=False, span=64,
             dtype="bf16"),
        # training over an odd number of tokens, an odd number of heads and neighbouring values turned together
        dict(name="turn train 4999 tokens", op="turn_train", n=4999, heads=6, d=72, rotary=72, paired=True, span=1 << 17,
             dtype="fp32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ask", "ask", "ask", "store", "store", "turn", "turn_train"])
    n = _log_int(rng, 1, 1 << 20)
    if op in ("turn", "turn_train"):
        heads, d = rng.choice([1, 2, 3, 4, 6, 8, 16]), rng.choice([32, 40, 64, 64, 72, 96, 128, 128])
        while n > 1 and n * heads * d > (1 << 29 if op == "turn" else 1 << 27):
            n = n * 3 // 4
        rotary = rng.choice([d, d, d, d // 2 // 2 * 2, 0])
        return dict(op=op, n=n, heads=heads, d=d, rotary=rotary, paired=rng.random() < 0.3,
                    span=_log_int(rng, 64, 1 << 20), dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    hkv = rng.choice([1, 2, 3, 4, 8])
    d = rng.choice([32, 40, 64, 64, 72, 96, 128, 128])
    if op == "store":
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        while n > 1 and n * hkv * d > (1 << (28 if dtype == "fp32" else 29)):
            n = n * 3 // 4
        count = _log_int(rng, 1, n)
        fetch = 0 if rng.random() < 0.5 else _log_int(rng, 1, n)
        return dict(op=op, n=n, first=rng.randint(0, n - count), count=count, fetch=fetch, hkv=hkv, d=d, dtype=dtype)
    T = _log_int(rng, 1, 1024)
    hq = hkv * rng.choice([1, 1, 2, 4])
    while n > 1 and (4 * T * hq * n * d > 2 * 10 ** 11 or n * hkv * d > 1 << 29):
        n = n * 3 // 4
    hops = rng.random() < 0.85
    sources = 0 if not hops else T if T <= 32 else rng.randint(1, 32)
    return dict(op=op, T=T, n=n, hq=hq, hkv=hkv, d=d, sources=sources,
                seen=round(rng.uniform(0.4, 1.0), 2) if hops else 1.0, buckets=rng.randint(2, 32) if hops else 0,
                dtype=rng.choice(["bf16", "bf16", "fp16"]))


def _edges(buckets):
    """First hop of each bucket: one bucket a hop for the first half, then growing ones up to 64 hops."""
    half = (buckets + 1) // 2
    grown = [half + b + int((64 - buckets) * ((b + 1) / (buckets - half)) ** 2) for b in range(buckets - half)]
    return list(range(half)) + grown


def _rand(g, *shape, dtype, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _states(g, n, heads, d, dtype):
    """Node states: the size of a node's states goes with its degree, which differs by a factor of ten."""
    size = torch.rand(n, 1, 1, generator=g, device="cuda").mul_(2.3).exp_().mul_(0.3)
    return torch.randn(n, heads, d, generator=g, device="cuda").mul_(size).to(dtype)


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
    if case["op"] in ("turn", "turn_train"):
        s["x"] = _states(g, n, case["heads"], d, dt)
        s["weight"] = (1 + _rand(g, d, dtype=torch.float32, scale=0.1)).to(dt)
        s["positions"] = torch.randint(0, case["span"], (n,), generator=g, device="cuda", dtype=torch.int32)
        if case["op"] == "turn_train":
            s["dy"] = _rand(g, n, case["heads"], d, dtype=dt)
        return s
    hkv = case["hkv"]
    if case["op"] == "store":
        if case["count"] < n:      # what the cache holds before the call
            s["k_old"], s["v_old"] = _states(g, n, hkv, d, dt), _states(g, n, hkv, d, dt)
        s["k"], s["v"] = _states(g, case["count"], hkv, d, dt), _states(g, case["count"], hkv, d, dt)
        s["nodes"] = torch.randint(0, n, (case["fetch"],), generator=g, device="cuda", dtype=torch.int32) if case["fetch"] else None
        return s
    T, hq = case["T"], case["hq"]
    s["q"] = _rand(g, T, hq, d, dtype=dt)
    s["k"], s["v"] = _states(g, n, hkv, d, dt), _states(g, n, hkv, d, dt)
    s["hops"] = s["bias"] = s["source"] = None
    if case["sources"]:
        s["hops"] = _hops(g, n, case["sources"], case["seen"])
        s["bias"] = _rand(g, hq, case["buckets"], dtype=dt, scale=0.7)
        if case["sources"] != T:
            s["source"] = torch.randint(-1, case["sources"], (T,), generator=g, device="cuda", dtype=torch.int32)
    return s


def _power(exponents):
    """2 to the power of whole numbers from -126 on, exactly."""
    return (exponents.clamp(min=-127) + 127 << 23).view(torch.float32)


def _plain_cache(n, heads, d):
    """A cache in plain tensors: e4m3 values, whole blocks of nodes, and the exponents of their scales."""
    blocks = -(-n // BLOCK)
    return {"values": torch.zeros(blocks * BLOCK, heads, d, device="cuda").to(torch.float8_e4m3fn),
            "exponents": torch.full((blocks, heads), LEAST, device="cuda", dtype=torch.int32)}


def _plain_write(cache, x, first, n):
    """Rows [first, first + len(x)) of a cache of n nodes become x.  A block's exponent is the least that holds its new
    rows, and where rows of it stay, not less than it was: those are rounded again."""
    values, exponents = cache["values"], cache["exponents"]
    b0, b1 = first // BLOCK, -(-(first + len(x)) // BLOCK)
    heads, d = values.shape[1:]
    rows = slice(b0 * BLOCK, b1 * BLOCK)
    fresh = torch.zeros((b1 - b0) * BLOCK, heads, d, device="cuda")
    fresh[first - b0 * BLOCK:first - b0 * BLOCK + len(x)] = x.float()
    top = fresh.abs().view(b1 - b0, BLOCK, heads, d).amax((1, 3))
    mantissa, exponent = torch.frexp(top)
    need = exponent - 9 + (mantissa > LARGEST / 512).to(torch.int32)
    need = torch.where(top == 0, LEAST, need.clamp(LEAST, MOST))
    row = torch.arange(b0 * BLOCK, b1 * BLOCK, device="cuda")
    written = (row >= first) & (row < first + len(x))
    whole = (written | (row >= n)).view(b1 - b0, BLOCK).all(1, keepdim=True)
    old = exponents[b0:b1]
    kept = torch.where(whole, need, torch.maximum(need, old))
    wide = kept.repeat_interleave(BLOCK, 0)[:, :, None]
    stay = values[rows].float() * _power(old.repeat_interleave(BLOCK, 0)[:, :, None] - wide)
    values[rows] = torch.where(written[:, None, None], fresh * _power(-wide), stay).to(torch.float8_e4m3fn)
    exponents[b0:b1] = kept


def _plain_read(cache, rows):
    """The values that rows (a slice, or node numbers) of a cache stand for, in 32 bits."""
    wide = cache["exponents"].repeat_interleave(BLOCK, 0) if isinstance(rows, slice) else cache["exponents"][rows // BLOCK]
    return cache["values"][rows].float() * _power(wide[rows] if isinstance(rows, slice) else wide)[:, :, None]


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    dt, n, d = DTYPES[case["dtype"]], case["n"], case["d"]
    if own:
        import compressed_graph_spmv_gb300 as k2t
    if case["op"] in ("turn", "turn_train"):
        if own:
            s["op"] = k2t.HeadNorm(n, case["heads"], d, dt, rotary_dim=case["rotary"], paired=case["paired"], eps=EPS)
            s["y"] = torch.empty_like(s["x"])
            if case["op"] == "turn_train":
                s["dx"], s["dw"] = torch.empty_like(s["x"]), torch.empty_like(s["weight"])
        return s
    hkv = case["hkv"]
    old = (s.pop("k_old", None), s.pop("v_old", None)) if case["op"] == "store" else (s.pop("k"), s.pop("v"))
    if own:
        s["cache"] = k2t.NodeCache(n, hkv, d, dt)
        if old[0] is not None:
            s["cache"].write(*old)
    else:
        s["cache"] = [_plain_cache(n, hkv, d), _plain_cache(n, hkv, d)]
        if old[0] is not None:
            _plain_write(s["cache"][0], old[0], 0, n)
            _plain_write(s["cache"][1], old[1], 0, n)
    if case["op"] == "store":
        if own:
            back = case["fetch"] or case["count"]
            s["k_back"], s["v_back"] = (torch.empty(back, hkv, d, device="cuda", dtype=dt) for _ in range(2))
        return s
    edges = _edges(case["buckets"]) if case["buckets"] else None
    if own:
        s["op"] = k2t.CachedAttention(case["T"], n, case["hq"], hkv, d, dt, sources=case["sources"], edges=edges)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(case["T"], case["hq"], dtype=torch.float32, device="cuda")
    elif edges:
        s["edges"] = torch.tensor(edges, dtype=torch.int32, device="cuda")
    return s


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    case = s["case"]
    if case["op"] in ("turn", "turn_train"):
        s["op"].forward(s["x"], s["weight"], s["y"], positions=s["positions"])
        if case["op"] == "turn":
            return {"y": s["y"]}
        s["op"].backward(s["dy"], s["x"], s["weight"], s["dx"], s["dw"], positions=s["positions"])
        return {"y": s["y"], "dx": s["dx"], "dweight": s["dw"]}
    if case["op"] == "store":
        s["cache"].write(s["k"], s["v"], first=case["first"])
        s["cache"].read(s["k_back"], s["v_back"], first=case["first"] if s["nodes"] is None else 0, nodes=s["nodes"])
        return {"k": s["k_back"], "v": s["v_back"]}
    s["op"].forward(s["q"], s["cache"], s["out"], s["lse"], hops=s["hops"], bias=s["bias"], query_source=s["source"])
    return {"out": s["out"], "lse": s["lse"]}


def _angles(case, positions):
    """Cosine and sine of each row's angles, [n, 1, rotary / 2]: position times base^(-2 i / rotary), in 64 bits."""
    rate = 10000.0 ** (-torch.arange(0, case["rotary"], 2, device="cuda", dtype=torch.float64) / case["rotary"])
    angle = positions.double()[:, None, None] * rate
    return angle.cos().float(), angle.sin().float()


def _turned(case, x, cos, sin):
    """x with its first `rotary` values turned: value i with i + rotary / 2, or neighbours where they are paired."""
    r = case["rotary"]
    a, b = (x[..., :r:2], x[..., 1:r:2]) if case["paired"] else (x[..., :r // 2], x[..., r // 2:r])
    pair = a * cos - b * sin, b * cos + a * sin
    first = torch.stack(pair, -1).flatten(-2) if case["paired"] else torch.cat(pair, -1)
    return torch.cat([first, x[..., r:]], -1)


def _plain_turn(s):
    case = s["case"]
    dt = DTYPES[case["dtype"]]
    x, w = s["x"].float(), s["weight"].float()
    rstd = (x.square().mean(2, keepdim=True) + EPS).rsqrt()
    cos, sin = _angles(case, s["positions"])
    xh = x * rstd
    out = {"y": _turned(case, xh * w, cos, sin).to(dt)}
    if case["op"] == "turn_train":
        g = _turned(case, s["dy"].float(), cos, -sin)
        wg = g * w
        out |= {"dx": ((wg - xh * (wg * xh).mean(2, keepdim=True)) * rstd).to(dt), "dweight": (g * xh).sum((0, 1)).to(dt)}
    return out


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
    return wide[:, index]


def _run_plain(s):
    case = s["case"]
    dt = DTYPES[case["dtype"]]
    if case["op"] in ("turn", "turn_train"):
        return _plain_turn(s)
    if case["op"] == "store":
        _plain_write(s["cache"][0], s["k"], case["first"], case["n"])
        _plain_write(s["cache"][1], s["v"], case["first"], case["n"])
        rows = slice(case["first"], case["first"] + case["count"]) if s["nodes"] is None else s["nodes"].long()
        return {"k": _plain_read(s["cache"][0], rows).to(dt), "v": _plain_read(s["cache"][1], rows).to(dt)}
    T, n, hq, hkv, d = (case[k] for k in ("T", "n", "hq", "hkv", "d"))
    group, scale = hq // hkv, 1.0 / math.sqrt(d)
    q = s["q"].float().permute(1, 0, 2).reshape(hkv, group * T, d)
    k = _plain_read(s["cache"][0], slice(0, n)).permute(1, 0, 2)
    scores = (q @ k.transpose(1, 2)).mul_(scale).view(hq, T, n)
    del k
    if s["hops"] is not None:
        scores += _plain_bias(s, hq)
    top = scores.amax(2, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = scores.sub_(top).exp_()
    total = p.sum(2, keepdim=True)
    v = _plain_read(s["cache"][1], slice(0, n)).permute(1, 0, 2)
    o = (p.view(hkv, group * T, n) @ v).view(hq, T, d) / torch.where(total == 0, 1.0, total)
    return {"out": o.permute(1, 0, 2).to(dt).contiguous(), "lse": (top + total.log()).squeeze(2).t().contiguous()}


def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    n, d = case["n"], case["d"]
    if case["op"] == "turn":
        return {"bytes": 2 * n * case["heads"] * d * e + 4 * n + d * e, "flops": 8 * n * case["heads"] * d}
    if case["op"] == "turn_train":  # x and dy in, y and dx out
        return {"bytes": 4 * n * case["heads"] * d * e + 4 * n + 2 * d * e, "flops": 24 * n * case["heads"] * d}
    hkv = case["hkv"]
    if case["op"] == "store":  # keys and values in, their 8 bits out; the 8 bits of those asked for in again and out
        count, back = case["count"], case["fetch"] or case["count"]
        return {"bytes": 2 * hkv * d * (count + back) * (e + 1) + 2 * hkv * (count + back) // BLOCK + 4 * case["fetch"],
                "flops": 2 * hkv * d * (3 * count + back)}
    T, hq = case["T"], case["hq"]
    seen = case["seen"] * n  # a node that no query sees need not be read
    reads = 2 * seen * hkv * (d + 1.0 / BLOCK) + 4 * n * case["sources"]
    return {"bytes": reads + 2 * T * hq * d * e + 4 * T * hq, "flops": 4 * T * hq * seen * d}


def _two_to(e):
    """2 to the power of whole numbers held in 64 bits, exactly (a device's pow may be off in the last place)."""
    return (e.clamp(-1022, 1023).long() + 1023 << 52).view(torch.float64)


def _exact_store(x, before, first, n):
    """(values, exponents) of a cache of n nodes in 64 bits, one block of nodes after another in a batch: `before` is
    (values, exponents) of what it held, x its new rows from `first` on."""
    blocks, (heads, d) = -(-n // BLOCK), x.shape[1:]
    at = torch.arange(blocks * BLOCK, device="cuda")
    new = ((at >= first) & (at < first + len(x))).view(blocks, BLOCK)
    rows = torch.zeros(blocks, BLOCK, heads, d, dtype=torch.float64, device="cuda")
    rows[new] = x.double()
    largest = rows.abs().flatten(2).view(blocks, BLOCK, heads, d).amax(3).amax(1)
    e = torch.ceil(torch.log2(largest / LARGEST)).clamp(LEAST, MOST)      # -inf of nothing but zeros: the least
    e = torch.where((largest > LARGEST * _two_to(e)) & (e < MOST), e + 1, e)
    e = torch.where((largest <= LARGEST * _two_to(e - 1)) & (e > LEAST), e - 1, e)
    if before is not None:
        partly = ~(new | (at >= n).view(blocks, BLOCK)).all(1)
        e = torch.where(new.any(1)[:, None], torch.where(partly[:, None], torch.maximum(e, before[1]), e), before[1])
        rows = torch.where(new[:, :, None, None], rows, before[0])
    scale = _two_to(e)[:, None, :, None]
    rows /= scale
    place = torch.floor(torch.log2(rows.abs())).clamp(min=-6)
    step = _two_to(place - 3)
    rows = torch.round(rows / step) * step * scale                          # to the even one where two are as near
    return rows, e


def _exact_turn(case, s):
    f = {k: v.double() for k, v in s.items() if v.is_floating_point()}
    r, d = case["rotary"], case["d"]
    j = torch.arange(r // 2, device="cuda")
    first, second = (2 * j, 2 * j + 1) if case["paired"] else (j, j + r // 2)
    angle = torch.outer(s["positions"].double(), torch.exp(j.double() * (-2.0 / max(r, 1) * math.log(10000.0))))
    turn = torch.polar(torch.ones_like(angle), angle)[:, None, :]
    norm = torch.sqrt(torch.einsum("nhd,nhd->nh", f["x"], f["x"])[..., None] / d + EPS)
    xh = f["x"] / norm

    def rotate(x, by):
        z = torch.complex(x[..., first], x[..., second]) * by
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    out = {"y": rotate(xh * f["weight"], turn)}
    if case["op"] == "turn_train":
        g = rotate(f["dy"], turn.conj())
        a = g * f["weight"]
        out |= {"dx": (a - xh * torch.einsum("nhd,nhd->nh", a, xh)[..., None] / d) / norm, "dweight": torch.einsum("nhd,nhd->d", g, xh)}
    return out


def exact(case, seed):
    """The definitions in 64 bits, one head (or one tensor) at a time."""
    s = _inputs(case, seed)
    if case["op"] in ("turn", "turn_train"):
        return _exact_turn(case, s)
    n, d = case["n"], case["d"]
    if case["op"] == "store":
        out = {}
        for name in ("k", "v"):
            old = _exact_store(s[name + "_old"], None, 0, n) if name + "_old" in s else None
            rows = _exact_store(s[name], old, case["first"], n)[0].flatten(0, 1)
            out[name] = rows[s["nodes"].long()] if s["nodes"] is not None else rows[case["first"]:case["first"] + case["count"]].clone()
            del old, rows
        return out
    T, hq, hkv = case["T"], case["hq"], case["hkv"]
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
    for kv in range(hkv):
        k, v = (_exact_store(s[x][:, kv:kv + 1], None, 0, n)[0].flatten(0, 1)[:n, 0] for x in ("k", "v"))
        for h in range(kv * hq // hkv, (kv + 1) * hq // hkv):
            a = torch.einsum("td,nd->tn", s["q"][:, h].double(), k) / math.sqrt(d)
            if s["hops"] is not None:
                a += torch.where(informed[:, None], s["bias"][h].double()[bucket], 0.0)
                a[hidden] = -math.inf
            lse[:, h] = torch.logsumexp(a, 1)
            p = torch.exp(a - lse[:, h, None])
            p[lse[:, h] == -math.inf] = 0
            out[:, h] = p @ v
    return {"out": out, "lse": lse}
