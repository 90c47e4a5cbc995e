"""64-bit references of the graph-reading operators, and how far a kernel may
be off, element by element, from rounding alone.

Tolerances.  u is the unit roundoff of the element type (bf16 2^-8, fp16
2^-11, fp32 2^-24).  A score is a fp32 dot product of d exact products plus a
bias: its error is at most es = (d + 8) 2^-24 (scale sum|q k| + |bias|), the
largest over the case.  A weight exp(s - lse) is then off by a factor within
2.5 es + 2^-20 (score, lse, exp2 in fp32), called w.  Sums in fp32 add at most
2^-18 of their absolute terms here (a few thousand terms in trees of at most
64 in a row).  With weights rounded to u before they multiply v:
  out   <= u |out| + (u + w + 2^-18) sum p |v|
  delta <= sum_d |dout| tol(out)
  ds    <= p (w |dp - delta| + tol(delta) + d 2^-24 sum|dout v|) + u |ds|
  dv    <= u |dv| + (u + w + 2^-18) sum p |dout|
  dk    <= u |dk| + scale sum (tol(ds) + 2^-18 |ds|) |q|, dq alike
  dbias <= u |dbias| + sum (tol(ds) + 2^-18 |ds|)
"""
import numpy as np

U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
MASKED = {"bf16": -1e38, "fp16": -65504.0}


def bucket_of(hops, edges):
    return np.searchsorted(np.asarray(edges), np.maximum(hops, 0), side="right") - 1


def scores(q, k, scale, dtype="bf16", hops=None, bias=None, edges=None, source=None):
    """s [T, hq, n] (-inf where masked) and the bucket [T, n] of each pair (-1: no gradient for the table)."""
    T, hq, d = q.shape
    n, hkv = k.shape[0], k.shape[1]
    s = scale * np.einsum("thd,nhd->thn", q, np.repeat(k, hq // hkv, axis=1))
    bucket = np.full((T, n), -1)
    if hops is not None:
        for t in range(T):
            c = t if source is None else int(source[t])
            if not 0 <= c < hops.shape[1]:
                continue
            bucket[t] = bucket_of(hops[:, c], edges) if edges else -1
            for h in range(hq):
                if bias is not None:
                    table = np.where(bias[h] <= MASKED[dtype], -np.inf, bias[h])
                    s[t, h] += table[bucket[t]]
                s[t, h][hops[:, c] < 0] = -np.inf
    return s, bucket


def attention(q, k, v, scale, **table):
    s, bucket = scores(q, k, scale, **table)
    group = q.shape[1] // k.shape[1]
    if s.shape[2]:
        top = s.max(axis=2, keepdims=True)
    else:
        top = np.full(s.shape[:2] + (1,), -np.inf)
    e = np.where(np.isneginf(top), 0.0, np.exp(s - np.where(np.isneginf(top), 0.0, top)))
    total = e.sum(axis=2, keepdims=True)
    p = e / np.where(total == 0, 1.0, total)
    with np.errstate(divide="ignore"):
        lse = (top + np.log(total))[:, :, 0]
    out = np.einsum("thn,nhd->thd", p, np.repeat(v, group, axis=1))
    return out, lse, p, s, bucket


def gradients(q, k, v, dout, scale, n_buckets=0, **table):
    out, lse, p, s, bucket = attention(q, k, v, scale, **table)
    T, hq, d = q.shape
    n, hkv = k.shape[:2]
    group = hq // hkv
    kk, vv = np.repeat(k, group, axis=1), np.repeat(v, group, axis=1)
    dp = np.einsum("thd,nhd->thn", dout, vv)
    ds = p * (dp - (dout * out).sum(axis=2)[:, :, None])
    dq = scale * np.einsum("thn,nhd->thd", ds, kk)
    dk = scale * np.einsum("thn,thd->nhd", ds, q).reshape(n, hkv, group, d).sum(axis=2)
    dv = np.einsum("thn,thd->nhd", p, dout).reshape(n, hkv, group, d).sum(axis=2)
    dbias = np.zeros((hq, n_buckets))
    for b in range(n_buckets):
        dbias[:, b] = np.where((bucket == b)[:, None, :], ds, 0.0).sum(axis=(0, 2))
    return dict(out=out, lse=lse, dq=dq, dk=dk, dv=dv, dbias=dbias, p=p, ds=ds, dp=dp, bucket=bucket)


def attention_tolerances(q, k, v, scale, dtype, bias=None, dout=None, ref=None):
    """Per-element bounds (see above); ref is gradients()' dict (dout given) or attention()'s (out, lse, p, ...)."""
    u, sums = U[dtype], 2.0 ** -18
    group = q.shape[1] // k.shape[1]
    T, hq, d = q.shape
    n, hkv = k.shape[:2]
    kk, vv = np.repeat(k, group, axis=1), np.repeat(v, group, axis=1)
    p = ref["p"] if dout is not None else ref[2]
    out = ref["out"] if dout is not None else ref[0]
    size = scale * np.einsum("thd,nhd->thn", np.abs(q), np.abs(kk))
    size = size.max() if size.size else 0.0
    if bias is not None:
        fine = bias[np.isfinite(bias) & (bias > MASKED[dtype])]
        size += np.abs(fine).max() if fine.size else 0.0
    es = (d + 8) * 2.0 ** -24 * size
    w = 2.5 * es + 2.0 ** -20
    tol = {"out": u * np.abs(out) + (u + w + sums) * np.einsum("thn,nhd->thd", p, np.abs(vv)),
           "lse": np.full((T, hq), es + 1e-5 + 2.0 ** -22 * size)}
    if dout is None:
        return tol
    ds, dp = ref["ds"], ref["dp"]
    delta = (dout * out).sum(axis=2)[:, :, None]
    e_delta = (np.abs(dout) * tol["out"]).sum(axis=2)[:, :, None] + d * 2.0 ** -24 * np.abs(dout * out).sum(axis=2)[:, :, None]
    e_dp = d * 2.0 ** -24 * np.einsum("thd,nhd->thn", np.abs(dout), np.abs(vv))
    e_ds = p * (w * np.abs(dp - delta) + e_delta + e_dp) + (u + sums) * np.abs(ds)
    fold = lambda x: x.reshape(n, hkv, group, d).sum(axis=2)  # noqa: E731
    tol["dv"] = u * np.abs(ref["dv"]) + (u + w + sums) * fold(np.einsum("thn,thd->nhd", p, np.abs(dout)))
    tol["dk"] = u * np.abs(ref["dk"]) + scale * fold(np.einsum("thn,thd->nhd", e_ds, np.abs(q)))
    tol["dq"] = u * np.abs(ref["dq"]) + scale * np.einsum("thn,nhd->thd", e_ds, np.abs(kk))
    nb = ref["dbias"].shape[1]
    tol["dbias"] = u * np.abs(ref["dbias"])
    for b in range(nb):
        tol["dbias"][:, b] += np.where((ref["bucket"] == b)[:, None, :], e_ds, 0.0).sum(axis=(0, 2))
    if dtype == "fp16":   # fp16 results and rounded terms below 2^-14 are subnormal: half a step of 2^-24 each
        step = 2.0 ** -25
        pq, pk, pd = (np.abs(x).max() if x.size else 0.0 for x in (q, k, dout))
        for name in ("out", "dq", "dk", "dv", "dbias"):
            tol[name] = tol[name] + step
        tol["out"] += step * (np.abs(vv).sum(axis=0)[None] if n else 0.0)
        tol["dv"] += step * pd * T * group
        tol["dk"] += step * scale * pq * T * group
        tol["dq"] += step * scale * pk * n
        tol["dbias"] += step * T * n
    return tol


def norm(x, weight, bias, eps, residual=None, round_to=lambda z: z):
    z = x if residual is None else round_to(x + residual)
    mean = z.mean(axis=1, keepdims=True)
    var = ((z - mean) ** 2).mean(axis=1, keepdims=True)
    xh = (z - mean) / np.sqrt(var + eps)
    return weight * xh + (0.0 if bias is None else bias), z, mean, 1 / np.sqrt(var + eps), xh


def norm_gradients(dy, xh, rstd, weight, dz=None):
    a = dy * weight
    dx = rstd * (a - a.mean(axis=1, keepdims=True) - xh * (a * xh).mean(axis=1, keepdims=True))
    return dx + (0.0 if dz is None else dz), (dy * xh).sum(axis=0), dy.sum(axis=0)
