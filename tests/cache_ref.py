"""64-bit references of the 8-bit node cache and of the head norm, and how far
a kernel may be off from rounding alone.

Cache: nothing is off.  A value times a power of two is exact, the rounding to
e4m3 is defined for every value, and reading back multiplies exactly.

Head norm.  u: unit roundoff of the element type.  fp32 sums of at most 256
squares in trees of at most 16 in a row, a reciprocal square root (2 ulp) and
three products: a relative 2^-19 at most.  An angle in turns is rounded to
fp32 (2^-26 turns) and, in 16 bits, sine and cosine are off by 2^-21.1 in
[-pi, pi] after a product (2^-24 pi): 2^-19 in all; in fp32 2^-20.  With E the
sum of both (2^-18 and 2^-18.4, 2^-18 here) and (a, b) a pair before it turns:
  y  <= u |y| + E (|a| + |b|)
  g  <= E (|dy_a| + |dy_b|) =: G            (fp32 inside the kernel)
  dx <= u |dx| + r (|w| G + |x| r^2 mean(|w| G |x|)) + E r (|w g| + |x| r^2 mean |w g x|)
  dw <= u |dw| + sum G |x| r + 2^-18 sum |g x| r
(sums of dw: at most 64 terms a thread in a row, then trees).
fp16 results below 2^-14 are subnormal: half a step of 2^-24 more.
"""
import numpy as np

from reader_ref import U

LEAST, MOST, BLOCK = -64, 63, 32


def to_e4m3(x):
    """x (|x| <= 448, or NaN) rounded to the nearest e4m3 value, ties to even."""
    with np.errstate(divide="ignore", invalid="ignore"):
        place = np.maximum(np.floor(np.log2(np.abs(x))), -6)
        place = np.where(np.abs(x) >= 2.0 ** (place + 1), place + 1, np.where((np.abs(x) < 2.0 ** place) & (place > -6), place - 1, place))
        step = 2.0 ** (place - 3)
        y = np.round(x / step) * step
    return np.where(np.isnan(x), np.nan, np.clip(np.where(x == 0, 0.0, y), -448, 448))


def exponent_for(top):
    e = LEAST
    while e < MOST and top > 448.0 * 2.0 ** e:
        e += 1
    return e


class Cache:
    """What a cache holds, node by node."""

    def __init__(self, n, heads, d):
        self.values = np.zeros((n, heads, d))                       # e4m3 values, before the scale
        self.e = np.full((-(-n // BLOCK), heads), LEAST)
        self.n = n

    def write(self, x, first):
        n, heads = self.n, self.values.shape[1]
        for b in range(first // BLOCK, -(-(first + len(x)) // BLOCK) if len(x) else 0):
            rows = np.arange(b * BLOCK, min(n, (b + 1) * BLOCK))
            new = (rows >= first) & (rows < first + len(x))
            for h in range(heads):
                fresh = x[rows[new] - first, h].astype(np.float64)
                fine = np.abs(fresh[np.isfinite(fresh)])
                e = exponent_for(fine.max() if fine.size else 0.0)
                if not new.all():
                    e = max(e, self.e[b, h])
                    self.values[rows[~new], h] = to_e4m3(self.values[rows[~new], h] * 2.0 ** (self.e[b, h] - e))
                fresh = np.where(np.isfinite(fresh), np.clip(fresh * 2.0 ** -e, -448, 448), np.nan)
                self.values[rows[new], h] = to_e4m3(fresh)
                self.e[b, h] = e

    def read(self):
        return self.values * 2.0 ** np.repeat(self.e, BLOCK, axis=0)[:self.n, :, None]


def angles(positions, rotary, base=10000.0):
    m = np.arange(rotary // 2)
    return np.asarray(positions, np.float64)[:, None] * base ** (-2.0 * m / max(rotary, 1))


def turn(x, angle, rotary, paired):
    """The first `rotary` values of each head turned by angle [rows, rotary / 2]."""
    m = np.arange(rotary // 2)
    a, b = (2 * m, 2 * m + 1) if paired else (m, m + rotary // 2)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    y = x.copy()
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y


def partner(x, rotary, paired):
    """|a| + |b| of a value's pair (|x| of one that does not turn)."""
    m = np.arange(rotary // 2)
    a, b = (2 * m, 2 * m + 1) if paired else (m, m + rotary // 2)
    y = np.abs(x)
    y[..., a] = y[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y


def head_norm(x, weight, angle, rotary, paired, eps):
    r = 1 / np.sqrt((x * x).mean(axis=2, keepdims=True) + eps)
    return turn(x * r * weight, angle, rotary, paired), r


def head_norm_gradients(dy, x, weight, angle, rotary, paired, eps):
    r = 1 / np.sqrt((x * x).mean(axis=2, keepdims=True) + eps)
    g = turn(dy, -angle, rotary, paired)
    dx = r * (weight * g - x * r * r * (weight * g * x).mean(axis=2, keepdims=True))
    return dx, (g * x * r).sum(axis=(0, 1)), g, r


def head_norm_tolerances(dtype, x, dy, weight, angle, rotary, paired, eps):
    u, E, least = U[dtype], 2.0 ** -18, 2.0 ** -25 if dtype == "fp16" else 0.0
    y, r = head_norm(x, weight, angle, rotary, paired, eps)
    tol = {"y": u * np.abs(y) + E * partner(x * r * weight, rotary, paired) + least}
    dx, dw, g, r = head_norm_gradients(dy, x, weight, angle, rotary, paired, eps)
    G, w, a = E * partner(dy, rotary, paired), np.abs(weight), np.abs(x)
    mean = lambda z: z.mean(axis=2, keepdims=True)  # noqa: E731
    tol["dx"] = u * np.abs(dx) + r * (w * G + a * r * r * mean(w * G * a)) + E * r * (np.abs(w * g) + a * r * r * mean(np.abs(w * g * x))) + least
    tol["dweight"] = u * np.abs(dw) + (G * a * r).sum(axis=(0, 1)) + 2.0 ** -18 * np.abs(g * x * r).sum(axis=(0, 1)) + least
    return tol
