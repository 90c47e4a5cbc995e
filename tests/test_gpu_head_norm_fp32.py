"""The head norm in fp32 to the last bits: angles, sine and cosine apart from the norm, and the norm apart from them.

u is 2^-24.  Angles: a head of pairs (1, 0) shows r cos and r sin, and its row at position 0 the same r exactly.  An angle is held
to 2^-26 turns (24 bits of half a turn) and 2^-33 (rates), sine and cosine to 2 ulp of at most u, the product is rounded
once (values below 2: u):
  |y - r cos| <= r (2 pi (2^-26 + 2^-33) + 2 u) + u
The fast sine and cosine of 16-bit calls (2^-21.4 and 2^-21.2, and an angle rounded to 24 bits of pi) are outside of it.

Norm, without rotation: the sum of squares adds at most 14 values in a row (14 u, half of it after the root), the mean, eps and its
sum 2 u (half), the reciprocal root is 2 ulp (4 u), so that r is right to 12 u; y = x r w has two products more:
  |y|  14 u
  dx = r (w g - x r^2 m), m = mean(w g x):  16 u |r w g| + 42 u |r x r^2 m| + 16 u |r x r^2| mean |w g x| + u |dx|
(three r, their products and the sum of 14 in a row of the second term).
"""
import numpy as np
import pytest

from test_gpu_reader import close, f64

pytestmark = pytest.mark.gpu

K = pytest.importorskip("compressed_graph_spmv_gb300.k2t")
import compressed_graph_spmv_gb300 as pkg  # noqa: E402

torch = pytest.importorskip("torch")
u = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    K.load()


@pytest.mark.parametrize("paired", [False, True])
@pytest.mark.parametrize("n,heads,d,rotary", [(20000, 1, 8, 8), (40000, 2, 128, 128), (9000, 3, 72, 72), (7001, 2, 72, 36), (5000, 1, 248, 246)])
def test_angles(n, heads, d, rotary, paired):
    rng = np.random.default_rng(n)
    at = rng.integers(-(1 << 20), 1 << 20, size=n).astype(np.int32)       # positions times rates are exact to 2^-33 in 64 bits
    at[0] = 0
    m = np.arange(rotary // 2)
    first, second = (2 * m, 2 * m + 1) if paired else (m, m + rotary // 2)
    x = torch.zeros(n, heads, d, device="cuda")
    x[:, :, torch.from_numpy(first).cuda()] = 1
    y = torch.full_like(x, float("nan"))
    pkg.HeadNorm(n, heads, d, torch.float32, rotary_dim=rotary, paired=paired).forward(x, None, y, positions=torch.from_numpy(at).cuda())
    got = f64(y)
    r = got[0, 0, first[0]]
    assert np.all(got[0][:, first] == r) and not got[0][:, second].any()
    angle = at[:, None].astype(np.float64) * 10000.0 ** (-2.0 * m / rotary)
    tol = np.full((n, heads, rotary // 2), r * (2 * np.pi * (2.0 ** -26 + 2.0 ** -33) + 2 * u) + u)
    assert r < 2
    for part, want in ((first, np.cos(angle)), (second, np.sin(angle))):
        close("turned", y[:, :, torch.from_numpy(part).cuda()], np.repeat(r * want[:, None], heads, 1), tol)


@pytest.mark.parametrize("n,heads,d", [(3, 2, 8), (500, 3, 40), (70, 2, 256), (40000, 4, 128), (9001, 1, 72)])
def test_norm(n, heads, d):
    rng = np.random.default_rng(d)
    x, dy, w = (torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda() for s in ((n, heads, d), (n, heads, d), (d,)))
    x *= torch.from_numpy(np.exp(rng.uniform(-3, 3, size=(n, heads, 1))).astype(np.float32)).cuda()
    op = pkg.HeadNorm(n, heads, d, torch.float32, rotary_dim=0)
    y, dx, dw = torch.full_like(x, float("nan")), torch.full_like(x, float("nan")), torch.empty_like(w)
    op.forward(x, w, y)
    op.backward(dy, x, w, dx, dw)
    xs, g, ws = f64(x), f64(dy), f64(w)
    r = 1 / np.sqrt((xs * xs).mean(axis=2, keepdims=True) + float(np.float32(1e-6)))
    want = xs * r * ws
    close("y", y, want, 14 * u * np.abs(want))
    m, size = (ws * g * xs).mean(axis=2, keepdims=True), np.abs(ws * g * xs).mean(axis=2, keepdims=True)
    far = r * xs * r * r
    want = r * ws * g - far * m
    close("dx", dx, want, 16 * u * np.abs(r * ws * g) + 42 * u * np.abs(far * m) + 16 * u * np.abs(far) * size + u * np.abs(want))
