"""Tensors assigned to a node cache: a call takes what the attribute holds (no GPU but where marked)."""
import pytest

K = pytest.importorskip("compressed_graph_spmv_gb300.k2t")
torch = pytest.importorskip("torch")
import compressed_graph_spmv_gb300 as pkg  # noqa: E402

NAMES = ("k", "v", "k_scale", "v_scale")


def other(t):
    return torch.zeros(t.shape, dtype=torch.uint8, device=t.device).view(t.dtype)


def addresses(c):
    return [[getattr(a, name) for name in NAMES] for a in (c._a, c._held)]


def test_an_assigned_tensor_is_the_one_that_calls_take():
    c = pkg.NodeCache(100, 2, 72, torch.bfloat16, device="cpu")
    kept = [getattr(c, name) for name in NAMES]
    assert addresses(c) == [[t.data_ptr() for t in kept]] * 2
    for i, name in enumerate(NAMES):
        t = other(kept[i])
        setattr(c, name, t)
        assert getattr(c, name) is t
        kept[i] = t
        assert addresses(c) == [[t.data_ptr() for t in kept]] * 2 and not c._streams


def test_what_may_not_be_assigned():
    c = pkg.NodeCache(100, 2, 72, torch.bfloat16, device="cpu")
    before = addresses(c)
    wide = torch.zeros(2, 100, 96, dtype=torch.uint8).view(torch.float8_e4m3fn)
    odd = torch.zeros(2 * 100 * 80 + 8, dtype=torch.uint8)[8:].view(2, 100, 80).view(torch.float8_e4m3fn)
    for name, t, error in (("k", torch.zeros(2, 100, 72).to(torch.float8_e4m3fn), ValueError), ("k", wide[:, :, :80], ValueError),
                           ("v", torch.zeros(2, 100, 80, dtype=torch.uint8), TypeError), ("k_scale", torch.zeros(2, 16, dtype=torch.int8), TypeError),
                           ("v_scale", torch.zeros(2, 4, dtype=torch.uint8), ValueError), ("k", odd, ValueError),
                           ("k", torch.empty(2, 100, 80, dtype=torch.float8_e4m3fn, device="meta"), ValueError)):
        with pytest.raises(error):
            setattr(c, name, t)
        assert addresses(c) == before


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 20])
def test_a_cache_that_was_saved(T):
    """Saved tensors assigned to a new cache, whose own are given back: it reads, answers and is written as the old one."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    n, heads, d = 1000, 2, 64
    g = torch.Generator(device="cuda").manual_seed(T)
    k, v = (torch.randn(n, heads, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(T, heads, d, generator=g, device="cuda").bfloat16()
    old = pkg.NodeCache(n, heads, d, torch.bfloat16)
    old.write(k, v)
    new = pkg.NodeCache(n, heads, d, torch.bfloat16)
    op = pkg.CachedAttention(T, n, heads, heads, d, torch.bfloat16)
    answers = [(torch.empty_like(q), torch.empty(T, heads, device="cuda")) for _ in range(3)]
    op.forward(q, old, *answers[0])
    op.forward(q, new, *answers[1])
    for name in NAMES:
        saved = getattr(old, name).view(torch.uint8).cpu()
        setattr(new, name, saved.cuda().view(getattr(old, name).dtype))
    filler = [torch.full((heads, n, d), 0x7f, dtype=torch.uint8, device="cuda") for _ in range(4)]      # over what was given back
    op.forward(q, new, *answers[2])
    assert torch.equal(answers[0][0], answers[2][0]) and torch.equal(answers[0][1], answers[2][1])
    back = [torch.empty_like(k) for _ in range(4)]
    old.read(back[0], back[1])
    new.read(back[2], back[3])
    assert torch.equal(back[0], back[2]) and torch.equal(back[1], back[3])
    for c in (old, new):
        c.write(v[:33], k[:33], first=5)
    old.read(back[0], back[1])
    new.read(back[2], back[3])
    assert torch.equal(back[0], back[2]) and torch.equal(back[1], back[3]) and len(filler) == 4
