"""Rotary positions on the GPU against their definition in float64.

Tolerance: the angle, a fraction of a half turn rounded to float32, is off by at most
pi 2^-25, sine and cosine by 2^-23 more (two units in the last place), the two products
and their sum by 3 2^-24: less than 2^-21 (|u| + |v|) together.  16-bit types take the
hardware's sine and cosine, off by 2^-21.1 at most between -pi and pi: less than 2^-20
(|u| + |v|) together.  For positions x and
frequencies f, f / (2 pi) in float64 loses 2^-52 x f, the fraction of 2^64 another 2^-61
x, a float32 position's cut 2^-32 f.  The result is rounded once: half a step of its type.
"""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

F32, BF, HF = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def pkg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import differentiable_image_quality_gb300 as pkg
    from differentiable_image_quality_gb300 import _build

    _build.build()
    return pkg


def normal(gen, *shape, dtype=F32):
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def definition(x, positions, frequencies, pairs, layout, sign=1.0):
    """(result in float64, the largest error it may have)."""
    n, dim = sum(pairs), x.shape[-1]
    columns = torch.arange(2 * n, device="cuda").view(2, n) if layout == "half" else \
        torch.arange(2 * n, device="cuda").view(n, 2).T
    axis = torch.cat([torch.full((m,), i, device="cuda") for i, m in enumerate(pairs)])
    at = positions.double()[..., axis]
    angle = (at * frequencies)[..., None, :] * sign
    cos, sin = angle.cos(), angle.sin()
    wide = x.double()
    u, v = wide[..., columns[0]], wide[..., columns[1]]
    out, bound = wide.clone(), torch.zeros_like(wide)
    out[..., columns[0]] = u * cos - v * sin
    out[..., columns[1]] = u * sin + v * cos
    far = (at.abs() * (frequencies.abs() * 2.0 ** -51 + 2.0 ** -61) +
           frequencies.abs() * 2.0 ** -32)[..., None, :]
    size = (2.0 ** (-21 if x.dtype == F32 else -20) + far) * (u.abs() + v.abs())
    bound[..., columns[0]] = bound[..., columns[1]] = size
    u = torch.finfo(x.dtype).eps / 2
    rounding = u * out.abs() + (2.0 ** -25 if x.dtype == HF else 0.0)
    rounding[..., [c for c in range(dim) if c >= 2 * n]] = 0.0  # copied
    return out, bound * (1 + u) + rounding


def check(got, x, positions, frequencies, pairs, layout, sign=1.0):
    assert got.shape == x.shape and got.dtype == x.dtype and got.is_contiguous()
    ref, bound = definition(x, positions, frequencies, pairs, layout, sign)
    assert ((got.double() - ref).abs() <= bound).all(), \
        ((got.double() - ref).abs() / bound.clamp_min(1e-30)).max().item()


# tokens, q heads, k heads, dim, pairs, type
CASES = [
    (1, 1, 1, 2, (1,), F32),
    (64, 8, 8, 32, (8, 8), BF),
    (1000, 6, 2, 128, (16, 24, 24), BF),     # halves in whole chunks
    (333, 5, 3, 96, (16,), HF),              # columns without a position, in chunks
    (257, 3, 1, 64, (15, 16), F32),          # halves at any offset
    (257, 3, 1, 64, (15, 16), HF),
    (130, 7, 7, 72, (18, 18), BF),
    (50, 2, 2, 88, (20, 20), F32),
    (50, 1, 9, 40, (3, 2, 1), BF),
    (77, 4, 2, 30, (5, 4), HF),              # single columns
    (9, 3, 3, 7, (1, 1, 1), F32),
    (3, 2, 1, 512, (64, 64, 64, 64), BF),
    (3, 2, 1, 511, (200, 55), F32),
    (20000, 2, 1, 64, (16, 16), BF),         # more tokens than one round of blocks
]


@pytest.mark.parametrize("layout", ["half", "adjacent"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_rotary(pkg, case, layout):
    T, H, K, D, pairs, dtype = case
    gen = torch.Generator(device="cuda").manual_seed(1)
    f = pkg.rotary_frequencies(pairs)
    for positions in (torch.randint(-70, 5000, (T, len(pairs)), generator=gen, device="cuda"),
                      torch.randint(0, 2 ** 31 - 1, (2, T, len(pairs)), generator=gen,
                                    device="cuda", dtype=torch.int32),
                      normal(gen, T, len(pairs)) * 300):
        q, k = normal(gen, 2, T, H, D, dtype=dtype), normal(gen, 2, T, K, D, dtype=dtype)
        for inverse in (False, True):
            got = pkg.rotary(q, k, positions, f, pairs, layout=layout, inverse=inverse)
            for t, x in zip(got, (q, k)):
                check(t, x, positions, f, pairs, layout, -1.0 if inverse else 1.0)


def test_positions_that_are_far(pkg):
    """64-bit positions up to 2^40: what float64 keeps of the angle itself."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    f = pkg.rotary_frequencies((32,))
    at = torch.tensor([[2 ** 40 + 1], [-2 ** 33], [2 ** 24 + 1], [0]], device="cuda")
    q = normal(gen, 4, 2, 64)
    check(pkg.rotary(q, None, at, f, (32,))[0], q, at, f, (32,), "half")
    # whole turns and powers of two wrap without loss
    quarter = torch.full((1,), torch.pi / 2, dtype=torch.float64, device="cuda")
    turns = torch.tensor([[4 * 10 ** 6 + 1]], device="cuda")
    out = pkg.rotary(torch.tensor([[[1.0, 0.0]]], device="cuda"), None, turns, quarter, (1,))[0]
    assert (out.flatten() - torch.tensor([0.0, 1.0], device="cuda")).abs().max() < 1e-6


def test_nan_positions_and_frequencies(pkg):
    """They reach their tokens' pairs of that axis, nothing else."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    q = normal(gen, 5, 2, 24)
    pairs = (4, 4)
    f = pkg.rotary_frequencies(pairs)
    at = torch.rand(5, 2, device="cuda") * 10
    clean = pkg.rotary(q, None, at, f, pairs)[0]
    at[2, 1], at[3, 0] = float("nan"), float("inf")
    out = pkg.rotary(q, None, at, f, pairs)[0]
    bad = torch.zeros_like(q, dtype=torch.bool)
    bad[2, :, 4:8] = bad[2, :, 12:16] = bad[3, :, 0:4] = bad[3, :, 8:12] = True
    assert out[bad].isnan().all() and torch.equal(out[~bad], clean[~bad])
    # NaN among the columns without a position, and beside it
    q[1, 0, 20] = float("nan")
    out = pkg.rotary(q, None, at, f, pairs)[0]
    bad[1, 0, 20] = True
    assert torch.equal(out.isnan(), bad)


@pytest.mark.parametrize("layout", ["half", "adjacent"])
@pytest.mark.parametrize("D", [64, 60])
def test_strides(pkg, D, layout):
    """Slices of one product, heads before tokens, odd addresses, expanded heads."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    pairs = (12, 11)
    f, at = pkg.rotary_frequencies(pairs), torch.arange(120, device="cuda").view(60, 2)
    wide = normal(gen, 2, 60, 5 * D, dtype=BF)
    q, k = wide[..., :3 * D].unflatten(-1, (3, D)), wide[..., 3 * D:].unflatten(-1, (2, D))
    dense = pkg.rotary(q.contiguous(), k.contiguous(), at, f, pairs, layout=layout)
    odd = torch.empty(q.numel() + 3, dtype=BF, device="cuda")[3:].view(q.shape).copy_(q)
    turned = q.transpose(1, 2).contiguous().transpose(1, 2)
    for x in (q, odd, turned):
        got = pkg.rotary(x, k, at, f, pairs, layout=layout)
        assert torch.equal(got[0], dense[0]) and torch.equal(got[1], dense[1])
    one = k[:, :, :1].expand(-1, -1, 4, -1)
    got = pkg.rotary(one, None, at, f, pairs, layout=layout)
    assert got[1] is None
    for h in range(4):
        assert torch.equal(got[0][:, :, h], dense[1][:, :, 0])
    packed = pkg.rotary(q[0], k[0], at, f, pairs, layout=layout)
    assert torch.equal(packed[0], dense[0][0]) and torch.equal(packed[1], dense[1][0])


@pytest.mark.parametrize("layout", ["half", "adjacent"])
def test_gradients(pkg, layout):
    """Against autograd through the definition, and against differences: the operator is
    linear, so a difference is the operator of the step."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    pairs, T = (5, 6), 40
    f, at = pkg.rotary_frequencies(pairs), torch.randint(0, 99, (T, 2), generator=gen, device="cuda")
    q, k = normal(gen, 2, T, 3, 24).requires_grad_(), normal(gen, 2, T, 1, 24).requires_grad_()
    gq, gk = normal(gen, *q.shape), normal(gen, *k.shape)
    out = pkg.fused_rotary(q, k, at, f, pairs, layout=layout)
    got = torch.autograd.grad(out, (q, k), (gq, gk), retain_graph=True)
    for t, g, x in zip(got, (gq, gk), (q, k)):
        wide = x.detach().double().requires_grad_()
        ref, = torch.autograd.grad(definition(wide, at, f, pairs, layout)[0], wide, g.double())
        _, bound = definition(g, at, f, pairs, layout, -1.0)
        assert ((t.double() - ref).abs() <= bound).all()
    # one output's gradient alone; a gradient whose columns are no neighbours
    only, = torch.autograd.grad(out[1], k, gk, retain_graph=True)
    assert torch.equal(only, got[1])
    turned = gq.transpose(-1, -2).contiguous().transpose(-1, -2)
    again, = torch.autograd.grad(out[0], q, turned)
    assert torch.equal(again, got[0])
    step = normal(gen, *q.shape)
    moved = [definition(q.detach() + s * step, at, f, pairs, layout)[0] for s in (1, -1)]
    change = (moved[0] - moved[1]).mul(gq.double()).sum()
    along = (2 * step.double() * got[0].double()).sum()
    slack = (2 * step.abs().double() * definition(gq, at, f, pairs, layout, -1.0)[1]).sum()
    # the moved inputs themselves are rounded to float32
    slack += (gq.abs().double() * 2.0 ** -22 * (q.detach().abs() + step.abs()).sum(-1, keepdim=True)).sum()
    assert (change - along).abs() <= slack


def test_empty(pkg):
    f = pkg.rotary_frequencies((4,))
    q = torch.empty(2, 0, 3, 16, device="cuda")
    out, _ = pkg.rotary(q, None, torch.empty(0, 1, dtype=torch.int32, device="cuda"), f, (4,))
    assert out.shape == q.shape


def test_in_a_graph_and_on_another_stream(pkg):
    gen = torch.Generator(device="cuda").manual_seed(7)
    pairs = (8, 8)
    f, at = pkg.rotary_frequencies(pairs), torch.randint(0, 64, (50, 2), generator=gen, device="cuda")
    q = normal(gen, 2, 50, 4, 32, dtype=BF)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        first = pkg.rotary(q, None, at, f, pairs)[0]
    stream.synchronize()
    assert torch.equal(first, pkg.rotary(q, None, at, f, pairs)[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = pkg.rotary(q, None, at, f, pairs, inverse=True)[0]
    q.copy_(normal(gen, *q.shape, dtype=BF))
    at.add_(3)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, pkg.rotary(q, None, at, f, pairs, inverse=True)[0])


def test_refusals(pkg):
    f = pkg.rotary_frequencies((4, 4))
    q, at = torch.zeros(2, 6, 3, 32, device="cuda"), torch.zeros(6, 2, device="cuda")

    def bad(error, q=q, k=None, at=at, f=f, pairs=(4, 4), **kw):
        with pytest.raises(error):
            pkg.fused_rotary(q, k, at, f, pairs, **kw)

    bad(TypeError, q=q.double())
    bad(TypeError, at=at.half())
    bad(TypeError, f=f.float())
    bad(TypeError, pairs=(4.0, 4.0))
    bad(TypeError, k=q.cpu())
    bad(ValueError, at=at.cpu())
    bad(ValueError, f=f.cpu())
    bad(ValueError, layout="interleaved")
    bad(ValueError, pairs=(4, 5))
    bad(ValueError, pairs=(8, 0))
    bad(ValueError, pairs=())
    bad(ValueError, pairs=(8,))
    bad(ValueError, at=at[:5])
    bad(ValueError, at=at.expand(3, 6, 2))
    bad(ValueError, at=torch.zeros(2, 6, device="cuda").T)
    bad(ValueError, k=q[:, :5])
    bad(ValueError, k=q.bfloat16())
    bad(ValueError, q=q[0, 0])
    bad(ValueError, q=q.transpose(-1, -2).contiguous().transpose(-1, -2))
    bad(ValueError, q=torch.zeros(2, 6, 1, 514, device="cuda"))
    bad(ValueError, q=q[..., :14])
