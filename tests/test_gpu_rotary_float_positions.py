"""Rotary positions that are no whole numbers, with frequencies above a turn a unit or below
zero: what normalised image coordinates come with.

Tolerance: the angle x f in float64, here and in the definition, is off by 2^-51 |x f|;
positions are cut at 2^-64 of a unit and fractions of a turn at 2^-64, 2^-61 (|f| + |x|)
together in radians; from there on as in test_gpu_rotary: less than 2^-21 (float32) or
2^-20 (16 bits) of |u| + |v|, and the result's one rounding.
"""
import math

import pytest

from test_gpu_rotary import BF, F32, HF, definition, normal, pkg  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

RATES = [-0.75, -1.0, 7.0, 7.25, 20 * math.pi, -20 * math.pi, 0.3, -2.0 ** 20 * math.pi]


def within(got, x, at, f, pairs, layout, sign=1.0):
    ref, _ = definition(x, at, f, pairs, layout, sign)
    n = sum(pairs)
    axis = torch.cat([torch.full((m,), i, device="cuda") for i, m in enumerate(pairs)])
    where = at.double().abs()[..., axis]
    off = (where * f.abs() * 2.0 ** -51 + (where + f.abs()) * 2.0 ** -61)[..., None, :]
    off = off + 2.0 ** (-21 if x.dtype == F32 else -20)
    first, second = (slice(0, n), slice(n, 2 * n)) if layout == "half" else \
        (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    size = x.double().abs()[..., first] + x.double().abs()[..., second]
    u = torch.finfo(x.dtype).eps / 2
    tiny = 2.0 ** -25 if x.dtype == HF else 0.0
    for half in (first, second):
        bound = off * size * (1 + u) + u * ref[..., half].abs() + tiny
        assert ((got.double() - ref)[..., half].abs() <= bound).all(), \
            ((got.double() - ref)[..., half].abs() / bound).max().item()
    assert torch.equal(got[..., 2 * n:], x[..., 2 * n:])


@pytest.mark.parametrize("layout", ["half", "adjacent"])
@pytest.mark.parametrize("dtype", [F32, BF, HF], ids=str)
@pytest.mark.parametrize("dim", [32, 38])
def test_rates_of_any_size_and_sign(pkg, dtype, layout, dim):  # noqa: F811
    gen = torch.Generator(device="cuda").manual_seed(1)
    pairs = (8, 8)
    f = torch.tensor(RATES * 2, dtype=torch.float64, device="cuda")
    at = torch.rand(90, 2, generator=gen, device="cuda") * 2 - 1
    at[:6, 0] = torch.tensor([0.5, 0.375, -0.5, -0.375, 2.0 ** -40, -1.0])
    at[50:] *= 1000
    q, k = normal(gen, 2, 90, 3, dim, dtype=dtype), normal(gen, 2, 90, 1, dim, dtype=dtype)
    for inverse in (False, True):
        got = pkg.rotary(q, k, at, f, pairs, layout=layout, inverse=inverse)
        for t, x in zip(got, (q, k)):
            within(t, x, at, f, pairs, layout, -1.0 if inverse else 1.0)


def test_a_whole_number_is_one_in_either_type(pkg):  # noqa: F811
    """float32 positions that hold integers turn as the integers do, bit for bit."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    f = torch.tensor(RATES, dtype=torch.float64, device="cuda")
    at = torch.randint(-2 ** 24, 2 ** 24, (60, 1), generator=gen, device="cuda")
    q = normal(gen, 60, 2, 16)
    assert torch.equal(pkg.rotary(q, None, at, f, (8,))[0], pkg.rotary(q, None, at.float(), f, (8,))[0])


def test_gradient(pkg):  # noqa: F811
    gen = torch.Generator(device="cuda").manual_seed(3)
    f = torch.tensor(RATES, dtype=torch.float64, device="cuda")
    at = torch.rand(40, 1, generator=gen, device="cuda") * 2 - 1
    q = normal(gen, 40, 2, 16).requires_grad_()
    g = normal(gen, 40, 2, 16)
    got, = torch.autograd.grad(pkg.fused_rotary(q, None, at, f, (8,))[0], q, g)
    within(got, g, at, f, (8,), "half", -1.0)
