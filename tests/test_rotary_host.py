"""Host-side checks of rotary positions: the packed struct, refusals that come back
before any CUDA call, and the fixed-point angle."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

EINVAL, ESHAPE, EALIGN = -1, -2, -3
MB = 1 << 20
Q, K, QO, KO, POS, FREQ = (i * 64 * MB for i in range(1, 7))  # never dereferenced


class Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p)] + [(n, ctypes.c_longlong) for n in
                                              ("batch_stride", "token_stride", "head_stride")]


class Desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("batch", "tokens", "q_heads", "k_heads", "dim",
                                            "dtype", "layout", "inverse", "axes")] + \
               [("pairs", ctypes.c_int * 4), ("pos_type", ctypes.c_int), ("q", Heads),
                ("k", Heads), ("positions", ctypes.c_void_p),
                ("pos_batch_stride", ctypes.c_longlong), ("pos_token_stride", ctypes.c_longlong),
                ("frequencies", ctypes.c_void_p)]


@pytest.fixture(scope="module")
def lib():
    from differentiable_image_quality_gb300 import _abi, _build

    _build.build()
    return _abi.load()


def desc(**kw):
    d = Desc(2, 50, 4, 2, 64, 1, 0, 0, 2, (ctypes.c_int * 4)(16, 16), 1,
             Heads(Q, 50 * 256, 256, 64), Heads(K, 50 * 128, 128, 64), POS, 0, 2, FREQ)
    for k, v in kw.items():
        setattr(d, k, (ctypes.c_int * 4)(*v) if k == "pairs" else v)
    return d


def turn(lib, d, q=QO, k=KO):
    return lib.gbssim_rotary_turn(ctypes.byref(d) if d else None, q, k, None)


def test_packed_struct_matches():
    from differentiable_image_quality_gb300 import _rotary

    assert _rotary._DESC.size == ctypes.sizeof(Desc)


@pytest.mark.parametrize("status,bad", [
    (EINVAL, dict(dtype=3)), (EINVAL, dict(pos_type=3)), (EINVAL, dict(layout=2)),
    (EINVAL, dict(q=Heads())), (EINVAL, dict(k=Heads())), (EINVAL, dict(positions=None)),
    (EINVAL, dict(frequencies=None)), (EINVAL, dict(q=Heads(Q, -1, 256, 64))),
    (EINVAL, dict(pos_token_stride=-2)),
    (ESHAPE, dict(dim=1)), (ESHAPE, dict(dim=513)), (ESHAPE, dict(dim=62)),
    (ESHAPE, dict(axes=0)), (ESHAPE, dict(axes=5)), (ESHAPE, dict(pairs=(16, 0))),
    (ESHAPE, dict(batch=-1)), (ESHAPE, dict(tokens=-1)), (ESHAPE, dict(q_heads=1 << 16)),
    (EALIGN, dict(q=Heads(Q + 1, 50 * 256, 256, 64))), (EALIGN, dict(positions=POS + 4)),
    (EALIGN, dict(frequencies=FREQ + 4)),
], ids=str)
def test_refusals(lib, status, bad):
    assert turn(lib, desc(**bad)) == status


def test_output_refusals(lib):
    assert turn(lib, None) == EINVAL
    assert turn(lib, desc(), q=None) == EINVAL
    assert turn(lib, desc(), k=None) == EINVAL
    assert turn(lib, desc(), q=QO + 1) == EALIGN
    for on in (Q, K + 64, POS, FREQ + 8, KO):
        assert turn(lib, desc(), q=on) == EINVAL
    assert turn(lib, desc(batch=0)) == 0
    assert turn(lib, desc(q_heads=0, k_heads=0)) == 0


def test_python_refusals():
    import differentiable_image_quality_gb300 as pkg

    x, f = torch.zeros(4, 2, 16), pkg.rotary_frequencies((4,), device="cpu")
    assert f.dtype == torch.float64 and f.tolist() == [10000.0 ** (-i / 4) for i in range(4)]
    with pytest.raises(TypeError):
        pkg.rotary(x, None, torch.zeros(4, 1), f, (4,))
    with pytest.raises(TypeError):
        pkg.fused_rotary(x, None, torch.zeros(4, 1), f, (4,))


@pytest.mark.parametrize("position", [0, 1, -1, 77, -4096, 10 ** 6 + 3, 2 ** 31 - 1, -2 ** 40])
@pytest.mark.parametrize("f", [1.0, 0.5, 10000.0 ** -0.3, 1e-4, 7.25, -0.75])
def test_fixed_point_angle(position, f):
    """The kernel's angle, restated in integers: f / (2 pi) in float64, its fraction times
    2^64, times the position, modulo 2^64; against exact arithmetic."""
    turns = abs(f) * 0.15915494309189535
    fraction = int((turns - math.floor(turns)) * 2.0 ** 64) * (-1 if f < 0 else 1)
    phase = (position * fraction) % 2 ** 64
    pi = Fraction(3141592653589793238462643383279502884197, 10 ** 39)
    exact = Fraction(position) * Fraction(f) / (2 * pi)
    off = (Fraction(phase, 2 ** 64) - exact) % 1
    off = min(off, 1 - off)
    # the constant and the product round to 53 bits, the fraction is cut once
    assert off <= abs(position) * (Fraction(turns) * Fraction(2) ** -52 + Fraction(2) ** -62)
