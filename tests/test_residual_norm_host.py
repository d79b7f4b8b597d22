"""Host-side checks of the residual norm: the packed structs, and refusals that
come back before any CUDA call."""
import ctypes

import pytest
import torch

EINVAL, ESHAPE, EALIGN, EWORKSPACE = -1, -2, -3, -4
MB = 1 << 20
X, Y, XO, U, ST, GX, GU = (i * 64 * MB for i in range(1, 8))  # never dereferenced
G, W1, B1, W2, B2 = (8 * 64 * MB + i * MB for i in range(5))
OUT = 16 * 64 * MB
WS = 1 << 40


class Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_longlong),
                ("token_stride", ctypes.c_longlong)]


class Param(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int), ("per_sample", ctypes.c_int),
                ("sample_stride", ctypes.c_longlong)]


class Desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("batch", "tokens", "dim", "res_dtype", "blk_dtype",
                                            "post_norm", "pre_norm")] + \
               [(n, ctypes.c_float) for n in ("residual_scale", "weight_offset", "eps")] + \
               [(n, Rows) for n in ("x", "y", "gate_rows")] + \
               [(n, Param) for n in ("gate", "post_weight", "post_bias", "pre_weight", "pre_bias")]


class Grads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("x", "y", "gate", "post_weight", "post_bias",
                                               "pre_weight", "pre_bias")]


@pytest.fixture(scope="module")
def lib():
    from differentiable_image_quality_gb300 import _abi, _build

    _build.build()
    return _abi.load()


def desc(**kw):
    d = Desc(2, 8, 64, 0, 0, 1, 2, 1.0, 0.0, 1e-6)
    d.x, d.y = Rows(X, 512, 64), Rows(Y, 512, 64)
    d.post_weight, d.pre_weight, d.pre_bias = Param(W1), Param(W2), Param(B2, 1)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def fwd(lib, d, x_out=XO, u=U, stats=None):
    return lib.gbssim_residual_norm_fwd(ctypes.byref(d) if d else None, x_out, u, stats, None)


def bwd(lib, d, gx=(GX, 512, 64), gu=(GU, 512, 64), stats=ST, grads=None, ws=WS, wsb=1 << 30):
    g = Grads(**(grads or {"x": OUT, "y": OUT + MB}))
    return lib.gbssim_residual_norm_bwd(
        ctypes.byref(d), ctypes.byref(Rows(*gx)) if gx else None,
        ctypes.byref(Rows(*gu)) if gu else None, stats, ctypes.byref(g), ws, wsb, None)


def test_packed_structs_match():
    from differentiable_image_quality_gb300 import _residual_norm as rn

    assert rn._DESC.size == ctypes.sizeof(Desc)
    assert rn._ROWS.size == ctypes.sizeof(Rows)
    assert rn._GRADS.size == ctypes.sizeof(Grads)


def test_forward_refusals(lib):
    assert fwd(lib, None) == EINVAL
    for bad in (dict(res_dtype=3), dict(blk_dtype=-1), dict(res_dtype=1), dict(res_dtype=1, blk_dtype=2),
                dict(post_norm=3), dict(pre_norm=-1), dict(eps=-1.0), dict(eps=float("nan")),
                dict(x=Rows(None)), dict(x=Rows(X, -1, 64)), dict(y=Rows(Y, 512, -64)),
                dict(y=Rows(None)),  # a post norm without a block output
                dict(gate=Param(G, 5)), dict(gate=Param(G), gate_rows=Rows(G, 512, 64)),
                dict(gate=Param(G, 0, 1, -64))):
        assert fwd(lib, desc(**bad)) == EINVAL, bad
    for bad in (dict(dim=0), dict(dim=16385), dict(batch=-1), dict(tokens=-1),
                dict(batch=1 << 16, tokens=1 << 16)):
        assert fwd(lib, desc(**bad)) == ESHAPE, bad
    for bad in (dict(x=Rows(X + 2, 512, 64)), dict(y=Rows(Y + 1, 512, 64)),
                dict(pre_bias=Param(B2 + 1, 1))):
        assert fwd(lib, desc(**bad)) == EALIGN, bad
    assert fwd(lib, desc(), x_out=None) == EINVAL
    assert fwd(lib, desc(), x_out=XO + 2) == EALIGN
    assert fwd(lib, desc(), stats=ST + 8) == EALIGN
    nothing = dict(y=Rows(None), post_norm=0, post_weight=Param())
    assert fwd(lib, desc(**nothing), x_out=None, u=None) == EINVAL
    assert fwd(lib, desc(**nothing)) == EINVAL  # x_out without y
    # outputs on inputs and on one another
    assert fwd(lib, desc(), u=Y) == EINVAL
    assert fwd(lib, desc(), u=XO + 64) == EINVAL
    assert fwd(lib, desc(), u=W2) == EINVAL
    assert fwd(lib, desc(), x_out=X + 4) == EINVAL
    # in place only where x is dense: here samples and tokens are swapped
    assert fwd(lib, desc(x=Rows(X, 64, 128)), x_out=X) == EINVAL
    assert fwd(lib, desc(), stats=U) == EINVAL


def test_no_rows_is_no_work(lib):
    assert fwd(lib, desc(batch=0)) == 0
    assert fwd(lib, desc(tokens=0, x=Rows(None), y=Rows(None))) == 0
    assert lib.gbssim_residual_norm_workspace_bytes(ctypes.byref(desc(tokens=0))) == 0


def test_backward_refusals(lib):
    need = lib.gbssim_residual_norm_workspace_bytes(ctypes.byref(desc()))
    assert need > 0
    assert lib.gbssim_residual_norm_workspace_bytes(ctypes.byref(desc(dim=0))) == 0
    assert bwd(lib, desc(eps=-1.0)) == EINVAL
    assert bwd(lib, desc(), gx=None, gu=None) == EINVAL
    assert bwd(lib, desc(), stats=None) == EINVAL
    assert bwd(lib, desc(), stats=ST + 4) == EALIGN
    assert bwd(lib, desc(), gx=(GX, -512, 64)) == EINVAL
    assert bwd(lib, desc(), gu=(GU + 2, 512, 64)) == EALIGN
    assert bwd(lib, desc(), wsb=need - 1) == EWORKSPACE
    assert bwd(lib, desc(), ws=None) == EWORKSPACE
    assert bwd(lib, desc(), ws=WS + 8) == EWORKSPACE
    # gradients of what is not there
    assert bwd(lib, desc(), grads={"gate": OUT}) == EINVAL
    assert bwd(lib, desc(), grads={"post_bias": OUT}) == EINVAL
    # outputs on inputs, on one another, on the workspace
    assert bwd(lib, desc(), grads={"x": GX}) == EINVAL
    assert bwd(lib, desc(), grads={"x": OUT, "y": OUT + 64}) == EINVAL
    assert bwd(lib, desc(), grads={"pre_weight": W2 + 4}) == EINVAL
    assert bwd(lib, desc(), grads={"x": WS}) == EINVAL
    assert bwd(lib, desc(), grads={"x": OUT + 2}) == EALIGN
    assert bwd(lib, desc(), grads={"pre_bias": OUT + 1}) == EALIGN


def test_python_refuses_cpu_tensors():
    import differentiable_image_quality_gb300 as pkg

    x = torch.zeros(4, 16)
    with pytest.raises(TypeError):
        pkg.fused_residual_norm(x, x)
    with pytest.raises(TypeError):
        pkg.residual_norm_fwd(x, x)
    with pytest.raises(TypeError):
        pkg.residual_norm_bwd(x, x, x, x, torch.zeros(4, 4))
