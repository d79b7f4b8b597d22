"""The norms around a residual block, fused with its gate and residual scale:
torch tensors to gbssim_residual_norm_fwd and gbssim_residual_norm_bwd."""
from __future__ import annotations

import struct

import torch

from . import _abi, _memory

_KINDS = {None: 0, "none": 0, "rms": 1, "layer": 2}
_MAX_DIM = 16384

# gbssim_residual_norm, gbssim_rows, gbssim_residual_norm_grads
_DESC = struct.Struct("@7i3f" + "Pqq" * 3 + "Piiq" * 5)
_ROWS = struct.Struct("@Pqq")
_GRADS = struct.Struct("@7P")
_NO_ROWS = (0, 0, 0)
_NO_PARAM = (0, 0, 0, 0)


def _kind(name: str, kind) -> int:
    try:
        return _KINDS[kind]
    except (KeyError, TypeError):
        raise ValueError(f"{name} must be 'rms', 'layer' or None, got {kind!r}") from None


def _check(name: str, t, index) -> int:
    """The type's code of a CUDA tensor on device `index` (any, where that is None)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    code = _abi.DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    return code


def _extents(x: torch.Tensor) -> tuple:
    """(batch, tokens, dim): [tokens, dim] is one sample, the dimensions between
    the first and the last are tokens."""
    shape = x.shape
    if len(shape) == 3:
        return tuple(shape)
    if len(shape) == 0:
        raise ValueError("x must have at least one dimension")
    if len(shape) < 3:
        return 1, (shape[0] if len(shape) == 2 else 1), shape[-1]
    tokens = 1
    for n in shape[1:-1]:
        tokens *= n
    return shape[0], tokens, shape[-1]


def _rows(name: str, t: torch.Tensor, ext: tuple) -> tuple:
    """(address, batch stride, token stride) of a [..., dim] tensor."""
    batch, tokens, dim = ext
    if t.is_contiguous() or t.numel() == 0:
        return t.data_ptr(), tokens * dim, dim
    shape, stride = t.shape, t.stride()
    if dim > 1 and stride[-1] != 1:
        raise ValueError(f"the last dimension of {name} must have stride 1, got {stride}")
    if len(shape) == 1:
        return t.data_ptr(), dim, dim
    middle = range(1, len(shape) - 1) if len(shape) > 2 else range(0, 1)
    step, span = None, 0  # stride of one token, and of all tokens so far
    for i in reversed(middle):
        if shape[i] == 1:
            continue
        if step is None:
            step, span = stride[i], stride[i] * shape[i]
        elif stride[i] == span:
            span *= shape[i]
        else:
            raise ValueError(f"the tokens of {name} must lie at one stride, got shape "
                             f"{tuple(shape)} with strides {stride}")
    step = dim if step is None else step
    return t.data_ptr(), (stride[0] if len(shape) > 2 and batch > 1 else tokens * step), step


def _param(name: str, p, ndim, ext, index) -> tuple:
    if p is None:
        return _NO_PARAM
    code = _check(name, p, index)
    batch, _, dim = ext
    shape = p.shape
    if len(shape) == 1 and shape[0] == dim:
        if dim > 1 and p.stride(0) != 1:
            raise ValueError(f"{name} must be contiguous")
        return p.data_ptr(), code, 0, 0
    if (ndim >= 3 and len(shape) in (2, ndim) and shape[0] == batch and shape[-1] == dim
            and p.numel() == batch * dim):
        if dim > 1 and p.stride(-1) != 1:
            raise ValueError(f"the last dimension of {name} must have stride 1")
        return p.data_ptr(), code, 1, p.stride(0) if batch > 1 else 0
    raise ValueError(f"{name} must have shape ({dim},) or ({batch}, {dim}) beside x of "
                     f"{ndim} dimensions, got {tuple(shape)}")


def _describe(x, y, gate, post_norm, post_weight, post_bias, pre_norm, pre_weight, pre_bias,
              residual_scale, weight_offset, eps, u_dtype):
    """(packed description, extents, device index, type of u), all checked."""
    res = _check("x", x, None)
    index = x.get_device()
    ext = _extents(x)
    ndim, dim = x.dim(), ext[2]
    if not 1 <= dim <= _MAX_DIM:
        raise ValueError(f"the last dimension must be 1 to {_MAX_DIM}, got {dim}")
    post, pre = _kind("post_norm", post_norm), _kind("pre_norm", pre_norm)
    y_rows, gate_rows, gate_param = _NO_ROWS, _NO_ROWS, _NO_PARAM
    if y is None:
        if gate is not None or post or post_weight is not None or post_bias is not None:
            raise ValueError("without y there is nothing to gate or to normalise before the "
                             "residual sum")
        if residual_scale != 1.0:
            raise ValueError("without y the residual scale must be 1")
        u_type = x.dtype if u_dtype is None else u_dtype
        blk = _abi.DTYPES.get(u_type)
    else:
        blk = _check("y", y, index)
        if y.shape != x.shape:
            raise ValueError(f"x and y must have one shape, got {tuple(x.shape)} and "
                             f"{tuple(y.shape)}")
        u_type = y.dtype
        if u_dtype is not None and u_dtype != u_type:
            raise ValueError("u has the type of y")
        y_rows = _rows("y", y, ext)
        if gate is not None:
            if _gate_is_rows(gate, x, y, ext):
                if _check("gate", gate, index) != blk:
                    raise TypeError(f"a gate per row must have the type of y, got {gate.dtype}")
                gate_rows = _rows("gate", gate, ext)
            else:
                gate_param = _param("gate", gate, ndim, ext, index)
    if blk is None or (res != blk and res != 0):
        raise TypeError(f"x must be float32 or have the type of y and u, got {x.dtype} and "
                        f"{u_type}")
    desc = _DESC.pack(*ext, res, blk, post, pre, residual_scale, weight_offset, eps,
                      *_rows("x", x, ext), *y_rows, *gate_rows, *gate_param,
                      *_param("post_weight", post_weight, ndim, ext, index),
                      *_param("post_bias", post_bias, ndim, ext, index),
                      *_param("pre_weight", pre_weight, ndim, ext, index),
                      *_param("pre_bias", pre_bias, ndim, ext, index))
    return desc, ext, index, u_type


def _gate_is_rows(gate, x, y, ext) -> bool:
    """A gate of x's shape is one per row, except beside one token a sample: there it is
    also one per sample, [samples, 1, dim], and has to be where its type is its own."""
    if not isinstance(gate, torch.Tensor) or gate.dim() < 2 or gate.shape != x.shape:
        return False
    return gate.dim() < 3 or ext[1] != 1 or gate.dtype == y.dtype


def residual_norm_fwd(x, y=None, gate=None, *, post_norm=None, post_weight=None, post_bias=None,
                      pre_norm="rms", pre_weight=None, pre_bias=None, residual_scale=1.0,
                      weight_offset=0.0, eps=1e-6, u_dtype=None, x_out=None, want_stats=False):
    """The forward without autograd (fused_residual_norm has the arguments).

    Returns (x_out, u, stats).  x_out may be given: a dense tensor like x, or x
    itself, which then holds the new residual stream (a serving loop's form; no
    backward can follow).  stats, with want_stats, are what residual_norm_bwd
    needs: per row the mean and 1/deviation of the post norm and of the pre norm,
    float32 of shape [..., 4].  x_out is x where y is None, u is None where
    pre_norm is."""
    desc, _, index, u_type = _describe(x, y, gate, post_norm, post_weight, post_bias, pre_norm,
                                       pre_weight, pre_bias, residual_scale, weight_offset, eps,
                                       u_dtype)
    if y is None and x_out is not None:
        raise ValueError("without y there is no x_out")
    wants_u = _KINDS[pre_norm] != 0 or pre_weight is not None or pre_bias is not None
    if not wants_u and y is None:
        raise ValueError("neither y nor a norm: nothing to compute")
    if x_out is not None:
        _check("x_out", x_out, index)
        if x_out.shape != x.shape or x_out.dtype != x.dtype or not x_out.is_contiguous():
            raise ValueError("x_out must be contiguous and have the shape and type of x")
    given = x_out is not None
    with _memory.on_device(index):
        if x_out is None and y is not None:
            x_out = _memory.empty_like(x)
        u = None
        if wants_u:
            u = _memory.empty_like(y) if y is not None else \
                torch.empty(x.shape, dtype=u_type, device=x.device)
        stats = None
        if want_stats:
            stats = torch.empty((*x.shape[:-1], 4), dtype=torch.float32, device=x.device)
        st = _abi.load().gbssim_residual_norm_fwd(
            desc, None if x_out is None else x_out.data_ptr(), None if u is None else u.data_ptr(),
            None if stats is None else stats.data_ptr(), _memory.stream_of(index))
    _abi.check("gbssim_residual_norm_fwd", st)
    if y is None:
        return x, u, stats
    # a view or a buffer counts as written, like x itself (inference tensors count nothing)
    if given and not x_out.is_inference():
        torch.autograd.graph.increment_version(x_out)
    return x_out, u, stats


def _grad_rows(name, g, like, dtype, ext, index):
    if g is None:
        return None, None
    _check(name, g, index)
    if g.shape != like.shape or g.dtype != dtype:
        raise ValueError(f"{name} must have shape {tuple(like.shape)} and type {dtype}, got "
                         f"{tuple(g.shape)} and {g.dtype}")
    try:
        return _ROWS.pack(*_rows(name, g, ext)), g
    except ValueError:  # a gradient's strides are autograd's choice: take a dense copy
        g = g.contiguous()
        return _ROWS.pack(*_rows(name, g, ext)), g


def residual_norm_bwd(g_x, g_u, x, y, stats, gate=None, *, post_norm=None, post_weight=None,
                      post_bias=None, pre_norm="rms", pre_weight=None, pre_bias=None,
                      residual_scale=1.0, weight_offset=0.0, eps=1e-6, u_dtype=None, needs=None):
    """The backward without autograd: from the gradients of x_out and u (either may
    be None: zero), the forward's arguments and its stats, the gradients of
    (x, y, gate, post_weight, post_bias, pre_weight, pre_bias), dense, of their
    tensors' types and shapes; None for what was not given, or where ``needs``
    (seven truth values) is false."""
    desc, ext, index, u_type = _describe(x, y, gate, post_norm, post_weight, post_bias, pre_norm,
                                         pre_weight, pre_bias, residual_scale, weight_offset, eps,
                                         u_dtype)
    if g_x is None and g_u is None:
        raise ValueError("one of g_x and g_u must be given")
    if not isinstance(stats, torch.Tensor) or stats.get_device() != index or \
            stats.dtype != torch.float32 or not stats.is_contiguous() or \
            stats.numel() != ext[0] * ext[1] * 4:
        raise ValueError(f"stats must be the forward's: contiguous float32, {ext[0] * ext[1]} x 4")
    lib = _abi.load()
    empty_like = _memory.empty_like
    with _memory.on_device(index):
        gx, keep_x = _grad_rows("g_x", g_x, x, x.dtype, ext, index)
        gu, keep_u = _grad_rows("g_u", g_u, x, u_type, ext, index)
        inputs = (x, y, gate, post_weight, post_bias, pre_weight, pre_bias)
        if needs is None:
            grads = [None if t is None else empty_like(t) for t in inputs]
        else:
            grads = [empty_like(t) if n and t is not None else None
                     for t, n in zip(inputs, needs)]
        nbytes = lib.gbssim_residual_norm_workspace_bytes(desc)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
        st = lib.gbssim_residual_norm_bwd(
            desc, gx, gu, stats.data_ptr(),
            _GRADS.pack(*[0 if g is None else g.data_ptr() for g in grads]), ws.data_ptr(), nbytes,
            _memory.stream_of(index))
    _abi.check("gbssim_residual_norm_bwd", st)
    return tuple(grads)


class _FusedResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, y, gate, post_weight, post_bias, pre_weight, pre_bias, how):
        x_out, u, stats = residual_norm_fwd(
            x, y, gate, post_weight=post_weight, post_bias=post_bias, pre_weight=pre_weight,
            pre_bias=pre_bias, want_stats=True in ctx.needs_input_grad, **how)
        ctx.set_materialize_grads(False)
        ctx.how = how
        ctx.save_for_backward(x, y, stats, gate, post_weight, post_bias, pre_weight, pre_bias)
        # without y the residual stream passes by: its gradient needs no kernel
        return (None if y is None else x_out), u

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_x, g_u):
        if g_x is None and g_u is None:
            return (None,) * 8
        x, y, stats, gate, post_weight, post_bias, pre_weight, pre_bias = ctx.saved_tensors
        return (*residual_norm_bwd(
            g_x, g_u, x, y, stats, gate, post_weight=post_weight, post_bias=post_bias,
            pre_weight=pre_weight, pre_bias=pre_bias, needs=ctx.needs_input_grad, **ctx.how), None)


def fused_residual_norm(x, y=None, gate=None, *, post_norm=None, post_weight=None, post_bias=None,
                        pre_norm="rms", pre_weight=None, pre_bias=None, residual_scale=1.0,
                        weight_offset=0.0, eps=1e-6, u_dtype=None):
    """The norm after a residual block, its gate, the scaled residual sum and the
    norm before the next block, in one pass, differentiable in every tensor:

        z     = post(y)                      (y itself with post_norm=None)
        x_out = residual_scale * x + gate * z
        u     = pre(x_out)                   (None with pre_norm=None)

    Returns (x_out, u).  A norm is "rms", v / sqrt(mean(v^2) + eps), or "layer",
    which subtracts the mean first; then (weight + weight_offset), one offset for both
    norms, and bias apply, each optional.  x, the residual stream, and y, the block's output, are CUDA
    tensors of one shape [..., dim], dim up to 16384; with three or more
    dimensions the first counts samples.  Weights, biases and the gate are [dim],
    or [samples, dim] (conditioned norms and gates; [samples, 1, dim] as well);
    the gate may also have the shape of x, one factor for every element of y and of
    y's type.  y and u are float32, bfloat16 or float16, x the same or float32;
    parameters have any of the three.  Rows may lie at any stride, the columns of a
    row next to one another.

    Without y only the norm is taken: u = pre(x), of type u_dtype (default x's),
    and x_out is x -- the norm before the first block.  Arithmetic is float32,
    each output rounded once, u formed from x_out before its rounding; results
    repeat bit for bit."""
    how = {"post_norm": post_norm, "pre_norm": pre_norm, "residual_scale": float(residual_scale),
           "weight_offset": float(weight_offset), "eps": float(eps), "u_dtype": u_dtype}
    x_out, u = _FusedResidualNorm.apply(x, y, gate, post_weight, post_bias, pre_weight, pre_bias,
                                        how)
    return (x if y is None else x_out), u
