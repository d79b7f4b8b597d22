"""Rotary positions with several axes: torch tensors to gbssim_rotary_turn."""
from __future__ import annotations

import operator
import struct

import torch

from . import _abi, _memory

_LAYOUTS = {"half": 0, "adjacent": 1}
_POSITIONS = {torch.int32: 0, torch.int64: 1, torch.float32: 2}
_MAX_AXES, _MAX_DIM = 4, 512

# gbssim_rotary
_DESC = struct.Struct("@14i" + "Pqqq" * 2 + "PqqP")
_NO_TENSOR = (0, 0, 0, 0)
_NO_PAIRS = (0,) * _MAX_AXES


def rotary_frequencies(pairs, base: float = 10000.0, device=None) -> torch.Tensor:
    """The usual frequencies of ``pairs`` (how many pairs each axis turns): base^(-i / n)
    for pair i of an axis with n pairs; float64 [sum(pairs)], on the GPU by default."""
    device = torch.device("cuda") if device is None else device
    return torch.cat([float(base) ** (-torch.arange(n, dtype=torch.float64) / n)
                      for n in pairs]).to(device)


def _check(name: str, t, index, like) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    if t.dtype not in _abi.DTYPES:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    if t.dim() not in (3, 4):
        raise ValueError(f"{name} must have 3 or 4 dimensions, [batch, tokens, heads, dim] or "
                         f"[tokens, heads, dim], got {tuple(t.shape)}")
    if like is not None and (t.dtype != like.dtype or t.shape[:-2] != like.shape[:-2] or
                             t.shape[-1] != like.shape[-1]):
        raise ValueError(f"q and k must agree in type, batch, tokens and dim, got "
                         f"{tuple(like.shape)} of {like.dtype} and {tuple(t.shape)} of {t.dtype}")


def _heads(name: str, t) -> tuple:
    """(address, batch, token and head stride)."""
    if t is None:
        return _NO_TENSOR
    s = t.stride()
    if s[-1] != 1 and t.shape[-1] > 1 and t.numel():
        raise ValueError(f"the last dimension of {name} must have stride 1, got {s}")
    return t.data_ptr(), (s[0] if len(s) == 4 else 0), s[-3], s[-2]


def _describe(q, k, positions, frequencies, pairs, layout, inverse):
    """(packed description, device index), all checked."""
    _check("q", q, None, None)
    index = q.get_device()
    if k is not None:
        _check("k", k, index, q)
    try:
        way = _LAYOUTS[layout]
    except (KeyError, TypeError):
        raise ValueError(f"layout must be 'half' or 'adjacent', got {layout!r}") from None
    shape = q.shape
    tokens, heads, dim = shape[-3:]
    pairs = [operator.index(m) for m in pairs]
    n, axes = sum(pairs), len(pairs)
    if not 1 <= axes <= _MAX_AXES or min(pairs) < 1:
        raise ValueError(f"pairs must be one to {_MAX_AXES} positive numbers, got {pairs}")
    if not 2 <= dim <= _MAX_DIM or 2 * n > dim:
        raise ValueError(f"dim must be at most {_MAX_DIM} and hold {n} pairs, got {dim}")
    kind = _POSITIONS.get(positions.dtype) if isinstance(positions, torch.Tensor) else None
    if kind is None:
        raise TypeError("positions must be an int32, int64 or float32 CUDA tensor")
    if positions.get_device() != index:
        raise ValueError(f"positions must be on cuda:{index}, got {positions.device}")
    at = positions.shape
    if at != (tokens, axes) and at != (*shape[:-2], axes):
        raise ValueError(f"positions must have shape ({tokens}, {axes}) or "
                         f"{(*shape[:-2], axes)}, got {tuple(at)}")
    steps = positions.stride()
    if steps[-1] != 1 and axes > 1 and positions.numel():
        raise ValueError("the last dimension of positions must have stride 1")
    if not isinstance(frequencies, torch.Tensor) or frequencies.dtype != torch.float64:
        raise TypeError("frequencies must be a float64 CUDA tensor")
    if frequencies.get_device() != index:
        raise ValueError(f"frequencies must be on cuda:{index}, got {frequencies.device}")
    if frequencies.shape != (n,) or not frequencies.is_contiguous():
        raise ValueError(f"frequencies must be contiguous of shape ({n},), got "
                         f"{tuple(frequencies.shape)}")
    return _DESC.pack(shape[0] if len(shape) == 4 else 1, tokens, heads,
                      0 if k is None else k.shape[-2], dim, _abi.DTYPES[q.dtype], way,
                      bool(inverse), axes, *pairs, *_NO_PAIRS[axes:], kind, *_heads("q", q),
                      *_heads("k", k), positions.data_ptr(), steps[0] if len(at) == 3 else 0,
                      steps[-2], frequencies.data_ptr()), index


def rotary(q, k, positions, frequencies, pairs, *, layout="half", inverse=False):
    """The rotation without autograd (fused_rotary has the arguments): (q', k'), dense,
    k' None where k is.  ``inverse`` turns back: it undoes the rotation and takes its
    outputs' gradients to its inputs'."""
    desc, index = _describe(q, k, positions, frequencies, pairs, layout, inverse)
    with _memory.on_device(index):
        q_out = _memory.empty_like(q)
        k_out = None if k is None else _memory.empty_like(k)
        st = _abi.load().gbssim_rotary_turn(desc, q_out.data_ptr(), _abi.ptr(k_out),
                                            _memory.stream_of(index))
    if st:
        _abi.check("gbssim_rotary_turn", st)
    return q_out, k_out


def _row_wise(t):
    """A gradient's strides are autograd's choice: as it is, or dense."""
    return t if t is None or t.shape[-1] < 2 or t.stride(-1) == 1 else t.contiguous()


class _FusedRotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, frequencies, how):
        ctx.set_materialize_grads(False)
        ctx.how = how
        ctx.save_for_backward(positions, frequencies)
        return rotary(q, k, positions, frequencies, **how)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_q, g_k):
        positions, frequencies = ctx.saved_tensors
        first, second = (g_q, g_k) if g_q is not None else (g_k, None)
        if first is None:
            return (None,) * 5
        a, b = rotary(_row_wise(first), _row_wise(second), positions, frequencies, **ctx.how,
                      inverse=True)
        return *((a, b) if g_q is not None else (None, a)), None, None, None


def fused_rotary(q, k, positions, frequencies, pairs, *, layout="half"):
    """Rotary positions on several axes, differentiable in q and k: the columns of a head
    form pairs, and pair p of an axis turns by positions[token, axis] * frequencies[p],

        (u, v) -> (u cos - v sin, u sin + v cos).

    ``pairs`` says how many pairs each of one to four axes turns (rows and columns of an
    image's patches; time, height and width of a video's; a volume's three), the axes'
    pairs one behind the other, n in all; ``frequencies`` are float64 [n], as
    rotary_frequencies(pairs) makes them.  With layout "half" pair p is columns p and p +
    n, with "adjacent" 2 p and 2 p + 1; columns from 2 n on stay as they are.

    q is [batch, tokens, heads, dim] or [tokens, heads, dim], float32, bfloat16 or
    float16, dim up to 512, k the same with its own number of heads, or None.  positions
    are int32, int64 or float32, [tokens, axes] for all samples or [batch, tokens, axes].
    Frequencies have any size and sign.  Angles are reduced in 64-bit fixed point: what far
    positions lose is the rounding of f / (2 pi) to float64, times the position.
    Positions and frequencies get no gradient, and are refused where they ask for one.
    Returns (q', k'), dense, rounded once from float32."""
    if torch.is_grad_enabled():
        for name, t in (("positions", positions), ("frequencies", frequencies)):
            if isinstance(t, torch.Tensor) and t.requires_grad:
                raise ValueError(f"{name} get no gradient here: detach them, or turn under no_grad")
    return _FusedRotary.apply(q, k, positions, frequencies,
                              {"pairs": tuple(pairs), "layout": layout})
