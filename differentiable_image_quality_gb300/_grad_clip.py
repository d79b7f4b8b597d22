"""The global gradient norm and clipping: torch tensors to gbssim_grad_norm and
gbssim_grad_clip."""
from __future__ import annotations

import math
from array import array

import torch

from . import _abi, _memory

_NORM_TYPES = {2: 2, 1: 1, math.inf: 0}


def _norm_type(norm_type) -> int:
    try:
        return _NORM_TYPES[float(norm_type)]
    except (KeyError, TypeError, ValueError):
        raise ValueError(f"norm_type must be 1, 2 or inf, got {norm_type!r}") from None


def _dense(t: torch.Tensor) -> bool:
    """Whether the elements fill one piece of memory, in any order of dimensions."""
    if t.layout != torch.strided:
        return False
    expected = 1
    for stride, size in sorted((s, n) for s, n in zip(t.stride(), t.shape) if n != 1):
        if stride != expected:
            return False
        expected *= size
    return True


def _same_order(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether dense tensors of one shape have their elements in one order: the strides
    of dimensions of one element, or of no element at all, reach nothing."""
    return a.numel() == 0 or all(s == t or n == 1
                                 for s, t, n in zip(a.stride(), b.stride(), a.shape))


_is_contiguous, _numel, _get_device, _data_ptr = (
    torch.Tensor.is_contiguous, torch.Tensor.numel, torch.Tensor.get_device, torch.Tensor.data_ptr)


class _List:
    """Tensors checked (CUDA, one device, a known type, dense) and as the arrays
    the library takes.  Passes over the tensors are C loops: a call's own time
    is mostly this."""

    __slots__ = ("tensors", "device", "addresses", "counts", "codes", "contiguous")

    def __init__(self, name: str, tensors):
        ts = self.tensors = [tensors] if isinstance(tensors, torch.Tensor) else list(tensors)
        if not ts:
            raise ValueError(f"{name} is empty: a norm needs a device to be computed on")
        try:
            devices = set(map(_get_device, ts))
            if -1 in devices:
                raise TypeError(f"{name} must be CUDA tensors")
        except TypeError:
            raise TypeError(f"{name} must be CUDA tensors") from None
        if len(devices) > 1:
            raise ValueError(f"{name} must be on one device")
        self.device = devices.pop()
        try:
            self.codes = bytes(map(_abi.DTYPES.__getitem__, [t.dtype for t in ts]))
        except KeyError as e:
            raise TypeError(f"{name} must be float32, bfloat16 or float16, got {e.args[0]}") \
                from None
        try:
            self.contiguous = all(map(_is_contiguous, ts))
        except RuntimeError:  # a layout without strides
            self.contiguous = False
        if not self.contiguous:
            for t in ts:
                if not (t.layout == torch.strided and (t.numel() == 0 or _dense(t))):
                    raise ValueError(f"{name} must be dense in memory, got shape "
                                     f"{tuple(t.shape)} with layout {t.layout}")
        self.addresses = array("Q", map(_data_ptr, ts))
        self.counts = array("q", map(_numel, ts))


def _at(a: array) -> int:
    return a.buffer_info()[0]


def grad_norm(grads, norm_type=2.0) -> torch.Tensor:
    """The norm of all elements of all tensors together, a 0-dim float32 CUDA tensor.

    grads: a CUDA tensor or an iterable of at least one (float32, bfloat16 and
    float16 may be mixed; any shapes, dense in memory).  norm_type: 2, 1 or inf.
    Nothing is copied to the host."""
    p = _norm_type(norm_type)
    ts = _List("grads", grads)
    n = len(ts.tensors)
    lib = _abi.load()
    with _memory.on_device(ts.device):
        out = torch.empty((), dtype=torch.float32, device=ts.tensors[0].device)
        stream = _memory.stream_of(ts.device)
        with _memory.zeroed_scratch(out.device, stream, lib.gbssim_grad_workspace_bytes(n)) as ws:
            st = lib.gbssim_grad_norm(_at(ts.addresses), _at(ts.counts), ts.codes, n, p,
                                      out.data_ptr(), ws.data_ptr(), ws.numel(), stream)
    _abi.check("gbssim_grad_norm", st)
    return out


def clip_grads(grads, max_norm: float, norm_type=2.0, out=None) -> torch.Tensor:
    """Scales all gradients by min(1, max_norm / (norm + 1e-6)) and returns their
    norm before that, a 0-dim float32 CUDA tensor.

    In place, or into the tensors of ``out``: as many, of the same shapes and
    memory orders, of any of the three types (float32 main gradients of 16-bit
    gradients, say); the gradients then stay as they are.  grads and norm_type
    are those of grad_norm.  A norm that is not finite is returned, not raised
    (raising would need a copy to the host): NaN makes every gradient NaN,
    infinity makes the finite ones 0, unless max_norm is infinite, which scales
    nothing."""
    p = _norm_type(norm_type)
    limit = float(max_norm)
    if not limit >= 0.0:
        raise ValueError(f"max_norm must not be negative, got {max_norm!r}")
    ts = _List("grads", grads)
    n, outs = len(ts.tensors), ts
    if out is not None:
        outs = _List("out", out)
        if len(outs.tensors) != n:
            raise ValueError(f"out must have {n} tensors, got {len(outs.tensors)}")
        if outs.device != ts.device:
            raise ValueError("grads and out must be on one device")
        for g, o in zip(ts.tensors, outs.tensors):
            if o.shape != g.shape or (not (ts.contiguous and outs.contiguous)
                                      and not _same_order(g, o)):
                raise ValueError(f"out must have the gradients' shapes and strides: {tuple(o.shape)}"
                                 f" {o.stride()} for {tuple(g.shape)} {g.stride()}")
    lib = _abi.load()
    with _memory.on_device(ts.device):
        norm = torch.empty((), dtype=torch.float32, device=ts.tensors[0].device)
        stream = _memory.stream_of(ts.device)
        with _memory.zeroed_scratch(norm.device, stream, lib.gbssim_grad_workspace_bytes(n)) as ws:
            st = lib.gbssim_grad_clip(_at(ts.addresses), _at(outs.addresses), _at(ts.counts),
                                      ts.codes, outs.codes, n, p, limit, norm.data_ptr(),
                                      ws.data_ptr(), ws.numel(), stream)
    _abi.check("gbssim_grad_clip", st)
    torch.autograd.graph.increment_version(outs.tensors)
    return norm


def clip_grad_norm_(parameters, max_norm: float, norm_type=2.0) -> torch.Tensor:
    """clip_grads of the parameters' ``.grad`` in place; parameters without one
    are left out.  With no gradient at all the norm is 0 (on the CPU)."""
    ps = [parameters] if isinstance(parameters, torch.Tensor) else list(parameters)
    grads = [p.grad for p in ps if p.grad is not None]
    if not grads:
        _norm_type(norm_type)
        return torch.zeros(())
    return clip_grads(grads, max_norm, norm_type)
