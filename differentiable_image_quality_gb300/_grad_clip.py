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


def _tensors(name: str, tensors) -> list:
    """The tensors as a list, checked: CUDA, one device, a known type, dense."""
    ts = [tensors] if isinstance(tensors, torch.Tensor) else list(tensors)
    if not all(isinstance(t, torch.Tensor) for t in ts):
        raise TypeError(f"{name} must be tensors")
    if not all([t.is_cuda for t in ts]):
        raise TypeError(f"{name} must be CUDA tensors")
    if len(set(map(torch.Tensor.get_device, ts))) > 1:
        raise ValueError(f"{name} must be on one device")
    for t in ts:
        if t.layout != torch.strided or not (t.is_contiguous() or t.numel() == 0 or _dense(t)):
            raise ValueError(f"{name} must be dense in memory, got shape {tuple(t.shape)} "
                             f"with layout {t.layout}")
    return ts


def _codes(name: str, ts: list) -> bytes:
    try:
        return bytes([_abi.DTYPES[t.dtype] for t in ts])
    except KeyError as e:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {e.args[0]}") from None


def _addresses(ts: list) -> array:
    return array("Q", [t.data_ptr() for t in ts])


def _at(a: array) -> int:
    return a.buffer_info()[0]


def grad_norm(grads, norm_type=2.0) -> torch.Tensor:
    """The norm of all elements of all tensors together, a 0-dim float32 CUDA tensor.

    grads: a CUDA tensor or an iterable of at least one (float32, bfloat16 and
    float16 may be mixed; any shapes, dense in memory).  norm_type: 2, 1 or inf.
    Nothing is copied to the host."""
    p = _norm_type(norm_type)
    ts = _tensors("grads", grads)
    if not ts:
        raise ValueError("grads is empty: a norm needs a device to be computed on")
    codes, addresses = _codes("grads", ts), _addresses(ts)
    counts = array("q", [t.numel() for t in ts])
    lib = _abi.load()
    device = ts[0].device
    with _memory.on_device(device.index):
        out = torch.empty((), dtype=torch.float32, device=device)
        stream = _memory.stream_of(device.index)
        nbytes = lib.gbssim_grad_workspace_bytes(len(ts))
        ws = _memory.zeroed_scratch(device, stream, nbytes)
        st = lib.gbssim_grad_norm(_at(addresses), _at(counts), codes, len(ts), p, out.data_ptr(),
                                  ws.data_ptr(), ws.numel(), stream)
    _abi.check("gbssim_grad_norm", st)
    return out


@torch.no_grad()
def clip_grads(grads, max_norm: float, norm_type=2.0, out=None) -> torch.Tensor:
    """Scales all gradients by min(1, max_norm / (norm + 1e-6)) and returns their
    norm before that, a 0-dim float32 CUDA tensor.

    In place, or into the tensors of ``out``: as many, of the same shapes and
    memory orders, of any of the three types (float32 main gradients of 16-bit
    gradients, say); the gradients then stay as they are.  grads and norm_type
    are those of grad_norm.  A norm that is not finite is returned, not raised
    (raising would need a copy to the host): NaN makes every gradient NaN,
    infinity makes the finite ones 0."""
    p = _norm_type(norm_type)
    limit = float(max_norm)
    if not limit >= 0.0:
        raise ValueError(f"max_norm must not be negative, got {max_norm!r}")
    ts = _tensors("grads", grads)
    if not ts:
        raise ValueError("grads is empty: a norm needs a device to be computed on")
    codes, addresses = _codes("grads", ts), _addresses(ts)
    counts = array("q", [t.numel() for t in ts])
    outs, out_codes, out_addresses = ts, codes, addresses
    if out is not None:
        outs = _tensors("out", out)
        if len(outs) != len(ts):
            raise ValueError(f"out must have {len(ts)} tensors, got {len(outs)}")
        for g, o in zip(ts, outs):
            if o.shape != g.shape or (o.stride() != g.stride() and not
                                      (o.is_contiguous() and g.is_contiguous())):
                raise ValueError(f"out must have the gradients' shapes and strides: {tuple(o.shape)}"
                                 f" {o.stride()} for {tuple(g.shape)} {g.stride()}")
        if outs[0].device != ts[0].device:
            raise ValueError("grads and out must be on one device")
        out_codes, out_addresses = _codes("out", outs), _addresses(outs)
    lib = _abi.load()
    device = ts[0].device
    with _memory.on_device(device.index):
        norm = torch.empty((), dtype=torch.float32, device=device)
        stream = _memory.stream_of(device.index)
        nbytes = lib.gbssim_grad_workspace_bytes(len(ts))
        ws = _memory.zeroed_scratch(device, stream, nbytes)
        st = lib.gbssim_grad_clip(_at(addresses), _at(out_addresses), _at(counts), codes,
                                  out_codes, len(ts), p, limit, norm.data_ptr(), ws.data_ptr(),
                                  ws.numel(), stream)
    _abi.check("gbssim_grad_clip", st)
    torch.autograd.graph.increment_version(outs)
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
