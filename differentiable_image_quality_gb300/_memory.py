"""Streams, devices and scratch memory of the training-step operators."""
from __future__ import annotations

import contextlib

import torch

_scratch: dict = {}
_here = contextlib.nullcontext()


def on_device(index: int):
    """The library launches on the current device: a context that makes the
    tensors' device current, and nothing where it already is."""
    return _here if torch.cuda.current_device() == index else torch.cuda.device(index)


def stream_of(index: int) -> int:
    # the raw handle: a Stream object costs more than the rest of a small call
    return torch._C._cuda_getCurrentRawStream(index)


def empty_like(t: torch.Tensor) -> torch.Tensor:
    """A dense tensor of t's shape, type and device."""
    return torch.empty_like(t, requires_grad=False) if t.is_contiguous() else \
        torch.empty(t.shape, dtype=t.dtype, device=t.device)


def zeroed_scratch(device: torch.device, stream: int, nbytes: int) -> torch.Tensor:
    """Scratch for calls on one stream of one device, zero-filled before its
    first use; every call leaves its completion counter zero, and the calls of
    a stream run one after another, so they share one buffer.  A call that is
    being captured into a graph gets a buffer of its own, whose zero fill is
    part of the graph: a replay then depends on no buffer of later calls."""
    if torch.cuda.is_current_stream_capturing():
        return torch.zeros(nbytes, dtype=torch.uint8, device=device)
    buf = _scratch.get((device.index, stream))
    if buf is None or buf.numel() < nbytes:
        buf = torch.zeros(max(nbytes, 1 << 16), dtype=torch.uint8, device=device)
        _scratch[(device.index, stream)] = buf
    return buf
