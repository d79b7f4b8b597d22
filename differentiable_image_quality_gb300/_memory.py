"""Streams, devices and scratch memory of the training-step operators."""
from __future__ import annotations

import contextlib
import threading

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


class _Buffer:
    """The scratch of a stream, and the lock of the call that uses it."""

    __slots__ = ("lock", "tensor")

    def __init__(self):
        self.lock = threading.RLock()  # a finalizer may make a call within a call
        self.tensor = None


class stream_scratch:
    """``with`` gives the scratch that the calls on a stream share (one of ``buffers``),
    zero-filled before its first use, grown on demand; it is one call's alone until
    the block ends.

    Every call leaves its completion counter zero, and what calls put on a stream
    runs one after another, so one buffer serves them all.  The lock keeps the
    launches of a call together: another host thread's on the same stream would
    otherwise come between them, and leave its own results in the buffer."""

    __slots__ = ("buffers", "device", "stream", "nbytes", "least", "held")

    def __init__(self, buffers: dict, device: torch.device, stream: int, nbytes: int, least: int):
        self.buffers, self.device, self.stream = buffers, device, stream
        self.nbytes, self.least = nbytes, least

    def __enter__(self) -> torch.Tensor:
        key = (self.device.index, self.stream)
        held = self.buffers.get(key)
        if held is None:
            held = self.buffers.setdefault(key, _Buffer())
        held.lock.acquire()
        self.held = held
        try:
            if held.tensor is None or held.tensor.numel() < self.nbytes:
                # allocated on the stream that will use it: the caching allocator orders
                # its zero fill before that stream's later work
                held.tensor = torch.zeros(max(self.nbytes, self.least), dtype=torch.uint8,
                                          device=self.device)
        except BaseException:
            held.lock.release()
            raise
        return held.tensor

    def __exit__(self, *error) -> None:
        self.held.lock.release()


def zeroed_scratch(device: torch.device, stream: int, nbytes: int):
    """The stream's scratch for one call, as a context.  A call that is being captured
    into a graph gets a buffer of its own, whose zero fill is part of the graph: a
    replay then depends on no buffer of later calls."""
    if torch.cuda.is_current_stream_capturing():
        return contextlib.nullcontext(torch.zeros(nbytes, dtype=torch.uint8, device=device))
    return stream_scratch(_scratch, device, stream, nbytes, 1 << 16)
