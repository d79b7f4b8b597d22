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


class _Scratch:
    """The buffer of a stream, and the lock of the call that uses it."""

    __slots__ = ("lock", "buffer")

    def __init__(self):
        self.lock = threading.RLock()  # a finalizer may make a call within a call
        self.buffer = None


class zeroed_scratch:
    """Scratch for one call of the library on a stream: ``with`` gives a buffer that is
    zero-filled before its first use, and is the call's alone until the block ends.

    Every call leaves its completion counter zero, and what calls put on a stream
    runs one after another, so a stream's calls share one buffer.  The lock keeps
    the launches of a call together: another host thread's on the same stream
    would otherwise come between them, and leave its own results in the buffer.  A
    call that is being captured into a graph gets a buffer of its own, whose zero
    fill is part of the graph: a replay then depends on no buffer of later calls."""

    __slots__ = ("device", "stream", "nbytes", "scratch")

    def __init__(self, device: torch.device, stream: int, nbytes: int):
        self.device, self.stream, self.nbytes, self.scratch = device, stream, nbytes, None

    def __enter__(self) -> torch.Tensor:
        if torch.cuda.is_current_stream_capturing():
            return torch.zeros(self.nbytes, dtype=torch.uint8, device=self.device)
        key = (self.device.index, self.stream)
        scratch = _scratch.get(key)
        if scratch is None:
            scratch = _scratch.setdefault(key, _Scratch())
        scratch.lock.acquire()
        self.scratch = scratch
        try:
            buffer = scratch.buffer
            if buffer is None or buffer.numel() < self.nbytes:
                buffer = scratch.buffer = torch.zeros(max(self.nbytes, 1 << 16), dtype=torch.uint8,
                                                      device=self.device)
        except BaseException:
            scratch.lock.release()
            raise
        return buffer

    def __exit__(self, *error) -> None:
        if self.scratch is not None:
            self.scratch.lock.release()
