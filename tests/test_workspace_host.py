"""The wrappers' own scratch, against a stand-in for the library: no two calls have one
buffer at the same time, whatever host threads and streams they come from."""
import threading
import time
import types

import pytest
import torch

import differentiable_image_quality_gb300 as pkg
from differentiable_image_quality_gb300 import _abi

SHAPE2, SHAPE3 = (1, 1, 12, 12), (1, 1, 12, 12, 12)


class Library:
    """Every size is 64 bytes; a call takes a moment and notes the workspace it got."""

    def __init__(self):
        self.inside, self.twice, self.calls, self.lock = [], False, 0, threading.Lock()

    def __getattr__(self, name):
        if name.endswith(("bytes", "floats")):
            return lambda *a: 64

        def call(*a):
            workspace = a[-3]  # then its size and the stream
            with self.lock:
                self.twice = self.twice or workspace in self.inside
                self.inside.append(workspace)
                self.calls += 1
            time.sleep(0.05)
            with self.lock:
                self.inside.remove(workspace)
            return 0

        return call


@pytest.fixture
def lib(monkeypatch):
    lib = Library()
    monkeypatch.setattr(_abi, "load", lambda: lib)
    monkeypatch.setattr(_abi, "ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(pkg, "_check_pair", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda device=None: types.SimpleNamespace(cuda_stream=23))
    return lib


def calls():
    flat, volume, mean = torch.zeros(SHAPE2), torch.zeros(SHAPE3), torch.zeros(1)
    return [lambda: pkg.ssim_fwd(flat, flat, "same", mean),
            lambda: pkg.ssim_fwd_bwd(flat, flat, "same", mean, mean, flat.clone()),
            lambda: pkg.ssim_pyramid(flat, flat, "same", 2),
            lambda: pkg.ssim3d_fwd(volume, volume, "same", mean),
            lambda: pkg.ssim3d_bwd(mean, volume, volume, "same", volume.clone()),
            lambda: pkg.ssim3d_fwd_bwd(volume, volume, "same", mean, mean, volume.clone())]


def test_threads_on_one_stream_share_no_workspace(lib):
    todo = calls()
    todo[0]()  # the stream's workspace is there
    start, errors = threading.Barrier(len(todo)), []

    def work(call):
        try:
            start.wait(30)
            call()
        except Exception as e:  # noqa: BLE001 - reported below
            errors.append(repr(e))

    threads = [threading.Thread(target=work, args=(call,)) for call in todo]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors, errors
    assert lib.calls == len(todo) + 1 and not lib.twice


def test_given_workspace_is_used(lib):
    seen = []
    lib.ssim_fwd = lambda *a: seen.append(a[-3:-1]) or 0
    workspace = torch.zeros(128, dtype=torch.uint8)
    image = torch.zeros(SHAPE2)
    pkg.ssim_fwd(image, image, "same", torch.zeros(1), workspace=workspace)
    assert seen == [(workspace.data_ptr(), 128)]
