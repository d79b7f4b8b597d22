"""Host-side checks of the gradient norm and clipping: every refusal comes back
before any CUDA call."""
import contextlib
import ctypes
import math
import threading
import time

import pytest
import torch

EINVAL, ESHAPE, EALIGN, EWORKSPACE = -1, -2, -3, -4
BASE = 1 << 30  # addresses that are never dereferenced: each call fails its checks first
F32, BF16, F16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    from differentiable_image_quality_gb300 import _abi, _build

    _build.build()
    return _abi.load()


def arrays(ptrs, counts, types):
    n = len(ptrs)
    return ((ctypes.c_void_p * n)(*ptrs), (ctypes.c_longlong * n)(*counts),
            (ctypes.c_ubyte * n)(*types))


def norm(lib, ptrs=(BASE,), counts=(100,), types=(F32,), n=None, p=2, out=BASE - 16, ws=1 << 40,
         wsb=1 << 20):
    g, c, t = arrays(ptrs, counts, types)
    return lib.gbssim_grad_norm(g, c, t, len(ptrs) if n is None else n, p, out, ws, wsb, None)


def clip(lib, ptrs=(BASE,), outs=(BASE,), counts=(100,), types=(F32,), out_types=(F32,), p=2,
         limit=1.0, out=BASE - 16, ws=1 << 40, wsb=1 << 20):
    g, c, t = arrays(ptrs, counts, types)
    o, _, ot = arrays(outs, counts, out_types)
    return lib.gbssim_grad_clip(g, o, c, t, ot, len(ptrs), p, limit, out, ws, wsb, None)


def test_workspace_grows_with_the_tensors(lib):
    assert lib.gbssim_grad_workspace_bytes(-1) == 0
    one = lib.gbssim_grad_workspace_bytes(0)
    assert one > 0 and lib.gbssim_grad_workspace_bytes(1024) == one
    assert lib.gbssim_grad_workspace_bytes(1025) > one


def test_norm_refusals(lib):
    assert norm(lib, n=-1) == EINVAL
    assert norm(lib, ptrs=(None,)) == EINVAL
    assert norm(lib, types=(3,)) == EINVAL
    assert norm(lib, counts=(-1,)) == ESHAPE
    assert norm(lib, ptrs=(BASE + 2,)) == EALIGN
    assert norm(lib, ptrs=(BASE + 1,), types=(BF16,)) == EALIGN
    assert norm(lib, p=3) == EINVAL
    assert norm(lib, p=-1) == EINVAL
    assert norm(lib, out=None) == EINVAL
    assert norm(lib, out=BASE + 2) == EALIGN
    assert norm(lib, ws=None) == EWORKSPACE
    assert norm(lib, ws=(1 << 40) + 8) == EWORKSPACE
    assert norm(lib, wsb=lib.gbssim_grad_workspace_bytes(1) - 1) == EWORKSPACE
    # more chunks than a launch counts
    assert norm(lib, counts=(1 << 60,)) == ESHAPE


def test_clip_refusals(lib):
    assert clip(lib, limit=-1.0) == EINVAL
    assert clip(lib, limit=math.nan) == EINVAL
    assert clip(lib, outs=(None,)) == EINVAL
    assert clip(lib, outs=(BASE + (1 << 20) + 2,)) == EALIGN
    assert clip(lib, out_types=(7,)) == EINVAL
    assert clip(lib, outs=(BASE + 4,)) == EINVAL                      # its own gradient, shifted
    assert clip(lib, outs=(BASE,), out_types=(BF16,)) == EINVAL       # in place, another type
    far = BASE + (1 << 20)
    two = dict(ptrs=(BASE, far), counts=(100, 100), types=(F32, F32), out_types=(F32, F32))
    assert clip(lib, outs=(BASE + 4096, BASE + 4096 + 396), **two) == EINVAL  # on one another
    assert clip(lib, outs=(far, BASE), **two) == EINVAL               # on another's gradient
    # one tensor twice, in place
    assert clip(lib, ptrs=(BASE, BASE), outs=(BASE, BASE), counts=(100, 100), types=(F32, F32),
                out_types=(F32, F32)) == EINVAL


def test_python_refusals():
    import differentiable_image_quality_gb300 as pkg

    with pytest.raises(TypeError):
        pkg.grad_norm(torch.zeros(3))
    with pytest.raises(TypeError):
        pkg.grad_norm([1.0])
    with pytest.raises(ValueError):
        pkg.grad_norm([])
    with pytest.raises(ValueError):
        pkg.grad_norm([torch.zeros(3)], norm_type=3)
    with pytest.raises(ValueError):
        pkg.grad_norm([torch.zeros(3)], norm_type="fro")
    with pytest.raises(ValueError):
        pkg.clip_grads([torch.zeros(3)], -1.0)
    with pytest.raises(ValueError):
        pkg.clip_grads([torch.zeros(3)], math.nan)
    with pytest.raises(TypeError):
        pkg.clip_grads([torch.zeros(3)], 1.0)


def test_parameters_without_gradients():
    import differentiable_image_quality_gb300 as pkg

    p = torch.nn.Parameter(torch.zeros(3))
    assert float(pkg.clip_grad_norm_([p], 1.0)) == 0.0
    assert float(pkg.clip_grad_norm_(p, 1.0)) == 0.0


def test_threads_on_one_stream_share_no_workspace(monkeypatch):
    """A call of several launches keeps its workspace to itself until it returns, also
    against another host thread on its stream (a stand-in for the library here)."""
    from differentiable_image_quality_gb300 import _abi, _grad_clip, _memory

    class Library:
        def __init__(self):
            self.inside, self.shared, self.calls, self.lock = [], False, 0, threading.Lock()

        def gbssim_grad_workspace_bytes(self, n):
            return 1024

        def call(self, workspace):
            with self.lock:
                self.shared = self.shared or workspace in self.inside
                self.inside.append(workspace)
                self.calls += 1
            time.sleep(0.05)
            with self.lock:
                self.inside.remove(workspace)
            return 0

        def gbssim_grad_norm(self, *a):
            return self.call(a[6])

        def gbssim_grad_clip(self, *a):
            return self.call(a[9])

    lib = Library()
    monkeypatch.setattr(_abi, "load", lambda: lib)
    monkeypatch.setattr(_grad_clip, "_get_device", lambda t: 0)
    monkeypatch.setattr(_memory, "on_device", lambda index: contextlib.nullcontext())
    monkeypatch.setattr(_memory, "stream_of", lambda index: 11)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    _grad_clip.grad_norm([torch.zeros(3)])  # the stream's workspace is there
    start, errors = threading.Barrier(4), []

    def work(k):
        try:
            start.wait(30)
            if k % 2:
                _grad_clip.grad_norm([torch.zeros(3)])
            else:
                _grad_clip.clip_grads([torch.zeros(3)], 1.0)
        except Exception as e:  # noqa: BLE001 - reported below
            errors.append(repr(e))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors, errors
    assert lib.calls == 5 and not lib.shared
