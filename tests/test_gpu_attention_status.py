"""The device status after waits of attention that run out when all copies have been asked
for: the copying warp has nothing left to notice it by."""
import ctypes

import pytest

from test_gpu_attention import BF, inputs, pkg  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("which", ["forward", "queries", "keys"])
def test_status_of_each_kernel(pkg, which):  # noqa: F811
    q, k, v = inputs(1, 1, 100, 100, 2, 2, 64, BF)
    flags = ctypes.c_uint(0)
    with pkg._abi.using_test_library() as lib:
        out, lse = pkg.attention_fwd(q, k, v, want_stats=True)
        assert lib.gbssim_device_status(ctypes.byref(flags)) == 0 and flags.value == 0
        lib.gbssim_tune_attention(16)
        try:
            if which == "forward":
                got = pkg.attention_fwd(q, k, v)[:1]
            else:
                needs = (which == "queries", which == "keys", which == "keys")
                got = [t for t in pkg.attention_bwd(out, q, k, v, out, lse, needs=needs) if t is not None]
            torch.cuda.synchronize()
        finally:
            lib.gbssim_tune_attention(0)
        assert all(t.isnan().all() for t in got)
        assert lib.gbssim_device_status(ctypes.byref(flags)) == 0
        assert flags.value == 4  # GBSSIM_DEV_ATTENTION_TIMEOUT
        assert torch.equal(pkg.attention_fwd(q, k, v)[0], out)
        assert lib.gbssim_device_status(ctypes.byref(flags)) == 0 and flags.value == 0
