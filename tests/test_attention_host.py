"""Host-side checks of attention: the packed structs, and refusals that come back
before any CUDA call."""
import ctypes

import pytest
import torch

EINVAL, ESHAPE, EALIGN, EWORKSPACE = -1, -2, -3, -4
MB = 1 << 20
Q, K, V, OUT, G, DQ, DK, DV = (i * 64 * MB for i in range(1, 9))  # never dereferenced
LSE, LENGTHS, OFFSETS = (9 * 64 * MB + i * MB for i in range(3))
WS = 1 << 40
F32, BF16, F16 = 0, 1, 2


class Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p)] + [(n, ctypes.c_longlong) for n in
                                              ("batch_stride", "token_stride", "head_stride")]


class Desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("sequences", "q_tokens", "k_tokens", "heads",
                                            "kv_heads", "dim", "dtype", "causal")] + \
               [("scale", ctypes.c_float)] + [(n, Heads) for n in ("q", "k", "v")] + \
               [(n, ctypes.c_void_p) for n in ("kv_lengths", "q_offsets", "k_offsets")]


@pytest.fixture(scope="module")
def lib():
    from differentiable_image_quality_gb300 import _abi, _build

    _build.build()
    return _abi.load()


def dense(data, tokens, heads, dim=64):
    return Heads(data, tokens * heads * dim, heads * dim, dim)


def desc(**kw):
    d = Desc(2, 100, 200, 4, 2, 64, BF16, 0, 0.125, dense(Q, 100, 4), dense(K, 200, 2),
             dense(V, 200, 2))
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def fwd(lib, d, out=OUT, lse=LSE, ws=WS, wsb=1 << 30):
    return lib.gbssim_attention_fwd(ctypes.byref(d) if d else None, out, lse, ws, wsb, None)


def bwd(lib, d, g=None, out=None, lse=LSE, dq=DQ, dk=DK, dv=DV, ws=WS, wsb=1 << 30):
    g = dense(G, 100, 4) if g is None else g
    out = dense(OUT, 100, 4) if out is None else out
    return lib.gbssim_attention_bwd(ctypes.byref(d), ctypes.byref(g), ctypes.byref(out), lse, dq,
                                    dk, dv, ws, wsb, None)


def test_packed_structs_match():
    from differentiable_image_quality_gb300 import _attention

    assert _attention._DESC.size == ctypes.sizeof(Desc)
    assert _attention._HEADS.size == ctypes.sizeof(Heads)


BAD = [
    (EINVAL, dict(dtype=F32)), (EINVAL, dict(dtype=3)),
    (EINVAL, dict(scale=0.0)), (EINVAL, dict(scale=-1.0)), (EINVAL, dict(scale=float("nan"))),
    (EINVAL, dict(scale=float("inf"))),
    (EINVAL, dict(q_offsets=OFFSETS)), (EINVAL, dict(k_offsets=OFFSETS)),
    (EINVAL, dict(q_offsets=OFFSETS, k_offsets=OFFSETS, kv_lengths=LENGTHS)),
    (EINVAL, dict(q=Heads())), (EINVAL, dict(k=Heads())), (EINVAL, dict(v=Heads())),
    (EINVAL, dict(k=Heads(K, 200 * 128, 128, 0))),   # heads that are expanded
    (EINVAL, dict(v=Heads(V, 200 * 128, -128, 64))),
    (ESHAPE, dict(dim=0)), (ESHAPE, dict(dim=60)), (ESHAPE, dict(dim=136)),
    (ESHAPE, dict(heads=3)), (ESHAPE, dict(kv_heads=0)), (ESHAPE, dict(heads=1)),
    (ESHAPE, dict(sequences=-1)), (ESHAPE, dict(q_tokens=-1)), (ESHAPE, dict(k_tokens=1 << 30)),
    (ESHAPE, dict(heads=1 << 16)), (ESHAPE, dict(q=Heads(Q, 1 << 39, 256, 64))),
    (EALIGN, dict(q=dense(Q + 8, 100, 4))), (EALIGN, dict(k=Heads(K, 200 * 128, 128, 68))),
    (EALIGN, dict(v=Heads(V, 200 * 128, 132, 64))), (EALIGN, dict(kv_lengths=LENGTHS + 2)),
]


@pytest.mark.parametrize("status,bad", BAD, ids=str)
def test_description_refusals(lib, status, bad):
    assert fwd(lib, desc(**bad)) == status
    assert bwd(lib, desc(**bad)) == status
    for backward in (0, 1):
        assert lib.gbssim_attention_workspace_bytes(ctypes.byref(desc(**bad)), backward) == 0


def test_forward_refusals(lib):
    assert fwd(lib, None) == EINVAL
    assert fwd(lib, desc(), out=None) == EINVAL
    assert fwd(lib, desc(), out=OUT + 8) == EALIGN
    assert fwd(lib, desc(), lse=LSE + 2) == EALIGN
    for on in (Q, K + 64, V):
        assert fwd(lib, desc(), out=on) == EINVAL
    assert fwd(lib, desc(), lse=OUT + 16) == EINVAL
    assert fwd(lib, desc(kv_lengths=OUT + 64)) == EINVAL
    # one query over many keys: the keys in parts, which need a workspace
    one = desc(q_tokens=1, k_tokens=1 << 16, q=dense(Q, 1, 4), k=dense(K, 1 << 16, 2),
               v=dense(1 << 41, 1 << 16, 2))
    need = lib.gbssim_attention_workspace_bytes(ctypes.byref(one), 0)
    assert need > 0
    assert fwd(lib, one, wsb=need - 1) == EWORKSPACE
    assert fwd(lib, one, ws=None) == EWORKSPACE
    assert fwd(lib, one, ws=WS + 4) == EWORKSPACE
    assert fwd(lib, one, ws=Q) == EINVAL


def test_backward_refusals(lib):
    need = lib.gbssim_attention_workspace_bytes(ctypes.byref(desc()), 1)
    assert need > 0
    assert bwd(lib, desc(), g=Heads()) == EINVAL
    assert bwd(lib, desc(), out=Heads()) == EINVAL
    assert bwd(lib, desc(), g=dense(G + 2, 100, 4)) == EALIGN
    assert bwd(lib, desc(), g=Heads(G, 0, 256, 64)) == EINVAL
    assert bwd(lib, desc(), lse=None) == EINVAL
    assert bwd(lib, desc(), lse=LSE + 1) == EALIGN
    for name in ("dq", "dk", "dv"):
        assert bwd(lib, desc(), **{name: DQ + 8}) == EALIGN
        for on in (Q, K, V, G, OUT, LSE):
            assert bwd(lib, desc(), **{name: on}) == EINVAL
    assert bwd(lib, desc(), dq=DK + 64) == EINVAL
    assert bwd(lib, desc(), dk=WS + 256) == EINVAL
    assert bwd(lib, desc(), wsb=need - 1) == EWORKSPACE
    assert bwd(lib, desc(), ws=None) == EWORKSPACE
    assert bwd(lib, desc(), ws=WS + 8) == EWORKSPACE


def test_no_rows_is_no_work(lib):
    assert fwd(lib, desc(q_tokens=0, q=Heads())) == 0
    assert fwd(lib, desc(sequences=0, q=Heads(), k=Heads(), v=Heads())) == 0
    assert bwd(lib, desc(sequences=0)) == 0
    assert lib.gbssim_attention_workspace_bytes(ctypes.byref(desc(q_tokens=0)), 0) == 0
    for backward in (0, 1):
        assert lib.gbssim_attention_workspace_bytes(ctypes.byref(desc(sequences=0)), backward) == 0


def test_python_refuses_cpu_tensors():
    import differentiable_image_quality_gb300 as pkg

    x = torch.zeros(1, 4, 2, 16, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        pkg.fused_attention(x, x, x)
    with pytest.raises(TypeError):
        pkg.attention_fwd(x, x, x)
    with pytest.raises(TypeError):
        pkg.attention_bwd(x, x, x, x, x, torch.zeros(1, 2, 4))
    with pytest.raises(TypeError):
        pkg.attention_fwd(None, x, x)


# what find_place brings packed offsets to, restated: nothing outside the rows whatever
# the offsets hold, and no row in two sequences where they ascend
def spans(offsets, rows):
    out = []
    for s in range(len(offsets)):
        first = 0 if s == 0 else min(max(offsets[s], 0), rows)
        end = rows if s == len(offsets) - 1 else min(max(offsets[s + 1], first), rows)
        out.append((first, end))
    return out


@pytest.mark.parametrize("offsets", [[0], [0, 5, 5, 9], [0, 20], [3, -4, 100, 7], [0, 9, 2, 9],
                                     [-(1 << 31), (1 << 31) - 1]])
def test_offsets_stay_in_range(offsets):
    rows = 12
    for first, end in spans(offsets, rows):
        assert 0 <= first <= end <= rows
    if offsets == sorted(offsets) and offsets[0] == 0 and offsets[-1] <= rows:
        covered = [i for first, end in spans(offsets, rows) for i in range(first, end)]
        assert covered == list(range(rows))
