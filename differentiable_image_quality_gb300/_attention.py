"""Attention between the tokens of a batch: torch tensors to gbssim_attention_fwd
and gbssim_attention_bwd."""
from __future__ import annotations

import struct

import torch

from . import _abi, _memory

_MAX_DIM = 128
_CODES = {t: _abi.DTYPES[t] for t in (torch.bfloat16, torch.float16)}

# gbssim_attention
_DESC = struct.Struct("@8if" + "Pqqq" * 3 + "PPP")
_HEADS = struct.Struct("@Pqqq")  # gbssim_heads
_NO_TENSOR = (0, 0, 0, 0)


def _refuse(name: str, t, index, dtype) -> None:
    """Why t is no tensor of dtype (None: bfloat16 or float16) on device index."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    if dtype is None:
        raise TypeError(f"{name} must be bfloat16 or float16, got {t.dtype}")
    raise TypeError(f"{name} must have the type of q, {dtype}, got {t.dtype}")


def _place(t: torch.Tensor, kept: list) -> tuple:
    """(address, batch, token and head stride) of t where the copy unit can read it in
    place, else of a dense copy, which goes to ``kept``: a head's elements side by side,
    strides and address multiples of 16 bytes, no element twice."""
    shape, stride, at = t.shape, t.stride(), t.data_ptr()
    if len(shape) == 4:
        n, tokens, heads, dim = shape
        batch, token, head, one = stride
    else:
        n, batch = 1, 0
        tokens, heads, dim = shape
        token, head, one = stride
    if at % 16 == 0 and one == 1 and (token | head | batch) % 8 == 0 and \
            token > 0 and head > 0 and (batch > 0 or n == 1):
        return at, batch, token, head
    if n == 0 or tokens == 0:
        return _NO_TENSOR
    # the stride along a single element counts for nothing
    if at % 16 or one != 1 or any(m > 1 and (s < 1 or s % 8) for m, s in
                                  ((n, batch), (tokens, token), (heads, head))):
        t = t.clone(memory_format=torch.contiguous_format)
        kept.append(t)
        return t.data_ptr(), tokens * heads * dim, heads * dim, dim
    return at, batch, token, head


def _counts(name: str, t, index, n) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.int32:
        raise TypeError(f"{name} must be an int32 CUDA tensor")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    if t.dim() != 1 or not t.is_contiguous() or (n is not None and t.shape[0] != n):
        raise ValueError(f"{name} must be contiguous of shape "
                         f"({'sequences + 1' if n is None else n},), got {tuple(t.shape)}")
    return t.data_ptr()


def _describe(q, k, v, causal, scale, kv_lengths, offsets, kv_offsets, kept):
    """(packed description, device index), all checked; copies it points to go to
    ``kept``."""
    code = _CODES.get(q.dtype) if isinstance(q, torch.Tensor) and q.is_cuda else None
    if code is None:
        _refuse("q", q, None, None)
    index, dtype = q.get_device(), q.dtype
    for name, t in (("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.get_device() != index or t.dtype != dtype:
            _refuse(name, t, index, dtype)
    packed = offsets is not None
    q_shape, k_shape = q.shape, k.shape
    if k_shape != v.shape:
        raise ValueError(f"k and v must have one shape, got {tuple(k_shape)} and {tuple(v.shape)}")
    if len(q_shape) != (3 if packed else 4) or len(k_shape) != len(q_shape):
        raise ValueError(f"q, k and v must be [{'' if packed else 'batch, '}tokens, heads, dim], "
                         f"got {tuple(q_shape)} and {tuple(k_shape)}")
    tokens, heads, dim = q_shape[-3:]
    keys, kv_heads, k_dim = k_shape[-3:]
    if k_dim != dim or (not packed and k_shape[0] != q_shape[0]):
        raise ValueError(f"q, k and v must agree in batch and dim, got {tuple(q_shape)} and "
                         f"{tuple(k_shape)}")
    if dim % 8 or not 8 <= dim <= _MAX_DIM:
        raise ValueError(f"dim must be a multiple of 8 up to {_MAX_DIM}, got {dim}")
    if kv_heads < 1 or heads < 1 or heads % kv_heads:
        raise ValueError(f"the heads of q must be a multiple of k's, got {heads} and {kv_heads}")
    scale = dim ** -0.5 if scale is None else float(scale)
    if not 0.0 < scale < float("inf"):
        raise ValueError(f"scale must be positive and finite, got {scale}")
    lengths = q_off = k_off = 0
    if packed:
        if kv_lengths is not None:
            raise ValueError("a packed batch has offsets, no kv_lengths")
        q_off = _counts("offsets", offsets, index, None)
        if offsets.shape[0] < 1:
            raise ValueError("offsets must have at least one element")
        if kv_offsets is None:
            if keys != tokens:
                raise ValueError("without kv_offsets, k has the rows of q")
            kv_offsets = offsets
        k_off = _counts("kv_offsets", kv_offsets, index, offsets.shape[0])
        sequences = offsets.shape[0] - 1
    else:
        if kv_offsets is not None:
            raise ValueError("kv_offsets need offsets")
        sequences = q_shape[0]
        if kv_lengths is not None:
            lengths = _counts("kv_lengths", kv_lengths, index, sequences)
    return _DESC.pack(sequences, tokens, keys, heads, kv_heads, dim, code, bool(causal), scale,
                      *_place(q, kept), *_place(k, kept), *_place(v, kept), lengths, q_off,
                      k_off), index


def _stats_shape(q) -> tuple:
    return (*q.shape[:-3], q.shape[-2], q.shape[-3])


def attention_fwd(q, k, v, *, causal=False, scale=None, kv_lengths=None, offsets=None,
                  kv_offsets=None, want_stats=False):
    """The forward without autograd (fused_attention has the arguments).

    Returns (out, lse): out dense, of q's shape and type; lse, with want_stats, the
    logarithm of each row's sum of exponentials, float32 [batch, heads, tokens]
    ([heads, rows] of a packed batch), which attention_bwd needs; else None."""
    kept = []
    desc, index = _describe(q, k, v, causal, scale, kv_lengths, offsets, kv_offsets, kept)
    lib = _abi.load()
    with _memory.on_device(index):
        out = _memory.empty_like(q)
        lse = torch.empty(_stats_shape(q), dtype=torch.float32, device=q.device) \
            if want_stats else None
        nbytes = lib.gbssim_attention_workspace_bytes(desc, 0)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=q.device) if nbytes else None
        st = lib.gbssim_attention_fwd(desc, out.data_ptr(), _abi.ptr(lse), _abi.ptr(ws), nbytes,
                                      _memory.stream_of(index))
    if st:
        _abi.check("gbssim_attention_fwd", st)
    return out, lse


def _like(name, t, index, q):
    if not isinstance(t, torch.Tensor) or t.get_device() != index or t.dtype != q.dtype:
        _refuse(name, t, index, q.dtype)
    if t.shape != q.shape:
        raise ValueError(f"{name} must have shape {tuple(q.shape)}, got {tuple(t.shape)}")


def attention_bwd(g_out, q, k, v, out, lse, *, causal=False, scale=None, kv_lengths=None,
                  offsets=None, kv_offsets=None, needs=(True, True, True)):
    """The backward without autograd: from the gradient of out, the forward's arguments
    and what it returned (out and lse), the gradients of (q, k, v), dense, of their
    types and shapes; None where ``needs`` is false."""
    kept = []
    desc, index = _describe(q, k, v, causal, scale, kv_lengths, offsets, kv_offsets, kept)
    _like("g_out", g_out, index, q)
    _like("out", out, index, q)
    if not isinstance(lse, torch.Tensor) or lse.get_device() != index or \
            lse.dtype != torch.float32 or lse.shape != _stats_shape(q) or \
            not lse.is_contiguous():
        raise ValueError(f"lse must be the forward's: contiguous float32 {_stats_shape(q)}")
    lib = _abi.load()
    with _memory.on_device(index):
        g, o = _HEADS.pack(*_place(g_out, kept)), _HEADS.pack(*_place(out, kept))
        grads = [_memory.empty_like(t) if n else None for t, n in zip((q, k, v), needs)]
        nbytes = lib.gbssim_attention_workspace_bytes(desc, 1)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
        st = lib.gbssim_attention_bwd(desc, g, o, lse.data_ptr(), *map(_abi.ptr, grads),
                                      ws.data_ptr(), nbytes, _memory.stream_of(index))
    if st:
        _abi.check("gbssim_attention_bwd", st)
    return tuple(grads)


class _FusedAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, how):
        wanted = True in ctx.needs_input_grad
        out, lse = attention_fwd(q, k, v, want_stats=wanted, **how)
        if wanted:
            ctx.how = how
            ctx.save_for_backward(q, k, v, out, lse, how["kv_lengths"], how["offsets"],
                                  how["kv_offsets"])
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g_out):
        q, k, v, out, lse, kv_lengths, offsets, kv_offsets = ctx.saved_tensors
        return (*attention_bwd(g_out, q, k, v, out, lse, causal=ctx.how["causal"],
                               scale=ctx.how["scale"], kv_lengths=kv_lengths, offsets=offsets,
                               kv_offsets=kv_offsets, needs=ctx.needs_input_grad[:3]), None)


def fused_attention(q, k, v, *, causal=False, scale=None, kv_lengths=None, offsets=None,
                    kv_offsets=None):
    """Softmax attention, differentiable in q, k and v: per head

        out_i = sum_j softmax_j(scale * q_i . k_j) v_j

    over the keys j that query i sees; zero where it sees none.

    q is [batch, tokens, heads, dim], k and v [batch, keys, kv_heads, dim], bfloat16 or
    float16, dim a multiple of 8 up to 128; heads is a multiple of kv_heads, whose
    neighbouring query heads share keys and values.  scale, positive, is dim ** -0.5 by
    default.  With ``causal``, query i sees the keys up to i + (keys - tokens): the last
    query sees all.  ``kv_lengths``, int32 [batch] on the GPU, are how many of a sample's
    keys count; what lies behind them is not used and gets a zero gradient.  They do not
    move ``causal``'s diagonal, which ends at the last key of the shape: several new tokens
    against caches of different lengths are a packed batch, where it ends at each one's own.

    Packed batches: with ``offsets``, int32 [sequences + 1] on the GPU, ascending from 0, q
    is [rows, heads, dim] and sequence s its rows offsets[s] to offsets[s + 1] - 1, of any
    length; k and v likewise by ``kv_offsets`` (offsets by default).  Rows behind the last
    sequence get zeros.  The lengths stay on the GPU: nothing waits for them.

    Tensors are read in place at any strides, a head's elements side by side on 16-byte
    boundaries; others (expanded ones, odd addresses) are copied first.  Scores,
    statistics and sums are float32, probabilities are rounded to the tensors' type for
    their products, outputs once; results repeat bit for bit.  One query over many keys
    (a token at a time) splits the keys over the GPU."""
    how = {"causal": bool(causal), "scale": scale, "kv_lengths": kv_lengths, "offsets": offsets,
           "kv_offsets": kv_offsets}
    return _FusedAttention.apply(q, k, v, how)
