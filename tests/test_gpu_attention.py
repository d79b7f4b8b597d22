"""Attention on the GPU against its definition in float64.

Tolerances.  u is half a step of the tensors' type.  A score sums dim products in
float32: it is off by at most e = (dim + 8) 2^-22 scale sum|q k| (a sum that truncates
loses 2^-23 a step), and so is the logarithm of a probability, plus 2^-20 for the
exponential and its argument's rounding (arguments up to 2^4 in steps of 2^-20).  A
probability is rounded once to the type: relative u.  So the output is off by at most
(u + 2 e + 2^-18) sum p|v| + u |o|: errors of the numerator, and the unrounded
denominator's.
"""
import random

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def pkg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import differentiable_image_quality_gb300 as pkg
    from differentiable_image_quality_gb300 import _build

    _build.build()
    return pkg


def normal(gen, *shape, dtype=BF, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def inputs(seed, B, Tq, Tk, H, K, D, dtype):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    shapes = ((Tq, H, D), (Tk, K, D), (Tk, K, D))
    return [normal(gen, *(s if B is None else (B, *s)), dtype=dtype) for s in shapes]


def visible(q, k, causal, width):
    """[queries, keys] of one sequence, `width` keys ending the causal diagonal."""
    seen = torch.ones(q, k, dtype=torch.bool, device="cuda")
    return seen.tril(width - q) if causal else seen


def definition(q, k, v, scale, seen):
    """One sequence [tokens, heads, dim] in float64: out, lse [heads, queries], and the
    largest errors that the output and the lse may have (see above)."""
    group = q.shape[1] // k.shape[1]
    u = torch.finfo(v.dtype).eps / 2
    dim = q.shape[-1]
    q, k, v = q.double(), k.double(), v.double()
    k, v = (t.repeat_interleave(group, 1) for t in (k, v))
    s = torch.einsum("ihd,jhd->hij", q, k) * scale
    e = torch.einsum("ihd,jhd->hij", q.abs(), k.abs()) * scale * (dim + 8) * 2.0 ** -22
    s = s.masked_fill(~seen, -float("inf"))
    lse = torch.logsumexp(s, -1) if k.shape[0] else torch.full(s.shape[:2], -float("inf"),
                                                               device="cuda", dtype=s.dtype)
    p = torch.exp(s - lse.nan_to_num(neginf=0.0)[..., None])
    out = torch.einsum("hij,jhd->ihd", p, v)
    most = e.masked_fill(~seen, 0.0).amax(-1) if k.shape[0] else torch.zeros_like(lse)
    absolute = torch.einsum("hij,jhd->ihd", p, v.abs())
    bound = (u + 2 * most.T[..., None] + 2.0 ** -18) * absolute + u * out.abs() + 1e-30
    return out, lse, bound, most + 2.0 ** -18 + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0.0)


def check_sequence(out, lse, q, k, v, scale, seen):
    ref, ref_lse, bound, lse_bound = definition(q, k, v, scale, seen)
    assert ((out.double() - ref).abs() <= bound).all(), \
        ((out.double() - ref).abs() / bound).max().item()
    none = ref_lse == -float("inf")
    assert torch.equal(lse == -float("inf"), none)
    assert ((lse.double() - ref_lse).abs() <= lse_bound)[~none].all()


# B, Tq, Tk, H, K, D, type, causal
BATCHES = [
    (1, 1, 1, 1, 1, 8, BF, False),
    (1, 128, 128, 1, 1, 64, BF, False),
    (1, 128, 128, 1, 1, 128, BF, False),
    (2, 64, 64, 8, 8, 32, BF, False),
    (2, 130, 257, 3, 3, 72, HF, False),
    (1, 300, 300, 4, 2, 128, BF, True),
    (3, 257, 129, 6, 2, 40, HF, True),      # the first 128 queries see nothing
    (2, 129, 1000, 2, 1, 96, BF, True),
    (1, 1, 5000, 32, 8, 128, BF, True),     # one token over many: the keys in parts
    (2, 7, 1300, 12, 4, 64, HF, True),      # several tokens, heads of a group in one tile
    (1, 3, 700, 6, 1, 104, BF, False),      # a group that is no power of two
    (4, 1, 77, 4, 4, 16, HF, False),
    (1, 1, 65600, 2, 1, 120, BF, False),
    (4, 1024, 1024, 16, 16, 72, HF, False),
    (2, 1500, 1500, 32, 8, 128, BF, True),
    (1, 5, 0, 2, 1, 64, BF, False),
    (1, 255, 3, 2, 2, 56, HF, False),
    (1, 1500, 300, 16, 1, 64, BF, False),   # query heads of a key head in parts
    (2, 700, 260, 21, 3, 96, HF, True),
]


@pytest.mark.parametrize("case", BATCHES, ids=str)
def test_forward_batch(pkg, case):
    B, Tq, Tk, H, K, D, dtype, causal = case
    q, k, v = inputs(1, B, Tq, Tk, H, K, D, dtype)
    out, lse = pkg.attention_fwd(q, k, v, causal=causal, want_stats=True)
    assert out.shape == q.shape and out.dtype == dtype and lse.shape == (B, H, Tq)
    for b in range(B):
        check_sequence(out[b], lse[b], q[b], k[b], v[b], D ** -0.5,
                       visible(Tq, Tk, causal, Tk))


# lengths; H, K, D, type, causal
PACKS = [
    ([5], 1, 1, 64, BF, False),
    ([128, 1, 0, 129, 300], 4, 2, 128, BF, False),
    ([0, 0, 17, 256, 0], 3, 3, 72, HF, True),
    ([1] * 70 + [513], 2, 1, 40, BF, True),
    ([1000, 3, 900, 128, 256, 511], 8, 8, 64, HF, False),
    ([600, 75, 0, 333, 140], 24, 3, 96, HF, True),  # query heads of a key head in parts
]


def pack_offsets(lengths):
    ends = [sum(lengths[:i]) for i in range(len(lengths) + 1)]
    return ends, torch.tensor(ends, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("tail", [0, 9])
@pytest.mark.parametrize("case", PACKS, ids=str)
def test_forward_packed(pkg, case, tail):
    lengths, H, K, D, dtype, causal = case
    ends, offsets = pack_offsets(lengths)
    n = ends[-1] + tail
    q, k, v = inputs(2, None, n, n, H, K, D, dtype)
    out, lse = pkg.attention_fwd(q, k, v, causal=causal, offsets=offsets, want_stats=True)
    for a, b in zip(ends, ends[1:]):
        check_sequence(out[a:b], lse[:, a:b], q[a:b], k[a:b], v[a:b], D ** -0.5,
                       visible(b - a, b - a, causal, b - a))
    assert (out[ends[-1]:] == 0).all() and (lse[:, ends[-1]:] == -float("inf")).all()


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Tq", [1, 150])
def test_forward_key_lengths(pkg, Tq, causal):
    """What lies behind the keys that count is not used, whatever it holds."""
    B, Tk, H, K, D = 5, 1200, 4, 2, 80
    q, k, v = inputs(3, B, Tq, Tk, H, K, D, BF)
    lengths = [1200, 0, 1, 128, 777]
    for b, n in enumerate(lengths):
        k[b, n:] = float("nan")
        v[b, n:] = float("inf")
    kv = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out, lse = pkg.attention_fwd(q, k, v, causal=causal, kv_lengths=kv, want_stats=True)
    for b, n in enumerate(lengths):
        check_sequence(out[b], lse[b], q[b], k[b, :n], v[b, :n], D ** -0.5,
                       visible(Tq, Tk, causal, Tk)[:, :n])


# ------------------------------------------------------------------ backward

def definition_bwd(g, q, k, v, out, scale, seen, lse):
    """Gradients of one sequence in float64, and the largest errors they may have.

    With u and e as above: p is off by relative w = u + 2 e + 2^-18 (its rounding for dv,
    the score's and lse's errors), dp - D by the float32 sums' (dim + 8) 2^-22 of
    absolute sums, and by u sum|g o| since D takes the rounded output; ds is rounded once
    more (u).  float16 scales by powers of two, whose rounding is u too; below them it
    keeps 2^-24 of the scaled range: 2^-39 of the bound 2 dim |g| |v| on dp.  The sums of
    n products lose n 2^-22 at most; each gradient is rounded once (u)."""
    group = q.shape[1] // k.shape[1]
    half = v.dtype == HF
    u = torch.finfo(v.dtype).eps / 2
    dim, n, m = q.shape[-1], q.shape[0], k.shape[0]
    q, k, v, g, out = (t.double() for t in (q, k, v, g, out))
    wide_k, wide_v = (t.repeat_interleave(group, 1) for t in (k, v))

    def heads(t):  # sums of the heads that share
        return t.unflatten(1, (k.shape[1], group)).sum(2)

    step = (dim + 8) * 2.0 ** -22
    s = torch.einsum("ihd,jhd->hij", q, wide_k) * scale
    e = torch.einsum("ihd,jhd->hij", q.abs(), wide_k.abs()) * scale * step
    p = torch.exp(s - lse.nan_to_num(neginf=0.0)[..., None]).masked_fill(~seen, 0.0)
    e = e.masked_fill(~seen, 0.0)
    most = e.amax(-1, keepdim=True) if m else e.sum(-1, keepdim=True)
    w = u + e + most + 2.0 ** -18
    dp = torch.einsum("ihd,jhd->hij", g, wide_v)
    dp_abs = torch.einsum("ihd,jhd->hij", g.abs(), wide_v.abs())
    exact_o = torch.einsum("hij,jhd->ihd", p, wide_v)
    D = (g * exact_o).sum(-1).T[..., None]
    D_err = (g * (out - exact_o)).sum(-1).abs().T[..., None] + \
        (g * out).abs().sum(-1).T[..., None] * step
    ds = p * (dp - D)
    floor = (2 * dim * g.abs().max() * v.abs().max()) * 2.0 ** -38 if half and g.numel() and m else 0.0
    ds_err = ds.abs() * (w + u) + p * (dp_abs * step + D_err) * (1 + w) + seen * floor
    p_err = p * w + (seen * 2.0 ** -38 if half else 0.0)
    ax = lambda *t: torch.einsum(*t)  # noqa: E731
    dq = ax("hij,jhd->ihd", ds, wide_k) * scale
    dk = heads(ax("hij,ihd->jhd", ds, q)) * scale
    dv = heads(ax("hij,ihd->jhd", p, g))
    dq_err = (ax("hij,jhd->ihd", ds_err, wide_k.abs()) +
              ax("hij,jhd->ihd", ds.abs(), wide_k.abs()) * (m + 8) * 2.0 ** -22) * scale
    dk_err = heads(ax("hij,ihd->jhd", ds_err, q.abs()) +
                   ax("hij,ihd->jhd", ds.abs(), q.abs()) * (n * group + 8) * 2.0 ** -22) * scale
    dv_err = heads(ax("hij,ihd->jhd", p_err, g.abs()) +
                   ax("hij,ihd->jhd", p, g.abs()) * (n * group + 8) * 2.0 ** -22)
    # the least float16 is 2^-24
    tiny = 2.0 ** -25 if half else 1e-30
    return [(t, err * (1 + u) + u * t.abs() + tiny) for t, err in ((dq, dq_err), (dk, dk_err),
                                                                  (dv, dv_err))]


def check_gradients(got, g, q, k, v, out, scale, seen):
    _, lse, _, _ = definition(q, k, v, scale, seen)
    for name, t, (ref, bound) in zip("qkv", got, definition_bwd(g, q, k, v, out, scale, seen, lse)):
        ratio = ((t.double() - ref).abs() / bound)
        assert (ratio <= 1).all(), (name, ratio.max().item())


@pytest.mark.parametrize("case", [c for c in BATCHES if c[2] <= 2000], ids=str)
def test_backward_batch(pkg, case):
    B, Tq, Tk, H, K, D, dtype, causal = case
    q, k, v = inputs(4, B, Tq, Tk, H, K, D, dtype)
    g = normal(torch.Generator(device="cuda").manual_seed(5), *q.shape, dtype=dtype, std=0.1)
    out, lse = pkg.attention_fwd(q, k, v, causal=causal, want_stats=True)
    got = pkg.attention_bwd(g, q, k, v, out, lse, causal=causal)
    for t, like in zip(got, (q, k, v)):
        assert t.shape == like.shape and t.dtype == dtype and t.is_contiguous()
    for b in range(B):
        check_gradients([t[b] for t in got], g[b], q[b], k[b], v[b], out[b], D ** -0.5,
                        visible(Tq, Tk, causal, Tk))


@pytest.mark.parametrize("tail", [0, 9])
@pytest.mark.parametrize("case", PACKS, ids=str)
def test_backward_packed(pkg, case, tail):
    lengths, H, K, D, dtype, causal = case
    ends, offsets = pack_offsets(lengths)
    n = ends[-1] + tail
    q, k, v = inputs(6, None, n, n, H, K, D, dtype)
    g = normal(torch.Generator(device="cuda").manual_seed(7), *q.shape, dtype=dtype, std=0.1)
    if tail:  # what lies behind the last sequence reaches nothing
        for t in (q, k, v, g):
            t[ends[-1]:] = float("nan")
    out, lse = pkg.attention_fwd(q, k, v, causal=causal, offsets=offsets, want_stats=True)
    got = pkg.attention_bwd(g, q, k, v, out, lse, causal=causal, offsets=offsets)
    for a, b in zip(ends, ends[1:]):
        check_gradients([t[a:b] for t in got], g[a:b], q[a:b], k[a:b], v[a:b], out[a:b],
                        D ** -0.5, visible(b - a, b - a, causal, b - a))
    for t in got:
        assert (t[ends[-1]:] == 0).all()


def test_packed_sequences_do_not_meet(pkg):
    """A sequence full of NaN beside others changes nothing in them."""
    lengths, H, D = [40, 77, 130, 5], 3, 64
    ends, offsets = pack_offsets(lengths)
    q, k, v = inputs(8, None, ends[-1], ends[-1], H, H, D, BF)
    g = normal(torch.Generator(device="cuda").manual_seed(9), *q.shape)

    def run():
        out, lse = pkg.attention_fwd(q, k, v, offsets=offsets, want_stats=True)
        return (out, *pkg.attention_bwd(g, q, k, v, out, lse, offsets=offsets))

    before = run()
    for t in (q, k, v, g):
        t[ends[1]:ends[2]] = float("nan")
    after = run()
    for x, y in zip(before, after):
        assert torch.equal(x[:ends[1]], y[:ends[1]]) and torch.equal(x[ends[2]:], y[ends[2]:])
        assert y[ends[1]:ends[2]].isnan().all()


@pytest.mark.parametrize("causal", [False, True])
def test_backward_key_lengths(pkg, causal):
    B, Tq, Tk, H, K, D = 5, 150, 400, 4, 2, 80
    q, k, v = inputs(10, B, Tq, Tk, H, K, D, BF)
    g = normal(torch.Generator(device="cuda").manual_seed(11), *q.shape)
    lengths = [400, 0, 1, 128, 277]
    for b, n in enumerate(lengths):
        k[b, n:] = float("inf")
        v[b, n:] = float("nan")
    kv = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out, lse = pkg.attention_fwd(q, k, v, causal=causal, kv_lengths=kv, want_stats=True)
    got = pkg.attention_bwd(g, q, k, v, out, lse, causal=causal, kv_lengths=kv)
    for b, n in enumerate(lengths):
        check_gradients([got[0][b], got[1][b, :n], got[2][b, :n]], g[b], q[b], k[b, :n], v[b, :n],
                        out[b], D ** -0.5, visible(Tq, Tk, causal, Tk)[:, :n])
        assert (got[1][b, n:] == 0).all() and (got[2][b, n:] == 0).all()


def test_cross_packed(pkg):
    """Queries and keys packed by offsets of their own, sequences without the one or the
    other among them."""
    ql, kl, H, K, D = [100, 0, 33, 200], [70, 50, 0, 300], 4, 2, 128
    qe, qo = pack_offsets(ql)
    ke, ko = pack_offsets(kl)
    gen = torch.Generator(device="cuda").manual_seed(12)
    q, g = normal(gen, qe[-1], H, D), normal(gen, qe[-1], H, D)
    k, v = normal(gen, ke[-1] + 3, K, D), normal(gen, ke[-1] + 3, K, D)
    out, lse = pkg.attention_fwd(q, k, v, offsets=qo, kv_offsets=ko, want_stats=True)
    got = pkg.attention_bwd(g, q, k, v, out, lse, offsets=qo, kv_offsets=ko)
    for a, b, c, d in zip(qe, qe[1:], ke, ke[1:]):
        seen = visible(b - a, d - c, False, 0)
        check_sequence(out[a:b], lse[:, a:b], q[a:b], k[c:d], v[c:d], D ** -0.5, seen)
        check_gradients([got[0][a:b], got[1][c:d], got[2][c:d]], g[a:b], q[a:b], k[c:d], v[c:d],
                        out[a:b], D ** -0.5, seen)
    assert (got[1][ke[-1]:] == 0).all()


@pytest.mark.parametrize("causal, dtype", [(False, BF), (True, BF), (False, HF)])
def test_many_short_sequences(pkg, causal, dtype):
    """More sequences than a block's searches pass at once, so that its items come from
    far apart, a run of empty ones among them, the queries' and keys' lengths their own."""
    rng = random.Random(13)
    ql = [rng.choice((0, 1, 5, 17, 40)) for _ in range(500)]
    kl = [rng.choice((0, 1, 9, 33, 150)) for _ in range(500)]
    ql[200:300] = kl[180:280] = [0] * 100
    H, K, D = 4, 2, 64
    qe, qo = pack_offsets(ql)
    ke, ko = pack_offsets(kl)
    gen = torch.Generator(device="cuda").manual_seed(14)
    q, g = (normal(gen, qe[-1] + 2, H, D, dtype=dtype) for _ in range(2))
    k, v = (normal(gen, ke[-1] + 3, K, D, dtype=dtype) for _ in range(2))
    out, lse = pkg.attention_fwd(q, k, v, causal=causal, offsets=qo, kv_offsets=ko, want_stats=True)
    got = pkg.attention_bwd(g, q, k, v, out, lse, causal=causal, offsets=qo, kv_offsets=ko)
    for a, b, c, d in zip(qe, qe[1:], ke, ke[1:]):
        if a == b:
            assert (got[1][c:d] == 0).all() and (got[2][c:d] == 0).all()
            continue
        seen = visible(b - a, d - c, causal, d - c)
        check_sequence(out[a:b], lse[:, a:b], q[a:b], k[c:d], v[c:d], D ** -0.5, seen)
        check_gradients([got[0][a:b], got[1][c:d], got[2][c:d]], g[a:b], q[a:b], k[c:d], v[c:d],
                        out[a:b], D ** -0.5, seen)
    assert (out[qe[-1]:] == 0).all() and (got[0][qe[-1]:] == 0).all()
    assert (got[1][ke[-1]:] == 0).all() and (got[2][ke[-1]:] == 0).all()


def test_small_float16_gradients(pkg):
    """Gradients far below float16's normal range times a probability keep their digits."""
    B, T, H, D = 1, 700, 2, 64
    q, k, v = inputs(13, B, T, T, H, H, D, HF)
    g = normal(torch.Generator(device="cuda").manual_seed(14), *q.shape, dtype=HF, std=2.0 ** -8)
    out, lse = pkg.attention_fwd(q, k, v, want_stats=True)
    got = pkg.attention_bwd(g, q, k, v, out, lse)
    check_gradients([t[0] for t in got], g[0], q[0], k[0], v[0], out[0], D ** -0.5,
                    visible(T, T, False, T))


@pytest.mark.parametrize("shape", [(2, 140, 260, 4, 2, 64), (1, 1500, 300, 16, 1, 64)], ids=str)
@pytest.mark.parametrize("needs", [(True, False, False), (False, True, False), (False, False, True)])
def test_single_gradients(pkg, needs, shape):
    q, k, v = inputs(15, *shape, BF)
    g = normal(torch.Generator(device="cuda").manual_seed(16), *q.shape)
    out, lse = pkg.attention_fwd(q, k, v, want_stats=True)
    every = pkg.attention_bwd(g, q, k, v, out, lse)
    some = pkg.attention_bwd(g, q, k, v, out, lse, needs=needs)
    for n, x, y in zip(needs, every, some):
        assert torch.equal(x, y) if n else y is None


def test_autograd_strided(pkg):
    """q, k and v as they lie in one product, and heads before tokens; an expanded
    gradient."""
    gen = torch.Generator(device="cuda").manual_seed(17)
    B, T, H, K, D = 2, 200, 4, 2, 72
    wide = normal(gen, B, T, (H + 2 * K) * D).requires_grad_()
    q, k, v = (t.unflatten(-1, (-1, D)) for t in wide.split([H * D, K * D, K * D], -1))
    out = pkg.fused_attention(q, k, v, causal=True)
    plain = pkg.fused_attention(q.detach().contiguous(), k.detach().contiguous(),
                                v.detach().contiguous(), causal=True)
    assert torch.equal(out, plain)
    turned = [t.detach().transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v)]
    assert torch.equal(pkg.fused_attention(*turned, causal=True), plain)
    out.sum().backward()  # its gradient is one element, expanded
    leaves = [t.detach().clone().requires_grad_() for t in (q, k, v)]
    pkg.fused_attention(*leaves, causal=True).backward(torch.ones_like(plain))
    want = torch.cat([t.grad.flatten(2) for t in leaves], -1)
    assert torch.equal(wide.grad, want)


def test_copies_what_cannot_be_read_in_place(pkg):
    q, k, v = inputs(18, 2, 50, 50, 2, 2, 64, BF)
    out = pkg.fused_attention(q, k, v)
    odd = [torch.empty(t.numel() + 1, dtype=BF, device="cuda")[1:].view(t.shape).copy_(t)
           for t in (q, k, v)]
    assert torch.equal(pkg.fused_attention(*odd), out)
    one = k[:, :, :1]
    assert torch.equal(pkg.fused_attention(q, one.expand(-1, -1, 2, -1), v[:, :, :1].expand(-1, -1, 2, -1)),
                       pkg.fused_attention(q, one, v[:, :, :1]))


def test_differences(pkg):
    """The gradient against central differences of the forward, along the gradient.

    What they may differ by is what the definition's own differ by in float64 (the
    step's third-order term) and what the outputs' errors add up to, each weighted by
    the loss's |g|, and the gradient's own."""
    T, H, D = 64, 2, 32
    q, k, v = inputs(19, 1, T, T, H, H, D, HF)
    gen = torch.Generator(device="cuda").manual_seed(20)
    g = normal(gen, *q.shape, dtype=HF, std=0.1)
    out, lse = pkg.attention_fwd(q, k, v, want_stats=True)
    grads = pkg.attention_bwd(g, q, k, v, out, lse)
    seen = visible(T, T, False, T)
    wide = [t[0].double().requires_grad_() for t in (q, k, v)]
    ref, ref_lse = definition(*wide, D ** -0.5, seen)[:2]
    exact = torch.autograd.grad(ref, wide, g[0].double())
    bounds = definition_bwd(g[0], q[0], k[0], v[0], out[0], D ** -0.5, seen, ref_lse.detach())
    for i in range(3):
        d = grads[i].double() / grads[i].double().norm()
        moved, ours, theirs, rounding = [], [], [], 0.0
        for sign in (1, -1):
            at = [q, k, v]
            at[i] = (at[i].double() + sign * d).to(HF)
            moved.append(at[i][0].double())
            ours.append(pkg.attention_fwd(*at)[0][0].double())
            right, _, bound, _ = definition(*[t[0] for t in at], D ** -0.5, seen)
            theirs.append(right)
            rounding += (bound * g[0].abs()).sum()
        step = moved[0] - moved[1]
        change = ((ours[0] - ours[1]) * g[0].double()).sum()
        truth = ((theirs[0] - theirs[1]) * g[0].double()).sum()
        along = (step * grads[i][0].double()).sum()
        curve = (truth - (step * exact[i]).sum()).abs()
        slack = (step.abs() * bounds[i][1]).sum()
        assert curve <= 0.2 * along.abs()  # the step is small enough to tell
        assert (change - along).abs() <= curve + rounding + slack


def test_repeats_bit_for_bit(pkg):
    q, k, v = inputs(21, 2, 1030, 1030, 8, 2, 128, BF)
    g = normal(torch.Generator(device="cuda").manual_seed(22), *q.shape)
    first = None
    for _ in range(3):
        out, lse = pkg.attention_fwd(q, k, v, causal=True, want_stats=True)
        all_ = (out, lse, *pkg.attention_bwd(g, q, k, v, out, lse, causal=True))
        first = first or all_
        assert all(torch.equal(x, y) for x, y in zip(first, all_))


def test_no_queries_and_no_keys(pkg):
    q, k, v = inputs(23, 2, 0, 30, 2, 2, 64, BF)
    out, lse = pkg.attention_fwd(q, k, v, want_stats=True)
    assert out.shape == q.shape
    dq, dk, dv = pkg.attention_bwd(out, q, k, v, out, lse)
    assert dq.shape == q.shape and (dk == 0).all() and (dv == 0).all()
    q, k, v = inputs(24, 2, 30, 0, 2, 2, 64, BF)
    out, lse = pkg.attention_fwd(q, k, v, want_stats=True)
    dq, dk, dv = pkg.attention_bwd(out, q, k, v, out, lse)
    assert (out == 0).all() and (dq == 0).all() and dk.shape == k.shape


def test_backward_first_on_a_new_thread(pkg):
    """A host thread whose first use of the device is the backward, as autograd's may be."""
    import threading

    q, k, v = inputs(25, 1, 64, 64, 2, 2, 64, BF)
    out, lse = pkg.attention_fwd(q, k, v, want_stats=True)
    want = pkg.attention_bwd(out, q, k, v, out, lse)
    got = []
    t = threading.Thread(target=lambda: got.extend(pkg.attention_bwd(out, q, k, v, out, lse)))
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and len(got) == 3


def test_output_strides(pkg):
    """The backward takes the output at any strides."""
    q, k, v = inputs(26, 2, 70, 70, 4, 2, 72, BF)
    out, lse = pkg.attention_fwd(q, k, v, want_stats=True)
    turned = out.transpose(1, 2).contiguous().transpose(1, 2)
    for a, b in zip(pkg.attention_bwd(out, q, k, v, out, lse),
                    pkg.attention_bwd(turned, q, k, v, turned, lse)):
        assert torch.equal(a, b)


# ------------------------------------------------------- streams, graphs, failures

def test_waits_that_run_out(pkg):
    """Copies announced larger than they are: the bounded waits run out, the rows of
    those blocks are NaN, the device status says so, and the next call is right."""
    import ctypes

    q, k, v = inputs(30, 1, 200, 200, 2, 1, 64, BF)
    g = normal(torch.Generator(device="cuda").manual_seed(31), *q.shape)

    def step():
        out, lse = pkg.attention_fwd(q, k, v, want_stats=True)
        return (out, lse, *pkg.attention_bwd(g, q, k, v, out, lse))

    flags = ctypes.c_uint(0)
    with pkg._abi.using_test_library() as lib:
        want = step()
        assert lib.gbssim_device_status(ctypes.byref(flags)) == 0 and flags.value == 0
        lib.gbssim_tune_attention(16)
        try:
            out, lse = pkg.attention_fwd(q, k, v, want_stats=True)
            torch.cuda.synchronize()
            grads = pkg.attention_bwd(g, q, k, v, want[0], want[1])
            torch.cuda.synchronize()
        finally:
            lib.gbssim_tune_attention(0)
        for t in (out, lse, *grads):
            assert t.isnan().all()
        assert lib.gbssim_device_status(ctypes.byref(flags)) == 0
        assert flags.value == 4  # GBSSIM_DEV_ATTENTION_TIMEOUT
        again = step()
        assert lib.gbssim_device_status(ctypes.byref(flags)) == 0 and flags.value == 0
    assert all(torch.equal(a, b) for a, b in zip(want, again))


# batch form with few blocks (keys in parts), packed, float16
GRAPHS = [dict(shape=((1, 2, 4, 64), (1, 1500, 2, 64)), dtype=BF, packed=None),
          dict(shape=((300, 4, 72), (300, 2, 72)), dtype=HF, packed=[100, 0, 170])]


@pytest.mark.parametrize("case", GRAPHS, ids=["batch", "packed"])
def test_in_a_graph(pkg, case):
    """Captured with the backward, replayed on new inputs and new offsets; two graphs
    whose replays overlap on two streams do not share memory."""
    q_shape, k_shape = case["shape"]

    def make(seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        t = [normal(gen, *s, dtype=case["dtype"]) for s in (q_shape, k_shape, k_shape, q_shape)]
        offsets = None
        if case["packed"]:
            lengths = case["packed"][seed % 3:] + case["packed"][:seed % 3]
            offsets = pack_offsets(lengths)[1]
        return t, offsets

    def step(t, offsets):
        q, k, v, g = t
        out, lse = pkg.attention_fwd(q, k, v, offsets=offsets, want_stats=True)
        return (out, lse, *pkg.attention_bwd(g, q, k, v, out, lse, offsets=offsets))

    graphs = []
    for n in range(2):
        held, offsets = make(40 + n)
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            step(held, offsets)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = step(held, offsets)
        graphs.append((graph, stream, held, offsets, got))
    for seed in (50, 51, 52):
        want = []
        for n, (graph, stream, held, offsets, got) in enumerate(graphs):
            fresh, fresh_offsets = make(seed + 10 * n)
            want.append([t.clone() for t in step(fresh, fresh_offsets)])
            for a, b in zip(held, fresh):
                a.copy_(b)
            if offsets is not None:
                offsets.copy_(fresh_offsets)
        torch.cuda.synchronize()
        for graph, stream, *_ in graphs:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for (*_, got), ref in zip(graphs, want):
            assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_streams_and_threads(pkg):
    """Calls from two host threads, on the default stream and on streams of their own."""
    import threading

    sets = [inputs(60 + n, 1, 1 + 70 * n, 1500, 4, 2, 64, BF) for n in range(2)]

    def step(n):
        q, k, v = sets[n]
        out, lse = pkg.attention_fwd(q, k, v, want_stats=True)
        return (out, *pkg.attention_bwd(out, q, k, v, out, lse))

    want = [step(n) for n in range(2)]
    torch.cuda.synchronize()
    for own in (False, True):
        got, errors = [[], []], []

        def worker(n):
            try:
                with torch.cuda.stream(torch.cuda.Stream() if own else torch.cuda.default_stream()):
                    for _ in range(50):
                        got[n].append(step(n))
            except Exception as e:  # noqa: BLE001 - reported below
                errors.append(repr(e))

        threads = [threading.Thread(target=worker, args=(n,)) for n in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        assert not errors, errors
        for n in range(2):
            assert len(got[n]) == 50
            for r in got[n]:
                assert all(torch.equal(a, b) for a, b in zip(r, want[n]))


def test_bad_offsets_touch_nothing_else(pkg):
    """Lengths and offsets out of their range: no result is promised, but every row that is
    written is one of the outputs', and the next call is right."""
    q, k, v = inputs(70, None, 200, 200, 2, 2, 64, BF)
    good = pack_offsets([120, 80])[1]
    want = pkg.attention_fwd(q, k, v, offsets=good)[0]
    for bad in ([5, 400, -7], [0, 2 ** 31 - 1, 200], [-2 ** 31, 100, 50]):
        offsets = torch.tensor(bad, dtype=torch.int32, device="cuda")
        out, lse = pkg.attention_fwd(q, k, v, offsets=offsets, want_stats=True)
        pkg.attention_bwd(out, q, k, v, out, lse, offsets=offsets)
    q4, k4, v4 = (t.view(2, 100, 2, 64) for t in (q, k, v))
    lengths = torch.tensor([-5, 1000], dtype=torch.int32, device="cuda")
    out = pkg.attention_fwd(q4, k4, v4, kv_lengths=lengths)[0]
    assert (out[0] == 0).all() and torch.equal(out[1:], pkg.attention_fwd(q4[1:], k4[1:], v4[1:])[0])
    assert torch.equal(pkg.attention_fwd(q, k, v, offsets=good)[0], want)


def test_refusals(pkg):
    q, k, v = inputs(71, 2, 10, 20, 4, 2, 64, BF)
    off = torch.tensor([0, 10], dtype=torch.int32, device="cuda")

    def bad(error, *a, **kw):
        with pytest.raises(error):
            pkg.fused_attention(*a, **kw)

    bad(TypeError, q.float(), k.float(), v.float())
    bad(TypeError, q, k.to(HF), v)
    bad(TypeError, q, k, v.cpu())
    bad(ValueError, q, k, v[:, :5])
    bad(ValueError, q, k[:1], v[:1])
    bad(ValueError, q[:, :, :3], k, v)
    bad(ValueError, q[..., :60], k[..., :60], v[..., :60])
    bad(ValueError, q[..., :56], k, v)
    bad(ValueError, q[0], k[0], v[0])
    bad(ValueError, q, k, v, offsets=off)
    bad(ValueError, q, k, v, kv_offsets=off)
    bad(ValueError, q[0], k[0], v[0], offsets=off)  # other rows without offsets of their own
    bad(ValueError, q[0], k[0], v[0], offsets=off, kv_offsets=off[:1])
    bad(ValueError, q[0], k[0], v[0], offsets=off, kv_lengths=off)
    bad(TypeError, q, k, v, kv_lengths=[10, 20])
    bad(TypeError, q, k, v, kv_lengths=off.long())
    bad(ValueError, q, k, v, kv_lengths=off[:1])
    bad(TypeError, q, k, v, kv_lengths=off.cpu())
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        bad(ValueError, q, k, v, scale=scale)
    out, lse = pkg.attention_fwd(q, k, v, want_stats=True)
    for args in ((out[:1], q, k, v, out, lse), (out, q, k, v, out[:, :5], lse),
                 (out, q, k, v, out, lse.transpose(1, 2)), (out, q, k, v, out, lse.double())):
        with pytest.raises(ValueError):
            pkg.attention_bwd(*args)
    with pytest.raises(TypeError):
        pkg.attention_bwd(out.float(), q, k, v, out, lse)


# ------------------------------------------------------------- as they are used together

def test_a_block_of_a_transformer(pkg):
    """The norm before a block, q, k and v of one product, their positions, attention, the
    output's product and the norms around the residual sum, against the same in float64,
    with every gradient.

    Each of the eleven tensors between the operators is rounded to bfloat16 (relative 2^-9
    as a root mean square, 2^-8 at most), probabilities and their gradients once more:
    errors that are independent add up to less than 2^-8 sqrt(13) of a gradient's norm
    forward and back, 2 % taken together."""
    gen = torch.Generator(device="cuda").manual_seed(80)
    B, side, H, K, D, dim = 2, 9, 4, 2, 32, 128
    T = side * side
    x = normal(gen, B, T, dim, dtype=torch.float32)
    w_in = normal(gen, (H + 2 * K) * D, dim, std=dim ** -0.5)
    w_out = normal(gen, dim, H * D, std=(H * D) ** -0.5)
    gain = (1 + 0.1 * torch.randn(dim, generator=gen, device="cuda"))
    at = torch.stack(torch.meshgrid(torch.arange(side), torch.arange(side), indexing="ij"),
                     -1).view(T, 2).cuda()
    pairs = (8, 8)
    f = pkg.rotary_frequencies(pairs)
    g_x, g_u = normal(gen, B, T, dim, dtype=torch.float32), normal(gen, B, T, dim)

    leaves = [t.clone().requires_grad_() for t in (x, w_in, w_out, gain)]
    lx, li, lo, lg = leaves
    _, u = pkg.fused_residual_norm(lx, pre_weight=lg, u_dtype=BF)
    q, k, v = (t.unflatten(-1, (-1, D)) for t in (u @ li.T).split([H * D, K * D, K * D], -1))
    q, k = pkg.fused_rotary(q, k, at, f, pairs)
    y = pkg.fused_attention(q, k, v, causal=True).flatten(2) @ lo.T
    x1, u1 = pkg.fused_residual_norm(lx, y, post_norm="rms", pre_weight=lg)
    got = torch.autograd.grad((x1, u1), leaves, (g_x, g_u))

    wide = [t.double().requires_grad_() for t in (x, w_in, w_out, gain)]
    wx, wi, wo, wg = wide
    rms = lambda t: t * (t.square().mean(-1, keepdim=True) + 1e-6).rsqrt()  # noqa: E731
    q, k, v = (t.unflatten(-1, (-1, D)) for t in
               ((rms(wx) * wg) @ wi.T).split([H * D, K * D, K * D], -1))
    angle = (at.double()[:, [0] * 8 + [1] * 8] * f)[:, None]
    turn = lambda t: torch.cat([t[..., :16] * angle.cos() - t[..., 16:] * angle.sin(),  # noqa: E731
                                t[..., :16] * angle.sin() + t[..., 16:] * angle.cos()], -1)
    q, k, v = turn(q), turn(k).repeat_interleave(H // K, 2), v.repeat_interleave(H // K, 2)
    s = torch.einsum("bihd,bjhd->bhij", q, k) * D ** -0.5
    s = s.masked_fill(torch.ones(T, T, dtype=torch.bool, device="cuda").triu(1), -float("inf"))
    o = torch.einsum("bhij,bjhd->bihd", s.softmax(-1), v).flatten(2)
    r1 = wx + rms(o @ wo.T)
    ref_u = rms(r1) * wg
    ref = torch.autograd.grad((r1, ref_u), wide, (g_x.double(), g_u.double()))
    for a, b in ((x1, r1), (u1, ref_u), *zip(got, ref)):
        assert (a.double() - b).norm() <= 0.02 * b.norm()


@pytest.mark.parametrize("shape", [(1, 1, 1500, 4, 2, 64), (1, 4, 3000, 4, 2, 64),
                                   (1, 50, 900, 2, 2, 128)], ids=str)
def test_rows_do_not_depend_on_others(pkg, shape):
    """Rows of a tile that are no query hold whatever shared memory held: results repeat bit
    for bit whatever ran before."""
    q, k, v = inputs(72, *shape, BF)
    want = pkg.attention_fwd(q, k, v, want_stats=True)
    loud = [300 * t for t in inputs(73, 2, 300, 300, 8, 8, 128, BF)]
    for n in range(20):
        if n % 2:
            pkg.attention_fwd(*loud)
        got = pkg.attention_fwd(q, k, v, want_stats=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), n


@pytest.mark.parametrize("dtype", [BF, HF], ids=str)
@pytest.mark.parametrize("keys", [1, 2, 3, 16])
def test_gradients_over_few_keys(pkg, keys, dtype):
    """Where a query sees one key, its gradient and the key's are zero exactly; where it
    sees a few, the output's rounding is not in them: ds is off by its own rounding (u)
    and float32 sums alone."""
    q, k, v = inputs(74, 2, 5, keys, 4, 2, 40, dtype)
    g = normal(torch.Generator(device="cuda").manual_seed(75), *q.shape, dtype=dtype)
    for causal in (False, True):
        out, lse = pkg.attention_fwd(q, k, v, causal=causal, want_stats=True)
        dq, dk, _ = pkg.attention_bwd(g, q, k, v, out, lse, causal=causal)
        if keys == 1:
            assert (dq == 0).all() and (dk == 0).all()
            continue
        for b in range(2):
            seen = visible(5, keys, causal, keys)
            _, ref_lse, _, _ = definition(q[b], k[b], v[b], 40 ** -0.5, seen)
            exact = definition(q[b], k[b], v[b], 40 ** -0.5, seen)[0]
            for t, (ref, bound) in zip((dq[b], dk[b]),
                                       definition_bwd(g[b], q[b], k[b], v[b], exact, 40 ** -0.5,
                                                      seen, ref_lse)):
                assert ((t.double() - ref).abs() <= bound).all()
        if causal and keys <= 5:
            first = 5 - keys  # the first query that sees a key sees one
            assert (dq[:, first] == 0).all()


@pytest.mark.parametrize("shape", [(2, 2383, 2383, 16, 8, 16), (1, 3001, 3001, 3, 1, 64)], ids=str)
def test_warps_apart(pkg, shape):
    """Many tiles of narrow heads, where a block's warps may be a tile apart."""
    q, k, v = inputs(76, *shape, BF)
    g = normal(torch.Generator(device="cuda").manual_seed(77), *q.shape)
    out, lse = pkg.attention_fwd(q, k, v, causal=True, want_stats=True)
    want = pkg.attention_bwd(g, q, k, v, out, lse, causal=True)
    assert all(t.isfinite().all() for t in want)
    for _ in range(30):
        got = pkg.attention_bwd(g, q, k, v, out, lse, causal=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
