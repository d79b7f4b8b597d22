"""Attention on the GPU against its definition in float64.

Tolerances.  u is half a step of the tensors' type.  A score sums dim products in
float32: it is off by at most e = (dim + 8) 2^-22 scale sum|q k| (a sum that truncates
loses 2^-23 a step), and so is the logarithm of a probability, plus 2^-20 for the
exponential and its argument's rounding (arguments up to 2^4 in steps of 2^-20).  A
probability is rounded once to the type: relative u.  So the output is off by at most
(u + 2 e + 2^-18) sum p|v| + u |o|: errors of the numerator, and the unrounded
denominator's.
"""
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
