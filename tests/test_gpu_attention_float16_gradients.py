"""Attention's backward in float16: the scale that small gradients are kept by comes from the
rows that they belong to.  Tolerances are test_gpu_attention's."""
import pytest

from test_gpu_attention import (HF, check_gradients, inputs, normal, pack_offsets,  # noqa: F401
                                pkg, visible)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

LENGTHS = [150, 0, 300, 40]


def packed(seed, tail, stretch=1.0):
    """stretch, a power of two: of keys, taken from queries; the scores stay, the gradients of
    queries grow by it, out of the type's subnormal numbers."""
    ends, offsets = pack_offsets(LENGTHS)
    q, k, v = inputs(seed, None, ends[-1] + tail, ends[-1] + tail, 4, 2, 64, HF)
    g = normal(torch.Generator(device="cuda").manual_seed(seed + 1), *q.shape, std=1e-6, dtype=HF)
    return ends, offsets, q / stretch, k * stretch, v, g


def both(pkg, q, k, v, g, **kw):  # noqa: F811
    out, lse = pkg.attention_fwd(q, k, v, want_stats=True, **kw)
    return (out, *pkg.attention_bwd(g, q, k, v, out, lse, **kw))


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("stretch", [1024.0, 1 / 1024])
@pytest.mark.parametrize("held", [float("nan"), float("inf"), 65504.0])
def test_rows_behind_the_last_sequence(pkg, held, stretch, causal):  # noqa: F811
    """What they hold changes no bit of any sequence's gradients."""
    ends, offsets, *t = packed(10, 9, stretch)
    got = []
    for x in (0.0, held):
        for a in t:
            a[ends[-1]:] = x
        got.append(both(pkg, *t, causal=causal, offsets=offsets))
    for a, b in zip(*got):
        assert torch.equal(a[:ends[-1]], b[:ends[-1]]) and (b[ends[-1]:] == 0).all()
    q, k, v, g = t
    for a, b in zip(ends, ends[1:]):
        check_gradients([x[a:b] for x in got[1][1:]], g[a:b], q[a:b], k[a:b], v[a:b],
                        got[1][0][a:b], 64 ** -0.5, visible(b - a, b - a, causal, b - a))


@pytest.mark.parametrize("held", [float("nan"), 1e4])
def test_sequences_do_not_meet(pkg, held):  # noqa: F811
    """One of NaN, or a much louder one, changes no bit of the others."""
    ends, offsets, *t = packed(12, 0)
    before = both(pkg, *t, offsets=offsets)
    for a in t[2:]:
        a[ends[2]:ends[3]] = held
    after = both(pkg, *t, offsets=offsets)
    for a, b in zip(before, after):
        assert torch.equal(a[:ends[2]], b[:ends[2]]) and torch.equal(a[ends[3]:], b[ends[3]:])


@pytest.mark.parametrize("lengths", [False, True])
@pytest.mark.parametrize("held", [float("nan"), 1e4])
def test_samples_do_not_meet(pkg, held, lengths):  # noqa: F811
    q, k, v = inputs(14, 3, 200, 260, 4, 4, 72, HF)
    g = normal(torch.Generator(device="cuda").manual_seed(15), *q.shape, std=1e-6, dtype=HF)
    kw = {"kv_lengths": torch.tensor([260, 100, 31], dtype=torch.int32, device="cuda")} if lengths else {}
    before = both(pkg, q, k, v, g, **kw)
    for a in (v, g):
        a[1] = held
    after = both(pkg, q, k, v, g, **kw)
    for a, b in zip(before, after):
        assert torch.equal(a[::2], b[::2])
    for n, b in ((260, 0), (31 if lengths else 260, 2)):
        check_gradients([after[1][b], after[2][b, :n], after[3][b, :n]], g[b], q[b], k[b, :n], v[b, :n],
                        after[0][b], 72 ** -0.5, visible(200, n, False, n))


def test_queries_that_see_no_key(pkg):  # noqa: F811
    """Their gradient, however large, changes no bit of the others'."""
    q, k, v = inputs(16, 1, 400, 250, 2, 2, 64, HF)
    g = normal(torch.Generator(device="cuda").manual_seed(17), *q.shape, std=1e-6, dtype=HF)
    got = []
    for x in (0.0, 65504.0):
        g[:, :150] = x
        got.append(both(pkg, q, k, v, g, causal=True))
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_a_query_whose_gradient_is_not_finite(pkg):  # noqa: F811
    """It spoils its own gradient (and the keys'), and no digit of the other queries'."""
    q, k, v = inputs(18, 1, 300, 300, 2, 1, 64, HF)
    g = normal(torch.Generator(device="cuda").manual_seed(19), *q.shape, std=1e-6, dtype=HF)
    got = []
    for x in (0.0, float("nan"), float("inf")):
        g[:, 77, 1, 5] = x
        got.append(both(pkg, q, k, v, g)[1])
    rest = torch.ones_like(q, dtype=torch.bool)
    rest[:, 77, 1] = False
    for t in got[1:]:
        assert torch.equal(t[rest], got[0][rest]) and t[:, 77, 1].isnan().all()
