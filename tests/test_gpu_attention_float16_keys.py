"""Attention's forward in float16 where its range counts: quiet keys beside a loud one.

Tolerances are test_gpu_attention's.  They add what lies below the type's range:
a probability is held to 2^-35 of the row's largest, which is off by half of that, 2^-36,
at most, for each key, times |v|.
"""
import pytest

from test_gpu_attention import HF, definition, inputs, normal, pkg, visible  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def check_quiet(out, lse, q, k, v, scale, seen):
    ref, ref_lse, bound, lse_bound = definition(q, k, v, scale, seen)
    group = q.shape[1] // k.shape[1]
    least = torch.einsum("ij,jhd->ihd", seen.double(), v.double().abs().repeat_interleave(group, 1))
    bound = bound + 2.0 ** -36 * least + 2.0 ** -25
    assert ((out.double() - ref).abs() <= bound).all(), \
        ((out.double() - ref).abs() / bound).max().item()
    assert ((lse.double() - ref_lse).abs() <= lse_bound).all()


@pytest.mark.parametrize("below", [16.0, 17.25, 18.0])
@pytest.mark.parametrize("queries, keys, causal", [(1, 65536, False), (300, 40000, True), (300, 40000, False)])
@pytest.mark.parametrize("where", ["first", "last"])
def test_quiet_keys(pkg, queries, keys, causal, below, where):  # noqa: F811
    """A loud key whose value is zero, as attention sinks have it, and thousands of quiet
    ones, in one packed sequence."""
    dim = 64
    q = torch.zeros(queries, 2, dim, dtype=HF, device="cuda")
    k, v = (torch.zeros(keys, 2, dim, dtype=HF, device="cuda") for _ in range(2))
    q[..., 0] = 8.0
    v[:] = torch.linspace(0.5, 1.5, dim, device="cuda").to(HF)
    loud = 0 if where == "first" else keys - queries  # seen by all
    k[loud, :, 0] = below / 8.0
    v[loud] = 0.0
    off = [torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (queries, keys)]
    out, lse = pkg.attention_fwd(q, k, v, scale=1.0, causal=causal, offsets=off[0], kv_offsets=off[1],
                                 want_stats=True)
    check_quiet(out, lse, q, k, v, 1.0, visible(queries, keys, causal, keys))
    assert (out > 0).all()


@pytest.mark.parametrize("queries, keys, dim", [(200, 5000, 64), (700, 3000, 128), (3, 30000, 72)])
def test_scores_far_apart(pkg, queries, keys, dim):  # noqa: F811
    """Scores of standard deviation 6: their running maximum grows over many tiles."""
    q, k, v = inputs(1, 1, queries, keys, 2, 1, dim, HF)
    out, lse = pkg.attention_fwd(q, k, v, scale=6 * dim ** -0.5, causal=True, want_stats=True)
    check_quiet(out[0], lse[0], q[0], k[0], v[0], 6 * dim ** -0.5, visible(queries, keys, True, keys))


def test_maxima_that_climb(pkg):  # noqa: F811
    """Scores that rise from key to key, by little a tile, and by much."""
    dim, keys = 64, 2000
    for rise in (0.001, 0.01, 0.03):
        gen = torch.Generator(device="cuda").manual_seed(2)
        q, k = (torch.zeros(n, 1, dim, dtype=HF, device="cuda") for n in (130, keys))
        q[..., 0] = 1.0
        k[:, 0, 0] = (torch.arange(keys, device="cuda") * rise).to(HF)
        v = normal(gen, keys, 1, dim, dtype=HF)
        out, lse = pkg.attention_fwd(q[None], k[None], v[None], scale=1.0, want_stats=True)
        check_quiet(out[0], lse[0], q, k, v, 1.0, visible(130, keys, False, keys))
