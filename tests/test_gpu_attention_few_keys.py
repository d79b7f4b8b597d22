"""Sequences of a few keys inside large packed and ragged calls: their gradients are those of
the same sequences alone.

Tolerance: over up to 16 keys the output's rounding is not in the gradients, so the bound
is test_gpu_attention's with the exact output in place of the rounded one."""
import pytest

from test_gpu_attention import (BF, HF, definition, definition_bwd, inputs, normal,  # noqa: F401
                                pack_offsets, pkg, visible)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def check_few(dq, dk, g, q, k, v, seen):
    scale = q.shape[-1] ** -0.5
    exact, lse, _, _ = definition(q, k, v, scale, seen)
    for t, (ref, bound) in zip((dq, dk), definition_bwd(g, q, k, v, exact, scale, seen, lse)):
        assert ((t.double() - ref).abs() <= bound).all(), ((t.double() - ref).abs() / bound).max().item()


@pytest.mark.parametrize("dtype", [BF, HF], ids=str)
@pytest.mark.parametrize("dim", [32, 56, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_packed(pkg, dim, dtype, causal):  # noqa: F811
    ql, kl = [40, 2, 2600, 16, 0, 5, 130], [2, 2, 2600, 16, 9, 3, 15]
    qe, qo = pack_offsets(ql)
    ke, ko = pack_offsets(kl)
    q = inputs(1, None, qe[-1], 1, 2, 2, dim, dtype)[0]
    _, k, v = inputs(2, None, 1, ke[-1], 2, 2, dim, dtype)
    g = normal(torch.Generator(device="cuda").manual_seed(3), *q.shape, dtype=dtype)
    out, lse = pkg.attention_fwd(q, k, v, causal=causal, offsets=qo, kv_offsets=ko, want_stats=True)
    got = pkg.attention_bwd(g, q, k, v, out, lse, causal=causal, offsets=qo, kv_offsets=ko)
    for n, m, a, c in zip(ql, kl, qe, ke):
        if m > 16 or n == 0:
            continue
        b, d = a + n, c + m
        check_few(got[0][a:b], got[1][c:d], g[a:b], q[a:b], k[c:d], v[c:d], visible(n, m, causal, m))
        o, l = pkg.attention_fwd(q[None, a:b], k[None, c:d], v[None, c:d], causal=causal, want_stats=True)
        alone = pkg.attention_bwd(g[None, a:b], q[None, a:b], k[None, c:d], v[None, c:d], o, l, causal=causal)
        assert torch.equal(got[0][a:b], alone[0][0])
        assert torch.equal(got[1][c:d], alone[1][0]) and torch.equal(got[2][c:d], alone[2][0])


def test_key_lengths(pkg):  # noqa: F811
    q, k, v = inputs(4, 3, 70, 3000, 4, 2, 64, BF)
    g = normal(torch.Generator(device="cuda").manual_seed(5), *q.shape)
    lengths = [3, 2500, 16]
    kv = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out, lse = pkg.attention_fwd(q, k, v, kv_lengths=kv, want_stats=True)
    got = pkg.attention_bwd(g, q, k, v, out, lse, kv_lengths=kv)
    for b, n in enumerate(lengths):
        if n <= 16:
            check_few(got[0][b], got[1][b, :n], g[b], q[b], k[b, :n], v[b, :n], visible(70, n, False, n))
