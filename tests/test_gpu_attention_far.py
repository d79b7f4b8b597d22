"""Attention over keys and values of more than 2^31 elements, the last of them the ones that
count: offsets beyond 32 bits, forward and backward, in place and along a batch.

Keys but the last `LOUD` are zero: their scores are 0 and, their values zero too, they
only add to the sum of exponentials.  So the definition needs the last keys and the
number of the others; tolerances are test_gpu_attention's, with the quiet keys' share of
the sums added."""
import math

import pytest

from test_gpu_attention import BF, normal, pkg  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DIM, LOUD = 128, 300


@pytest.fixture(scope="module")
def room(pkg):  # noqa: F811
    if torch.cuda.mem_get_info()[0] < 60e9:
        pytest.skip("needs 60 GB")


def close(got, want, terms, extra=0.0):
    """Within the type's rounding of the result and of the probabilities, and float32 sums:
    u of the result, and 2 u + 2^-14 of its terms' magnitudes."""
    u = torch.finfo(got.dtype).eps / 2
    assert ((got.double() - want).abs() <= u * want.abs() + (2 * u + 2.0 ** -14) * terms + extra).all(), \
        (got.double() - want).abs().max().item()


@pytest.mark.parametrize("batch", [1, 3])
def test_last_of_many(pkg, room, batch):  # noqa: F811
    # one sample of 2^31 elements and some, or three of 2^30: the third begins at 2^31
    tokens = 2 ** 24 + 1000 if batch == 1 else 2 ** 23
    gen = torch.Generator(device="cuda").manual_seed(1)
    k = torch.zeros(batch, tokens, 1, DIM, dtype=BF, device="cuda")
    v = torch.zeros_like(k)
    assert k.numel() > 2 ** 31
    k[-1, -LOUD:] = normal(gen, LOUD, 1, DIM, std=3.0)
    v[-1, -LOUD:] = normal(gen, LOUD, 1, DIM)
    q = normal(gen, batch, 4, 2, DIM, std=2.0)
    g = normal(gen, *q.shape)
    out, lse = pkg.attention_fwd(q, k, v, want_stats=True)
    dq, dk, dv = pkg.attention_bwd(g, q, k, v, out, lse)
    kl, vl = k[-1, -LOUD:, 0].double(), v[-1, -LOUD:, 0].double()
    qd, gd = q[-1].double(), g[-1].double()
    s = torch.einsum("ihd,jd->hij", qd, kl) * DIM ** -0.5
    quiet = torch.full((*s.shape[:2], 1), math.log(tokens - LOUD), dtype=torch.float64, device="cuda")
    ref_lse = torch.logsumexp(torch.cat([s, quiet], -1), -1)
    p = torch.exp(s - ref_lse[..., None])
    rest = torch.exp(quiet - ref_lse[..., None])[..., 0]
    assert (p.sum(-1) > 0.3).any()  # the loud ones count
    assert ((lse[-1].double() - ref_lse).abs() <= 2.0 ** -12).all()
    ref = torch.einsum("hij,jd->ihd", p, vl)
    terms = torch.einsum("hij,jd->ihd", p, vl.abs())
    close(out[-1], ref, terms)
    dp = torch.einsum("ihd,jd->hij", gd, vl)
    D = torch.einsum("ihd,ihd->hi", gd, ref)[..., None]
    ds = p * (dp - D)
    # ds is off by the output's rounding in D and by sums of dim products
    u = torch.finfo(BF).eps / 2
    off = p * (2 * u * torch.einsum("ihd,ihd->hi", gd.abs(), terms)[..., None] +
               2.0 ** -14 * torch.einsum("ihd,jd->hij", gd.abs(), vl.abs()))
    scale = DIM ** -0.5
    close(dq[-1], torch.einsum("hij,jd->ihd", ds, kl) * scale,
          torch.einsum("hij,jd->ihd", ds.abs(), kl.abs()) * scale,
          torch.einsum("hij,jd->ihd", off, kl.abs()) * scale)
    close(dk[-1, -LOUD:, 0], torch.einsum("hij,ihd->jd", ds, qd) * scale,
          torch.einsum("hij,ihd->jd", ds.abs(), qd.abs()) * scale,
          torch.einsum("hij,ihd->jd", off, qd.abs()) * scale)
    close(dv[-1, -LOUD:, 0], torch.einsum("hij,ihd->jd", p, gd), torch.einsum("hij,ihd->jd", p, gd.abs()))
    # the quiet keys' gradients: dk from -D alone, dv their share of g
    share = (rest / (tokens - LOUD))[..., None]
    dk_quiet = -torch.einsum("hix,hix,ihd->d", share, D, qd) * scale
    size = (share.squeeze(-1) * D.squeeze(-1).abs()).T[..., None] * qd.abs() * scale
    slack = (share * 2 * u).squeeze(-1) * torch.einsum("ihd,ihd->hi", gd.abs(), terms)
    for n in (0, tokens // 2, tokens - LOUD - 1):
        close(dk[-1, n, 0], dk_quiet, size.sum((0, 1)), (slack.T[..., None] * qd.abs()).sum((0, 1)) * scale)
        close(dv[-1, n, 0], torch.einsum("hix,ihd->d", share, gd),
              torch.einsum("hix,ihd->d", share, gd.abs()))
    if batch > 1:  # the other samples have quiet keys alone
        assert (out[0] == 0).all() and (dq[0] == 0).all()
        assert ((lse[0].double() - math.log(tokens)).abs() <= 2.0 ** -12).all()
