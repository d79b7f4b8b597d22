"""Gradient norm and clipping against float64.

Bars.  A thread sums at most 64 squares in float32 (each sum's relative error
at most 64 x 2^-24), everything beyond in double: the norm, a square root, is
within 32 x 2^-24 + 2^-24 < 2e-6 of its value (sums of |g| within 64 x 2^-24 <
4e-6, a maximum exact).  c takes two roundings more, c g one more in the
output's type: half an ulp, 2^-24 float32, 2^-8 bfloat16, 2^-11 float16 (and
2^-25 where float16 is subnormal).
"""
import math
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
ULP = {F32: 2.0**-24, BF16: 2.0**-8, F16: 2.0**-11}
TINY = {F32: 2.0**-149, BF16: 2.0**-133, F16: 2.0**-25}
NORM_TOL = {2: 2e-6, 1: 4e-6, math.inf: 0.0}


@pytest.fixture(scope="module")
def pkg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import differentiable_image_quality_gb300 as pkg
    from differentiable_image_quality_gb300 import _build

    _build.build()
    return pkg


def make(sizes, types, seed=0, offset=0, scale=1e-2):
    """Tensors of the given sizes, each `offset` elements into its storage."""
    gen = torch.Generator().manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        t = types[i % len(types)]
        buf = torch.empty(n + offset, dtype=t, device="cuda")
        v = buf[offset:]
        v.copy_((torch.randn(n, generator=gen) * scale * (1 + i % 5)).to(t))
        out.append(v)
    return out


def norm64(ts, p=2):
    parts = [t.detach().cpu().double().reshape(-1) for t in ts]
    v = torch.cat(parts) if parts else torch.zeros(0, dtype=torch.float64)
    if v.numel() == 0:
        return 0.0
    return float({2: lambda: v.square().sum().sqrt(), 1: lambda: v.abs().sum(),
                  math.inf: lambda: v.abs().max()}[p]())


def check_norm(got, ref, p=2):
    assert got.dtype == F32 and got.dim() == 0
    assert abs(float(got) - ref) <= NORM_TOL[p] * ref + 2.0**-149, (float(got), ref)


def check_scaled(outs, before, max_norm, ref):
    coef = min(1.0, max_norm / (ref + 1e-6))
    for o, g in zip(outs, before):
        want = g.cpu().double() * coef
        err = (o.cpu().double() - want).abs()
        bar = want.abs() * (ULP[o.dtype] + 2.5e-6) + TINY[o.dtype]
        assert bool((err <= bar).all()), float((err - bar).max())


RAGGED = [1, 7, 8192, 16384, 16385, 3, 40000, 0, 513, 8191, 100003]


@pytest.mark.parametrize("p", [2, 1, math.inf])
@pytest.mark.parametrize("types", [[F32], [BF16], [F16], [F32, BF16, F16]], ids=str)
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_norm(pkg, p, types, offset):
    ts = make(RAGGED, types, offset=offset)
    check_norm(pkg.grad_norm(ts, p), norm64(ts, p), p)


@pytest.mark.parametrize("n", [1, 32, 33, 1024, 1025, 2500])
def test_many_tensors(pkg, n):
    """Both table sizes, and more tensors than one launch takes."""
    ts = make([(i * 37) % 301 for i in range(n)], [F32, BF16])
    ref = norm64(ts)
    check_norm(pkg.grad_norm(ts), ref)
    before = [t.clone() for t in ts]
    check_norm(pkg.clip_grads(ts, ref / 3), ref)
    check_scaled(ts, before, ref / 3, ref)


def test_nothing_but_empty_tensors(pkg):
    ts = [torch.empty(0, device="cuda"), torch.empty((3, 0), device="cuda")]
    assert float(pkg.grad_norm(ts)) == 0.0
    assert float(pkg.clip_grads(ts, 1.0)) == 0.0


@pytest.mark.parametrize("max_norm", [0.0, 0.3, 1e9, math.inf])
@pytest.mark.parametrize("types", [[F32], [BF16], [F32, BF16, F16]], ids=str)
@pytest.mark.parametrize("offset", [0, 1, 5])
def test_clip_in_place(pkg, max_norm, types, offset):
    ts = make(RAGGED, types, offset=offset)
    ref, before = norm64(ts), [t.clone() for t in ts]
    check_norm(pkg.clip_grads(ts, max_norm), ref)
    check_scaled(ts, before, max_norm, ref)
    if max_norm > 1e8:
        assert all(torch.equal(a, b) for a, b in zip(ts, before))


@pytest.mark.parametrize("out_type", [F32, BF16, F16])
@pytest.mark.parametrize("offsets", [(0, 0), (1, 1), (4, 0), (5, 1), (1, 0), (0, 3)], ids=str)
@pytest.mark.parametrize("types", [[F32], [BF16], [F16]], ids=str)
def test_clip_into_other_tensors(pkg, types, out_type, offsets):
    """Every pair of types, with starts that agree and disagree about 16 bytes; the
    elements around each output stay as they were."""
    ts = make(RAGGED, types, offset=offsets[0])
    before, ref = [t.clone() for t in ts], norm64(ts)
    pads = [torch.full((t.numel() + offsets[1] + 9,), 7.0, dtype=out_type, device="cuda")
            for t in ts]
    outs = [b[offsets[1]:offsets[1] + t.numel()] for b, t in zip(pads, ts)]
    check_norm(pkg.clip_grads(ts, 0.5, out=outs), ref)
    check_scaled(outs, before, 0.5, ref)
    assert all(torch.equal(a, b) for a, b in zip(ts, before))
    for b, t in zip(pads, ts):
        assert bool((b[:offsets[1]] == 7.0).all())
        assert bool((b[offsets[1] + t.numel():] == 7.0).all())


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e25, 1e38])
@pytest.mark.parametrize("t", [F32, BF16], ids=str)
def test_squares_beyond_float32(pkg, scale, t):
    """Squares below 2^-149 or above 2^127: the norm itself is representable."""
    v = torch.linspace(0.1, 1.0, 5000, dtype=torch.float64) * scale / 100
    v[17] = scale
    g = [v.to(t).cuda(), torch.zeros(3000, dtype=t, device="cuda")]
    check_norm(pkg.grad_norm(g), norm64(g))


def test_one_loud_value_among_quiet_ones(pkg):
    v = torch.full((20000,), 1e-25)
    v[12345] = 1e-3
    g = [v.cuda()]
    check_norm(pkg.grad_norm(g), norm64(g))


@pytest.mark.parametrize("p", [2, 1, math.inf])
@pytest.mark.parametrize("t", [F32, BF16, F16], ids=str)
def test_nan_and_infinity(pkg, p, t):
    for value in (math.nan, math.inf, -math.inf):
        ts = make([5000, 100], [t])
        ts[1][37] = value
        n = float(pkg.grad_norm(ts, p))
        assert math.isnan(n) if math.isnan(value) else n == math.inf
        norm = float(pkg.clip_grads(ts, 1.0, p))
        if math.isnan(value):
            assert math.isnan(norm) and all(bool(x.isnan().all()) for x in ts)
        else:
            assert norm == math.inf and bool((ts[0] == 0).all()) and bool(ts[1][37].isnan())


def test_orders_of_dimensions(pkg):
    base = torch.randn(4, 6, 5, 8, device="cuda")
    ts = [base.clone(memory_format=torch.channels_last), base[0].transpose(0, 2).clone(),
          torch.randn(7, 9, device="cuda").t(), torch.randn((), device="cuda")]
    ref, before = norm64(ts), [t.clone() for t in ts]
    check_norm(pkg.clip_grads(ts, 0.1), ref)
    check_scaled(ts, before, 0.1, ref)


def test_refused_layouts(pkg):
    with pytest.raises(ValueError):
        pkg.grad_norm(torch.randn(8, 8, device="cuda")[:, :5])
    with pytest.raises(ValueError):
        pkg.grad_norm(torch.randn(8, 1, device="cuda").expand(8, 4))
    with pytest.raises(ValueError):
        pkg.grad_norm(torch.randn(8, 8, device="cuda").to_sparse())
    with pytest.raises(TypeError):
        pkg.grad_norm(torch.zeros(8, dtype=torch.float64, device="cuda"))
    g = torch.randn(6, 4, device="cuda")
    with pytest.raises(ValueError):
        pkg.clip_grads([g], 1.0, out=[])
    with pytest.raises(ValueError):
        pkg.clip_grads([g], 1.0, out=[torch.empty(4, 6, device="cuda").t()])
    with pytest.raises(ValueError):
        pkg.clip_grads([g], 1.0, out=[torch.empty(5, 4, device="cuda")])
    with pytest.raises(pkg.GbssimError):
        pkg.clip_grads([g, g], 1.0)
    with pytest.raises(pkg.GbssimError):
        pkg.clip_grads([g.view(-1)[:16]], 1.0, out=[g.view(-1)[4:20]])


def test_parameters(pkg):
    ps = [torch.nn.Parameter(torch.randn(5, 3, device="cuda")) for _ in range(3)]
    for p in ps[:2]:
        p.grad = torch.randn_like(p)
    ref, before = norm64([p.grad for p in ps[:2]]), [p.grad.clone() for p in ps[:2]]
    version = ps[0].grad._version
    check_norm(pkg.clip_grad_norm_(ps, 0.1), ref)
    check_scaled([p.grad for p in ps[:2]], before, 0.1, ref)
    assert ps[2].grad is None and ps[0].grad._version > version


def test_repeats_bit_for_bit_and_on_other_streams(pkg):
    ts = make([100003, 70001, 5], [F32, BF16])
    first = pkg.grad_norm(ts)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(pkg.grad_norm(ts))
    torch.cuda.synchronize()
    assert all(float(g) == float(first) for g in got)


def test_in_a_graph(pkg):
    ts = make([40000, 17], [F32, BF16])
    outs = [torch.empty_like(t) for t in ts]
    pkg.clip_grads(ts, 0.5, out=outs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = pkg.clip_grads(ts, 0.5, out=outs)
    for seed in (1, 2):
        new = make([40000, 17], [F32, BF16], seed=seed)
        for t, n in zip(ts, new):
            t.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        ref = norm64(new)
        check_norm(norm, ref)
        check_scaled(outs, new, 0.5, ref)


@pytest.mark.parametrize("many", [False, True])
def test_two_threads_on_one_stream(pkg, many):
    """Calls of two host threads on the stream that both have by default: each
    scales by its own norm."""
    sizes = [301] * 1100 if many else [40000, 17]
    lists = [make(sizes, [F32, BF16], seed=s, scale=10.0**-s) for s in (0, 3)]
    rounds = 40 if many else 400
    want = []
    for ts in lists:
        outs = [torch.empty_like(t) for t in ts]
        want.append((pkg.clip_grads(ts, 1e-4, out=outs), torch.cat([o.float() for o in outs])))
    flat = [torch.empty((rounds, sum(sizes)), device="cuda") for _ in lists]
    got, errors = [None, None], []
    torch.cuda.synchronize()
    start = threading.Barrier(2)

    def work(k):
        try:
            start.wait(30)
            got[k] = [pkg.clip_grads(lists[k], 1e-4, out=list(row.split(sizes))) for row in flat[k]]
        except Exception as e:  # noqa: BLE001 - reported below
            errors.append(repr(e))

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for k, (norm, out) in enumerate(want):
        assert all(torch.equal(n, norm) for n in got[k])
        coef = min(1.0, 1e-4 / (float(norm) + 1e-6))
        whole = torch.cat([t.float() for t in lists[k]]).double() * coef
        err = (flat[k].double() - whole).abs().amax(0)
        assert bool((err <= whole.abs() * (2.0**-24 + 2.5e-6) + 2.0**-149).all())


@pytest.mark.parametrize("p", [2, 1, math.inf])
def test_no_limit_and_infinity(pkg, p):
    """An infinite limit clips nothing, an infinite norm included; a NaN stays one."""
    for value in (math.inf, -math.inf, math.nan):
        ts = make([5000, 100], [F32, F16])
        ts[1][37] = value
        before = [t.clone() for t in ts]
        norm = float(pkg.clip_grads(ts, math.inf, p))
        if math.isnan(value):
            assert math.isnan(norm) and all(bool(x.isnan().all()) for x in ts)
        else:
            assert norm == math.inf and all(torch.equal(a, b) for a, b in zip(ts, before))


def test_strides_that_reach_no_element(pkg):
    """Dimensions of one element may have any stride, beside tensors of any order."""
    g = [torch.randn(4, 6, 5, 8, device="cuda").to(memory_format=torch.channels_last),
         torch.randn(1, 5, device="cuda"), torch.randn(7, 1, 3, 1, device="cuda")]
    outs = [torch.empty_like(g[0]), torch.empty(5, device="cuda").as_strided((1, 5), (1, 1)),
            torch.empty(21, device="cuda").as_strided((7, 1, 3, 1), (3, 99, 1, 50))]
    ref = norm64(g)
    check_norm(pkg.clip_grads(g, 0.1, out=outs), ref)
    check_scaled(outs, g, 0.1, ref)
    other = torch.empty((4, 6, 5, 8), device="cuda")  # dense, in another order
    with pytest.raises(ValueError):
        pkg.clip_grads(g[:2], 1.0, out=[other, outs[1]])
