"""The residual norm against float64, forward and backward.

The reference is the definition in float64, its gradients from torch's autograd
on that definition.  Bars: each output may be off by its type's rounding (half
an ulp: 2^-24 float32, 2^-8 bfloat16, 2^-11 float16, and 2^-25 below float16's
normal range), plus what float32 arithmetic costs.  The latter is bounded by the
formulas evaluated on magnitudes (every difference taken as a sum, every mean
as a mean of magnitudes): a value that is a sum of terms t_i, each a product of
at most eight rounded factors, of which the means come from sums of at most
8 + 5 + 4 + 4 additions in sequence (eight columns of a thread, the lanes, the
warps, the blocks of a row), is within K 2^-24 sum |t_i|, K = 64.  Column sums
add the rows of a block in sequence: K grows by their number.  What a row's
statistics lose to cancellation is in the magnitudes: x' as |s x| + |g z|, the
deviations as the row's largest magnitude, which the factor `loss` (at least 1)
puts into every use of x^ or y^.
"""
import itertools

import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
ULP = {F32: 2.0**-24, BF16: 2.0**-8, F16: 2.0**-11}
TINY = {F32: 2.0**-126, BF16: 2.0**-126, F16: 2.0**-25}
K = 64 * 2.0**-24
NAMES = ("x", "y", "gate", "post_weight", "post_bias", "pre_weight", "pre_bias")
PAIRS = [(F32, F32), (BF16, BF16), (F16, F16), (F32, BF16), (F32, F16)]


@pytest.fixture(scope="module")
def pkg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import differentiable_image_quality_gb300 as pkg
    from differentiable_image_quality_gb300 import _build

    _build.build()
    return pkg


def make(shape, res=F32, blk=F32, par=F32, post="rms", pre="rms", gate="dim", bias=True,
         per_sample=False, scale=1.0, offset=0.0, seed=0):
    """Inputs on the GPU and the operator's keywords."""
    gen = torch.Generator().manual_seed(seed)
    dim = shape[-1]

    def normal(size, std, mean, dtype):
        return (torch.randn(size, generator=gen) * std + mean).to(dtype).cuda()

    psize = (shape[0], dim) if per_sample else (dim,)
    t = {"x": normal(shape, 1.5, 0.3, res), "y": normal(shape, 0.7, -0.2, blk)}
    if gate == "dim":
        t["gate"] = normal(psize, 0.3, 0.6, par)
    elif gate == "rows":
        t["gate"] = normal(shape, 0.3, 0.6, blk)
    if post:
        t["post_weight"] = normal(psize, 0.2, 1.0 - offset, par)
        if bias:
            t["post_bias"] = normal(psize, 0.2, 0.0, par)
    if pre:
        t["pre_weight"] = normal(psize, 0.2, 1.0 - offset, par)
        if bias:
            t["pre_bias"] = normal(psize, 0.2, 0.0, par)
    g = {"x": normal(shape, 0.5, 0.0, res), "u": normal(shape, 0.5, 0.0, blk) if pre else None}
    how = dict(post_norm=post, pre_norm=pre, residual_scale=scale, weight_offset=offset, eps=1e-6)
    return t, g, how


def spread(p, shape):
    """A parameter against [..., dim]."""
    if p is None or p.dim() == 1 or p.shape == torch.Size(shape):
        return p
    return p.reshape(p.shape[0], *[1] * (len(shape) - 2), p.shape[-1])


def definition(t, how):
    """(x_out, u) in float64, and the intermediate values the bars need."""
    def norm(v, kind, weight, bias):
        if kind == "layer":
            v = v - v.mean(-1, keepdim=True)
        r = 1.0
        if kind:
            r = 1.0 / torch.sqrt((v * v).mean(-1, keepdim=True) + how["eps"])
        hat = v * r
        out = hat if weight is None else hat * (weight + how["weight_offset"])
        return hat, r, out if bias is None else out + bias

    shape = t["x"].shape
    p = {k: spread(v, shape) for k, v in t.items()}
    yh, r1, z = norm(t["y"], how["post_norm"], p.get("post_weight"), p.get("post_bias"))
    gz = z if "gate" not in p else z * p["gate"]
    x_out = how["residual_scale"] * t["x"] + gz
    xh, r2, u = norm(x_out, how["pre_norm"], p.get("pre_weight"), p.get("pre_bias"))
    return x_out, u, dict(yh=yh, r1=r1, z=z, gz=gz, xh=xh, r2=r2)


def magnitudes(t, g, how, mid):
    """Per output the sum of its terms' magnitudes (see the top)."""
    shape = t["x"].shape
    p = {k: spread(v, shape) for k, v in t.items()}
    o = how["weight_offset"]
    one = torch.ones((), dtype=torch.float64, device="cuda")
    w1 = (p["post_weight"] + o).abs() if "post_weight" in p else one
    w2 = (p["pre_weight"] + o).abs() if "pre_weight" in p else one
    gate = p["gate"].abs() if "gate" in p else one
    # the loss of each normalised value: its row's largest magnitude over its deviation
    y, r1, r2 = t["y"].abs(), mid["r1"], mid["r2"]
    top = y.amax(-1, keepdim=True)
    yh = mid["yh"].abs() + (top * r1 if how["post_norm"] else 0.0)
    z = yh * w1 + (p["post_bias"].abs() if "post_bias" in p else 0.0)
    x_out = abs(how["residual_scale"]) * t["x"].abs() + gate * z
    # (an error of x' reaches x^ of its column, and by the mean and the deviation all of the row)
    xh = mid["xh"].abs() * (1.0 + x_out.amax(-1, keepdim=True) * r2) + x_out * r2 \
        + x_out.mean(-1, keepdim=True) * r2 if how["pre_norm"] else x_out
    m = {"x_out": x_out, "u": xh * w2 + (p["pre_bias"].abs() if "pre_bias" in p else 0.0)}
    if g is None:
        return m
    gx = g["x"].abs() if g.get("x") is not None else torch.zeros_like(x_out)
    gu = g["u"].abs() if g.get("u") is not None else torch.zeros_like(x_out)
    mean = lambda v: v.mean(-1, keepdim=True)  # noqa: E731
    dxh = gu * w2
    T = gx + dxh
    if how["pre_norm"]:
        T = gx + r2 * (dxh + mean(dxh) + xh * mean(dxh * xh)) * (1.0 + mean(xh))
    m["d_x"] = abs(how["residual_scale"]) * T
    q = T * gate
    dyh = q * w1
    m["d_y"] = dyh if not how["post_norm"] else \
        r1 * (dyh + mean(dyh) + yh * mean(dyh * yh)) * (1.0 + mean(yh))
    rows = {"gate": T * z, "post_weight": q * yh, "post_bias": q, "pre_weight": gu * xh,
            "pre_bias": gu}
    for k, v in rows.items():
        if k in t:
            m["d_" + k] = over_rows(v.expand(shape), t[k])
    return m


def over_rows(v, like):
    if like.shape == v.shape and like.dim() > 1:
        return v
    if like.dim() == 1:
        return v.reshape(-1, v.shape[-1]).sum(0)
    return v.reshape(like.shape[0], -1, v.shape[-1]).sum(1).reshape(like.shape)


def close(name, got, ref, mag, k=K):
    assert got.shape == ref.shape, name
    err = (got.double() - ref).abs()
    bar = ULP[got.dtype] * ref.abs() + TINY[got.dtype] + (1 + ULP[got.dtype]) * k * mag
    worst = (err - bar).max().item() if err.numel() else 0.0
    assert not err.isnan().any() and worst <= 0, \
        f"{name}: over its bar by {worst:.3e} at {int((err - bar).argmax())}"


def check(pkg, t, g, how):
    """Forward and backward, by the two calls, against float64."""
    x_out, u, stats = pkg.residual_norm_fwd(t["x"], t["y"], want_stats=True,
                                            **{k: t[k] for k in NAMES[2:] if k in t}, **how)
    wide = {k: v.detach().double().requires_grad_() for k, v in t.items()}
    x64, u64, mid = definition(wide, how)
    m64 = {k: v.detach() if torch.is_tensor(v) else torch.full((), v, dtype=torch.float64,
                                                               device="cuda")
           for k, v in mid.items()}
    plain = {k: v.detach() for k, v in wide.items()}
    g64 = {k: None if v is None else v.double() for k, v in g.items()}
    mag = magnitudes(plain, g64, how, m64)
    assert x_out.dtype == t["x"].dtype
    close("x_out", x_out, x64.detach(), mag["x_out"])
    if how["pre_norm"]:
        assert u.dtype == t["y"].dtype
        close("u", u, u64.detach(), mag["u"])
    else:
        assert u is None
    outs = [(x64, g64["x"])] + ([(u64, g64["u"])] if g64["u"] is not None else [])
    outs = [(o, v) for o, v in outs if v is not None]
    refs = torch.autograd.grad([o for o, _ in outs], list(wide.values()), [v for _, v in outs],
                               allow_unused=True)
    grads = pkg.residual_norm_bwd(g["x"], g["u"], t["x"], t["y"], stats,
                                  **{k: t[k] for k in NAMES[2:] if k in t}, **how)
    rows = t["x"].numel() // t["x"].shape[-1]
    for name, got in zip(NAMES, grads):
        if name not in t:
            assert got is None
            continue
        ref = refs[list(wide).index(name)]
        ref = torch.zeros_like(wide[name]) if ref is None else ref
        assert got.dtype == t[name].dtype
        summed = name in NAMES[2:] and got.shape != t["x"].shape
        close("d_" + name, got, ref, mag["d_" + name], K + (rows * 2.0**-24 if summed else 0.0))


# every width a plan treats differently: one column, part of a thread, lanes of a
# warp, several teams of a block, blocks with a ragged last warp, clusters
DIMS = [1, 5, 8, 16, 40, 64, 250, 256, 264, 768, 1000, 1001, 1152, 4096, 4097, 4104, 8192, 9001,
        16384]


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("pair", [(F32, F32), (F32, BF16)], ids=str)
def test_widths(pkg, dim, pair):
    check(pkg, *make((2, 7, dim), *pair, post="layer" if dim % 3 else "rms", pre="layer", seed=dim))


@pytest.mark.parametrize("pair", PAIRS, ids=str)
@pytest.mark.parametrize("dim", [96, 333, 1152])
def test_types(pkg, pair, dim):
    check(pkg, *make((3, 11, dim), *pair, par=pair[1]))


@pytest.mark.parametrize("post,pre", list(itertools.product([None, "rms", "layer"], repeat=2)))
@pytest.mark.parametrize("gate", [None, "dim", "rows"])
@pytest.mark.parametrize("bias", [False, True])
def test_norms_and_gates(pkg, post, pre, gate, bias):
    for dim in (72, 515):
        check(pkg, *make((2, 9, dim), F32, BF16, post=post, pre=pre, gate=gate, bias=bias,
                         scale=0.5, offset=1.0))


@pytest.mark.parametrize("shape", [(1, 1, 64), (1, 1, 4096), (1, 1, 16384), (5, 1, 128), (1, 300, 24),
                                   (3, 1000, 64), (40, 2, 512), (2, 3, 5, 4, 80), (200, 48), (33,),
                                   (1, 2500, 1024), (1, 70, 4091), (2, 100, 9001), (1, 80, 16377),
                                   (1, 80, 16383), (3, 333, 45), (1, 999, 1002), (2, 90, 260)],
                         ids=str)
@pytest.mark.parametrize("per_sample", [False, True])
def test_shapes(pkg, shape, per_sample):
    if per_sample and len(shape) < 3:
        pytest.skip("parameters per sample need a sample dimension")
    check(pkg, *make(shape, BF16, BF16, pre="layer", per_sample=per_sample))


def test_no_rows(pkg):
    for shape in ((0, 5, 64), (2, 0, 64), (0, 64)):
        t, g, how = make(shape)
        args = {k: t[k] for k in NAMES[2:]}
        x_out, u, stats = pkg.residual_norm_fwd(t["x"], t["y"], want_stats=True, **args, **how)
        assert x_out.shape == shape and u.shape == shape
        grads = pkg.residual_norm_bwd(g["x"], g["u"], t["x"], t["y"], stats, **args, **how)
        assert all(bool((v == 0).all()) for v in grads[2:])


@pytest.mark.parametrize("dim,tokens", [(64, 10), (520, 10), (1001, 10), (1001, 70), (1002, 50)])
def test_strides_and_alignment(pkg, dim, tokens):
    """Tokens cut out of longer sequences, halves of wider products, odd starts,
    chunks of a modulation, gates in another order of samples and tokens."""
    t, g, how = make((3, tokens, dim), F32, BF16, pre="layer", per_sample=True)
    t["x"] = torch.cat([t["x"], t["x"]], 1)[:, 3:3 + tokens]
    t["y"] = torch.cat([t["y"], t["y"]], -1)[..., dim:]
    mod = torch.randn(3, 5 * dim, device="cuda")
    for i, k in enumerate(NAMES[2:]):
        t[k] = mod[:, i * dim:(i + 1) * dim]
    check(pkg, t, g, how)
    t["gate"] = torch.randn(tokens, 3, dim, device="cuda").to(BF16).transpose(0, 1)
    check(pkg, t, g, how)
    t["x"] = torch.randn(3 * tokens * dim + 1, device="cuda")[1:].view(3, tokens, dim)
    check(pkg, t, g, how)
    g = {"x": torch.randn(dim, device="cuda").expand(3, tokens, dim),
         "u": torch.randn(3, dim, tokens, device="cuda").to(BF16).transpose(1, 2)}
    check(pkg, t, g, how)


@pytest.mark.parametrize("dim", [8200, 9001, 12344])
@pytest.mark.parametrize("gate,post,pre", [("rows", "rms", "layer"), ("dim", None, "rms"),
                                           (None, "layer", None), ("dim", "rms", "rms")])
def test_rows_shared_by_blocks(pkg, dim, gate, post, pre):
    for pair in ((BF16, BF16), (F32, F16)):
        check(pkg, *make((2, 40, dim), *pair, gate=gate, post=post, pre=pre, bias=gate == "rows"))


@pytest.mark.parametrize("dim,tokens", [(70, 60), (1002, 40), (8202, 40)])
def test_rows_whose_alignment_changes_within_a_block(pkg, dim, tokens):
    """Slices of rows one element wider: every row of a block starts elsewhere."""
    for pair in ((F32, F32), (BF16, BF16)):
        t, g, how = make((2, tokens, dim + 1), *pair, pre="layer", gate="rows")
        for k in t:
            t[k] = t[k][..., :dim].contiguous() if t[k].dim() == 1 else t[k][..., :dim]
        check(pkg, t, {k: v[..., 1:] for k, v in g.items()}, how)


@pytest.mark.parametrize("which", ["x", "u"])
def test_one_gradient_missing(pkg, which):
    t, g, how = make((2, 9, 200), F32, BF16, post="layer", pre="layer", gate="rows")
    g[which] = None
    check(pkg, t, g, how)


def test_only_the_norm_before(pkg):
    """Without a block's output: a plain norm, with a 16-bit result of a float32 stream."""
    for kind, u_dtype in (("rms", BF16), ("layer", None), ("layer", F16)):
        t, g, how = make((2, 21, 264), post=None, pre=kind, gate=None)
        x = t["x"].clone().requires_grad_()
        w = t["pre_weight"].clone().requires_grad_()
        b = t["pre_bias"].clone().requires_grad_()
        x_out, u = pkg.fused_residual_norm(x, pre_norm=kind, pre_weight=w, pre_bias=b,
                                           u_dtype=u_dtype)
        assert x_out is x and u.dtype == (u_dtype or F32)
        gu = torch.randn(u.shape, device="cuda").to(u.dtype)
        got = torch.autograd.grad((u, x_out), (x, w, b), (gu, g["x"]))
        x6, w6, b6 = (v.detach().double().requires_grad_() for v in (x, w, b))
        _, ref_u, mid = definition({"x": x6, "y": torch.zeros_like(x6), "pre_weight": w6,
                                    "pre_bias": b6}, how)
        refs = torch.autograd.grad((ref_u, x6), (x6, w6, b6), (gu.double(), g["x"].double()))
        m = magnitudes({"x": x6.detach(), "y": torch.zeros_like(x6), "pre_weight": w6.detach(),
                        "pre_bias": b6.detach()}, {"x": g["x"].double(), "u": gu.double()}, how,
                       {k: v.detach() if torch.is_tensor(v) else v for k, v in mid.items()})
        close("u", u.detach(), ref_u.detach(), m["u"])
        for k, a, r in zip(("x", "pre_weight", "pre_bias"), got, refs):
            # the passing stream's gradient is added to the norm's in float32, after its rounding
            close("d_" + k, a, r, m["d_" + k], 2 * K)


@pytest.mark.parametrize("gate", ["dim", "rows"])
def test_autograd(pkg, gate):
    t, g, how = make((2, 33, 136), F32, BF16, post="layer", pre="rms", gate=gate, scale=0.5)
    leaves = {k: v.clone().requires_grad_() for k, v in t.items()}
    x_out, u = pkg.fused_residual_norm(leaves["x"], leaves["y"], **{k: leaves[k] for k in NAMES[2:]},
                                       **how)
    got = torch.autograd.grad((x_out, u), list(leaves.values()), (g["x"], g["u"]))
    x2, u2, stats = pkg.residual_norm_fwd(t["x"], t["y"], want_stats=True,
                                          **{k: t[k] for k in NAMES[2:]}, **how)
    direct = pkg.residual_norm_bwd(g["x"], g["u"], t["x"], t["y"], stats,
                                   **{k: t[k] for k in NAMES[2:]}, **how)
    assert torch.equal(x_out, x2) and torch.equal(u, u2)
    assert all(torch.equal(a, b) for a, b in zip(got, direct))
    # only some of them wanted, only one output used
    leaves["x"].requires_grad_(False)
    x_out, u = pkg.fused_residual_norm(leaves["x"], leaves["y"], **{k: leaves[k] for k in NAMES[2:]},
                                       **how)
    u.sum().backward()
    assert leaves["x"].grad is None and leaves["pre_bias"].grad is not None
    assert torch.allclose(leaves["pre_bias"].grad, torch.full((136,), 66.0, device="cuda"))


@pytest.mark.parametrize("post,pre,gate", [("rms", "layer", "dim"), ("layer", "rms", "rows"),
                                           (None, "layer", "dim")])
def test_gradients_by_differences(pkg, post, pre, gate):
    """dL along a direction v against (L(+h v) - L(-h v)) / 2h in float64: off by
    h^2 times a third derivative, and by float32's rounding of the gradient."""
    t, g, how = make((2, 5, 48), post=post, pre=pre, gate=gate, scale=0.75)
    _, _, stats = pkg.residual_norm_fwd(t["x"], t["y"], want_stats=True,
                                        **{k: t[k] for k in NAMES[2:] if k in t}, **how)
    grads = pkg.residual_norm_bwd(g["x"], g["u"], t["x"], t["y"], stats,
                                  **{k: t[k] for k in NAMES[2:] if k in t}, **how)
    wide = {k: v.double() for k, v in t.items()}

    def loss(moved):
        x_out, u, _ = definition(moved, how)
        return float((x_out * g["x"].double()).sum() + (u * g["u"].double()).sum())

    gen = torch.Generator().manual_seed(3)
    for name, grad in zip(NAMES, grads):
        if name not in t:
            continue
        v = torch.randn(t[name].shape, generator=gen).double().cuda()
        h = 1e-4
        up, down = (loss({**wide, name: wide[name] + s * h * v}) for s in (1, -1))
        slope = float((grad.double() * v).sum())
        size = float((grad.double() * v).abs().sum())
        assert abs(slope - (up - down) / (2 * h)) <= 1e-5 * size, name


def test_rows_without_anything(pkg):
    """Rows of zeros, and rows whose values are all equal: no deviation to divide by."""
    for post, pre in (("rms", "rms"), ("layer", "layer")):
        t, g, how = make((1, 6, 264), post=post, pre=pre)
        t["y"][0, 1] = 0.0
        t["x"][0, 2] = 0.0
        t["x"][0, 3] = 0.0
        t["y"][0, 3] = 0.0
        t["post_bias"].zero_()
        check(pkg, t, g, how)
        x_out, u, _ = pkg.residual_norm_fwd(t["x"], t["y"], **{k: t[k] for k in NAMES[2:]}, **how)
        assert torch.equal(x_out[0, 1], t["x"][0, 1])
        assert torch.equal(u[0, 3], t["pre_bias"])


@pytest.mark.parametrize("dim", [64, 515, 1152])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_one_bad_row(pkg, dim, value):
    """A NaN or an infinity reaches its own row and the sums over rows, no other row."""
    t, g, how = make((1, 12, dim), BF16, BF16, pre="layer")
    args = {k: t[k] for k in NAMES[2:]}
    good = pkg.residual_norm_fwd(t["x"], t["y"], want_stats=True, **args, **how)
    good_grads = pkg.residual_norm_bwd(g["x"], g["u"], t["x"], t["y"], good[2], **args, **how)
    t["y"][0, 5, dim // 2] = value
    x_out, u, stats = pkg.residual_norm_fwd(t["x"], t["y"], want_stats=True, **args, **how)
    grads = pkg.residual_norm_bwd(g["x"], g["u"], t["x"], t["y"], stats, **args, **how)
    others = [i for i in range(12) if i != 5]
    for a, b in ((x_out, good[0]), (u, good[1]), (grads[0], good_grads[0]), (grads[1], good_grads[1])):
        assert torch.equal(a[0, others], b[0, others])
        assert not bool(a[0, 5].isfinite().all())
    assert bool(grads[3].isnan().all())


@pytest.mark.parametrize("dim", [1152, 1001, 45])
def test_in_place_and_streams(pkg, dim):
    t, g, how = make((2, 70, dim), BF16, BF16)
    args = {k: t[k] for k in NAMES[2:]}
    x_out, u, _ = pkg.residual_norm_fwd(t["x"], t["y"], **args, **how)
    x = t["x"].clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        same, u2, _ = pkg.residual_norm_fwd(x, t["y"], x_out=x, **args, **how)
    torch.cuda.synchronize()
    assert same is x and torch.equal(x, x_out) and torch.equal(u, u2)


def test_repeats_bit_for_bit(pkg):
    t, g, how = make((4, 700, 264), BF16, BF16, per_sample=True, pre="layer")
    args = {k: t[k] for k in NAMES[2:]}
    _, _, stats = pkg.residual_norm_fwd(t["x"], t["y"], want_stats=True, **args, **how)
    first = pkg.residual_norm_bwd(g["x"], g["u"], t["x"], t["y"], stats, **args, **how)
    for _ in range(3):
        again = pkg.residual_norm_bwd(g["x"], g["u"], t["x"], t["y"], stats, **args, **how)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_in_a_graph(pkg):
    t, g, how = make((2, 64, 512), F32, BF16)
    args = {k: t[k] for k in NAMES[2:]}

    def step():
        x_out, u, stats = pkg.residual_norm_fwd(t["x"], t["y"], want_stats=True, **args, **how)
        return (x_out, u, *pkg.residual_norm_bwd(g["x"], g["u"], t["x"], t["y"], stats, **args,
                                                 **how))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    t["x"].copy_(torch.randn_like(t["x"]))
    t["y"].copy_(torch.randn_like(t["y"]))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, step()))


def test_many_rows_past_32_bits(pkg):
    """Offsets of the last rows pass 2^31 elements: checked on those rows alone."""
    rows, dim = 33_000_000, 72
    x = torch.zeros(rows, dim, dtype=BF16, device="cuda")
    y = torch.zeros(rows, dim, dtype=BF16, device="cuda")
    x[-5:] = torch.randn(5, dim, device="cuda").to(BF16)
    y[-5:] = torch.randn(5, dim, device="cuda").to(BF16)
    x_out, u, stats = pkg.residual_norm_fwd(x, y, post_norm="rms", want_stats=True)
    g = torch.zeros_like(x)
    g[-5:] = 1.0
    dx, dy = pkg.residual_norm_bwd(None, g, x, y, stats, post_norm="rms")[:2]
    tail = [v[-5:].clone() for v in (x, y)]
    a, b, st = pkg.residual_norm_fwd(*tail, post_norm="rms", want_stats=True)
    da, db = pkg.residual_norm_bwd(None, g[-5:].clone(), *tail, st, post_norm="rms")[:2]
    for big, small in ((x_out, a), (u, b), (dx, da), (dy, db)):
        assert torch.equal(big[-5:], small)


def test_more_samples_than_a_grid_dimension(pkg):
    """Parameters of 70000 samples: their gradients are 70000 groups of rows."""
    check(pkg, *make((70000, 1, 8), F32, BF16, per_sample=True))


@pytest.mark.parametrize("shape", [(300, 40, 1001), (3000, 2, 72), (2049, 1, 24), (33, 400, 7),
                                   (65, 16, 306)])
@pytest.mark.parametrize("own", [("gate",), ("post_weight", "post_bias"), ("pre_bias",)])
def test_many_samples_with_some_parameters_of_their_own(pkg, shape, own):
    """Gradients per sample and shared ones from the same sums, of many samples."""
    t, g, how = make(shape, F32, BF16, pre="layer", per_sample=True)
    for k in NAMES[2:]:
        if k not in own:
            t[k] = t[k][0].contiguous()
    check(pkg, t, g, how)


@pytest.mark.parametrize("shape", [(0, 5, 64), (2, 0, 64), (70, 0, 24)])
@pytest.mark.parametrize("own", [("gate",), ("post_weight", "pre_bias"), NAMES[2:]])
def test_no_rows_with_parameters_per_sample(pkg, shape, own):
    t, g, how = make(shape, F32, BF16, per_sample=True)
    for k in NAMES[2:]:
        if k not in own:
            t[k] = torch.ones(shape[-1], device="cuda")
    args = {k: t[k] for k in NAMES[2:]}
    stats = pkg.residual_norm_fwd(t["x"], t["y"], want_stats=True, **args, **how)[2]
    grads = pkg.residual_norm_bwd(g["x"], g["u"], t["x"], t["y"], stats, **args, **how)
    for k, v in zip(NAMES, grads):
        assert v.shape == t[k].shape and bool((v == 0).all())


@pytest.mark.parametrize("own", [("gate",), ("post_weight",), ("pre_weight", "pre_bias")])
@pytest.mark.parametrize("shape", [(5, 60, 264), (64, 3, 1001), (7, 130, 4096), (20, 40, 256)])
@pytest.mark.parametrize("par", [F16, BF16])
def test_shared_and_own_parameters_of_a_few_samples(pkg, shape, own, par):
    t, g, how = make(shape, F32, BF16, par, post="layer", per_sample=True)
    for k in NAMES[2:]:
        if k not in own:
            t[k] = t[k][0].contiguous()
    check(pkg, t, g, how)


def test_exchange_between_blocks_that_runs_out(pkg):
    """Rows of several blocks: a wait for another block's sums is bounded.  The test
    build announces more bytes than are sent: the outputs come out NaN, the device
    says so, and the next call is as ever."""
    import ctypes

    from differentiable_image_quality_gb300 import _abi

    t, g, how = make((1, 3, 9000), BF16, BF16, pre="layer")
    args = {k: t[k] for k in NAMES[2:]}

    def step():
        x_out, u, stats = pkg.residual_norm_fwd(t["x"], t["y"], want_stats=True, **args, **how)
        grads = pkg.residual_norm_bwd(g["x"], g["u"], t["x"], t["y"], stats, **args, **how)
        torch.cuda.synchronize()
        return x_out, u, *grads

    want = step()
    with _abi.using_test_library() as lib:
        flags = ctypes.c_uint()
        assert lib.gbssim_device_status(ctypes.byref(flags)) == 0 and flags.value == 0
        lib.gbssim_tune_exchange(16)
        try:
            x_out, u = pkg.residual_norm_fwd(t["x"], t["y"], **args, **how)[:2]
            torch.cuda.synchronize()
        finally:
            lib.gbssim_tune_exchange(0)
        assert bool(x_out.isnan().all()) and bool(u.isnan().all())
        assert lib.gbssim_device_status(ctypes.byref(flags)) == 0
        assert flags.value == 2  # GBSSIM_DEV_EXCHANGE_TIMEOUT
        again = step()
        assert lib.gbssim_device_status(ctypes.byref(flags)) == 0 and flags.value == 0
    assert all(torch.equal(a, b) for a, b in zip(want, again))


def test_refusals(pkg):
    t, g, how = make((2, 6, 64))
    x, y, args = t["x"], t["y"], {k: t[k] for k in NAMES[2:]}

    def bad(error, *a, **kw):
        with pytest.raises(error):
            pkg.fused_residual_norm(*a, **kw)

    bad(TypeError, x, y.cpu())
    bad(TypeError, x.double(), y.double())
    bad(TypeError, x.to(BF16), y)                      # the stream is narrower than the block
    bad(TypeError, x.to(BF16), y.to(F16))
    bad(ValueError, x, y[:, :5])
    bad(ValueError, x, y, pre_norm="batch")
    bad(ValueError, x, y, torch.zeros(63, device="cuda"))
    bad(ValueError, x, y, torch.zeros(6, 64, device="cuda"))
    bad(TypeError, x, y, torch.zeros(2, 6, 64, device="cuda", dtype=BF16))
    bad(ValueError, x, y, pre_weight=torch.zeros(128, device="cuda")[::2])
    bad(ValueError, x.transpose(1, 2), y.transpose(1, 2))  # columns apart
    bad(ValueError, torch.zeros((), device="cuda"), torch.zeros((), device="cuda"))
    wide = torch.zeros(1, 16385, device="cuda")
    bad(ValueError, wide, wide)
    bad(ValueError, x, None, torch.ones(64, device="cuda"))
    bad(ValueError, x, None, post_norm="rms")
    bad(ValueError, x, None, residual_scale=0.5)
    bad(ValueError, x, y, u_dtype=BF16)
    bad(ValueError, x, None, pre_norm=None)
    with pytest.raises(pkg.GbssimError):
        pkg.residual_norm_fwd(x, y, eps=-1.0)
    with pytest.raises(pkg.GbssimError):
        pkg.residual_norm_fwd(x, y, x_out=y)
    stats = pkg.residual_norm_fwd(x, y, want_stats=True)[2]
    with pytest.raises(ValueError):
        pkg.residual_norm_bwd(None, None, x, y, stats)
    with pytest.raises(ValueError):
        pkg.residual_norm_bwd(g["x"], None, x, y, stats[:1])
    with pytest.raises(ValueError):
        pkg.residual_norm_bwd(g["x"].to(BF16), None, x, y, stats)


def without(t, names):
    """The inputs with these parameters left out, and y's mean twice its deviation."""
    t = {k: v for k, v in t.items() if k not in names}
    t["y"] = (t["y"].float() + 1.6).to(t["y"].dtype)
    return t


@pytest.mark.parametrize("post,pre", list(itertools.product([None, "rms", "layer"], repeat=2)))
@pytest.mark.parametrize("gate", [None, "dim", "rows"])
@pytest.mark.parametrize("names", [("post_weight",), ("pre_weight",), ("post_weight", "pre_weight"),
                                   NAMES[3:]], ids=str)
def test_norms_without_weights(pkg, post, pre, gate, names):
    """A weight that is left out is one in the row's columns, and nothing beside them."""
    for dim in (72, 515):
        t, g, how = make((2, 9, dim), F32, BF16, post=post, pre=pre, gate=gate, scale=0.5)
        check(pkg, without(t, names), g, how)


@pytest.mark.parametrize("dim", DIMS + [960, 1408, 2880])
@pytest.mark.parametrize("pair", [(F32, F32), (BF16, BF16), (F32, F16)], ids=str)
@pytest.mark.parametrize("post,pre", [("layer", "rms"), ("layer", "layer"), ("rms", "layer")])
def test_widths_without_parameters(pkg, dim, pair, post, pre):
    t, g, how = make((2, 7, dim), *pair, post=post, pre=pre, seed=dim)
    check(pkg, without(t, NAMES[2:]), g, how)


@pytest.mark.parametrize("dim", [8200, 9001, 12344])
@pytest.mark.parametrize("gate", [None, "dim", "rows"])
def test_rows_shared_by_blocks_without_weights(pkg, dim, gate):
    for post, pre in (("layer", "rms"), ("layer", "layer"), ("rms", "layer")):
        t, g, how = make((2, 40, dim), BF16, BF16, gate=gate, post=post, pre=pre)
        check(pkg, without(t, NAMES[3:]), g, how)


@pytest.mark.parametrize("shape", [(5, 1, 128), (1, 1, 72), (3, 1, 1, 72), (2, 1, 1001)], ids=str)
@pytest.mark.parametrize("pair", [(F32, BF16), (BF16, BF16), (F16, F16)], ids=str)
def test_gate_of_each_sample_beside_one_token(pkg, shape, pair):
    """A gate [samples, 1, dim] has a type of its own however many tokens there are,
    and may be a chunk of something wider."""
    for tokens in (1, 2):
        wide = (shape[0], tokens, *shape[2:])
        t, g, how = make(wide, *pair, pre="layer")
        mod = torch.randn(*shape[:-1], 3 * shape[-1], device="cuda")
        t["gate"] = mod[..., shape[-1]:2 * shape[-1]]
        check(pkg, t, g, how)
    leaves = {k: v.detach().clone().requires_grad_() for k, v in t.items()}
    x_out, u = pkg.fused_residual_norm(leaves["x"], leaves["y"],
                                       **{k: leaves[k] for k in NAMES[2:]}, **how)
    torch.autograd.backward((x_out, u), (g["x"], g["u"]))
    assert leaves["gate"].grad.shape == shape and leaves["gate"].grad.dtype == F32


def test_given_output_counts_as_written(pkg):
    """Autograd refuses a backward through what an output has overwritten."""
    t, g, how = make((2, 9, 72))
    args = {k: t[k] for k in NAMES[2:]}
    for x_out in (torch.empty_like(t["x"]), t["x"].clone().view(18, 72).view(2, 9, 72)):
        version = x_out._version
        pkg.residual_norm_fwd(t["x"], t["y"], x_out=x_out, **args, **how)
        assert x_out._version > version
    x, w = t["x"].clone(), torch.ones(72, device="cuda", requires_grad=True)
    saved = (x * w).sum()
    pkg.residual_norm_fwd(x, t["y"], x_out=x.view(x.shape), **args, **how)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        saved.backward()
    with torch.inference_mode():
        buffer = torch.empty_like(x)
    pkg.residual_norm_fwd(x, t["y"], x_out=buffer, **args, **how)


def test_no_samples_by_the_c_interface(pkg):
    """Without samples, gradients that samples have of their own are empty, wherever
    they were to be written: nothing to do, and shared ones are zero."""
    from differentiable_image_quality_gb300 import _abi, _residual_norm as rn

    lib = _abi.load()
    own = torch.ones(64, device="cuda")
    shared = torch.ones(64, device="cuda")
    out = [torch.full((64,), 7.0, device="cuda") for _ in range(2)]
    none, at = (0, 0, 0), (shared.data_ptr(), 0, 64)
    for tokens in (0, 5):
        for wants_shared in (False, True):
            desc = rn._DESC.pack(0, tokens, 64, 0, 0, 1, 1, 1.0, 0.0, 1e-6, *at, *at, *none,
                                 0, 0, 0, 0, own.data_ptr(), 0, 1, 64, 0, 0, 0, 0,
                                 shared.data_ptr(), 0, 0, 0, 0, 0, 0, 0)
            grads = rn._GRADS.pack(0, 0, 0, out[0].data_ptr(), 0,
                                   out[1].data_ptr() if wants_shared else 0, 0)
            st = lib.gbssim_residual_norm_bwd(desc, None, None, None, grads, None, 0,
                                              torch.cuda.current_stream().cuda_stream)
            assert st == 0, (tokens, wants_shared)
            torch.cuda.synchronize()
            assert bool((out[0] == 7.0).all())
    assert bool((out[1] == 0.0).all())


def test_parameter_without_dimensions(pkg):
    t, g, how = make((2, 6, 64))
    for name in NAMES[3:]:
        with pytest.raises(ValueError, match=name):
            pkg.fused_residual_norm(t["x"], t["y"], **{name: torch.ones((), device="cuda")})
    with pytest.raises(ValueError, match="gate"):
        pkg.fused_residual_norm(t["x"], t["y"], torch.ones((), device="cuda"))
