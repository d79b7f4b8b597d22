"""Cases of the training-step operators beside the SSIM loss: the global gradient
norm and clipping over many tensors, and the norms around a residual block fused
with its gate and residual scale (forward, backward, and both under autograd).

With ``own`` false, run() evaluates the operators from elementary torch
operations in float32; with ``own`` true it calls the package.
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


def _tensors(op, tensors, total, grads, layout, max_norm=1.0, out="f32"):
    return {"op": op, "tensors": tensors, "total": total, "grads": grads, "layout": layout,
            "max_norm": max_norm, "out": out}


def _rows(op, batch, tokens, dim, res, blk, par, post, pre, bias, gate, scale=1.0, offset=0.0,
          view="whole"):
    return {"op": op, "batch": batch, "tokens": tokens, "dim": dim, "res": res, "blk": blk,
            "par": par, "post": post, "pre": pre, "bias": bias, "gate": gate, "scale": scale,
            "offset": offset, "view": view}


def listed():
    return [
        # a small convolutional denoiser on 64 x 64 crops: what counts is the call's own time
        dict(_tensors("norm", 26, 241_331, "f32", "apart"), name="norm denoiser f32"),
        # a large transformer, gradients in the buckets a data-parallel run keeps them in
        dict(_tensors("norm", 291, 1_003_520_017, "bf16", "packed"), name="norm transformer bf16"),
        # a splat model of a million Gaussians: means, scales, rotations, opacities, colours
        dict(_tensors("clip", 6, 59_000_000, "f32", "apart"), name="clip splats f32"),
        # 16- and 32-bit gradients clipped into 32-bit main gradients
        dict(_tensors("clip", 148, 123_456_789, "mixed", "packed"), name="clip mixed into f32"),
        # serving: one token through a sandwich of root-mean-square norms
        dict(_rows("forward", 1, 1, 4096, "bf16", "bf16", "bf16", "rms", "rms", False, "none"),
             name="forward one token bf16"),
        # eight 512 x 512 images in 16 x 16 patches, conditioned per image (gate, scale, shift)
        dict(_rows("forward", 8, 1024, 1152, "f32", "bf16", "bf16", "none", "layer", True,
                   "sample", 1.0, 1.0), name="forward conditioned 8x1024x1152"),
        # a long prefill, with learned gates
        dict(_rows("forward", 1, 65536, 4096, "bf16", "bf16", "f32", "rms", "rms", False, "dim"),
             name="forward 65536x4096 bf16"),
        # crops of 64 x 64 in patches of 8: a small model's backward
        dict(_rows("backward", 1, 64, 768, "f32", "f32", "f32", "layer", "layer", True, "dim"),
             name="backward 64x768 f32"),
        # a 1080 x 1920 image in patches of 8, an odd width, the block's output one half of a
        # wider product, residual scaled
        dict(_rows("backward", 1, 32400, 1001, "f16", "f16", "f32", "layer", "rms", True, "dim",
                   0.5, 0.0, "half"), name="backward 32400x1001 f16"),
        # the largest: every gate value its own, 16-bit throughout
        dict(_rows("backward", 2, 16200, 4096, "bf16", "bf16", "bf16", "rms", "rms", False,
                   "full", 1.0, 1.0), name="backward 2x16200x4096 bf16"),
        # the conditioned block under autograd, forward and backward
        dict(_rows("train", 8, 1024, 1152, "f32", "bf16", "bf16", "none", "layer", True, "sample",
                   1.0, 1.0), name="train conditioned 8x1024x1152"),
        # the sandwich under autograd
        dict(_rows("train", 4, 4096, 2048, "bf16", "bf16", "f32", "rms", "rms", False, "dim",
                   0.75), name="train sandwich 4x4096x2048"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "clip", "forward", "backward", "train"])
    if op in ("norm", "clip"):
        tensors = _log_int(rng, 1, 400)
        total = _log_int(rng, 20 * tensors + 1000, 200_000_000)
        return _tensors(op, tensors, total, rng.choice(["f32", "bf16", "f16", "mixed"]),
                        rng.choice(["apart", "packed"]), rng.choice([0.1, 1.0, 10.0]),
                        rng.choice(["f32", "same"]))
    # widths from small heads to wide models: whole vectors of 8, or any number
    dim = _log_int(rng, 32, 16384)
    if rng.random() < 0.6:
        dim = max(8, dim // 8 * 8)
    if dim == 3072:
        dim = 3080
    rows = _log_int(rng, 1, min(100_000, 120_000_000 // dim))
    batch = min(rows, rng.choice([1, 1, 2, 3, 8]))
    tokens = rows // batch
    res, blk = rng.choice([("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("f32", "bf16"),
                           ("f32", "f16")])
    return _rows(op, batch, tokens, dim, res, blk, rng.choice(["f32", blk]),
                 rng.choice(["none", "rms", "layer"]), rng.choice(["rms", "layer"]),
                 rng.random() < 0.5, rng.choice(["none", "dim", "sample", "full"]),
                 rng.choice([1.0, 0.5]), rng.choice([0.0, 1.0]), rng.choice(["whole", "half"]))


# ------------------------------------------------------------------ inputs

def _sizes(case):
    """Element counts of the case's tensors: weights spread over three decades,
    one tensor of a single element where there are several."""
    n, total = case["tensors"], case["total"]
    rng = random.Random(1_000_003 * n + total)
    w = [10.0 ** rng.uniform(0.0, 3.0) for _ in range(n)]
    s = sum(w)
    sizes = [max(1, int(x / s * total)) for x in w]
    if n > 2:
        sizes[n // 2] = 1
    sizes[0] += max(0, total - sum(sizes))
    return sizes


def _types(case):
    kinds = {"mixed": ["bf16", "f32", "f16"]}.get(case["grads"], [case["grads"]])
    return [TYPES[kinds[i % len(kinds)]] for i in range(case["tensors"])]


def _lay_out(sizes, types, layout, device):
    """Empty tensors, and per type the buffer that holds them: one behind the other
    ("packed"), or each from a 256-byte boundary as separate allocations are."""
    flat, views, at = {}, [None] * len(sizes), {}
    starts = []
    for n, t in zip(sizes, types):
        starts.append(at.get(t, 0))
        step = n if layout == "packed" else (n + 127) // 128 * 128
        at[t] = at.get(t, 0) + step
    for t, n in at.items():
        flat[t] = torch.zeros(n, dtype=t, device=device)
    for i, (n, t) in enumerate(zip(sizes, types)):
        views[i] = flat[t][starts[i]:starts[i] + n]
    return flat, views


def _prepare_tensors(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    sizes, types = _sizes(case), _types(case)
    flat, grads = _lay_out(sizes, types, case["layout"], dev)
    for g in grads:
        # per tensor its own scale, and one element in eight without a gradient
        scale = 1e-3 * 2.0 ** (6.0 * torch.rand((), generator=gen, device=dev) - 3.0)
        v = torch.randn(g.numel(), generator=gen, device=dev) * scale
        v *= torch.rand(g.numel(), generator=gen, device=dev) > 0.125
        g.copy_(v)
    state = {"case": case, "grads": grads}
    if case["op"] == "clip":
        out_types = types if case["out"] == "same" else [torch.float32] * len(types)
        state["flat_out"], state["out"] = _lay_out(sizes, out_types, case["layout"], dev)
        state["flat_out"] = [state["flat_out"][t] for t in TYPES.values()
                             if t in state["flat_out"]]
    return state


def _prepare_rows(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    B, T, D = case["batch"], case["tokens"], case["dim"]
    res, blk, par = TYPES[case["res"]], TYPES[case["blk"]], TYPES[case["par"]]

    def normal(shape, std, mean=0.0, dtype=torch.float32):
        return (torch.randn(shape, generator=gen, device=dev) * std + mean).to(dtype)

    # a residual stream with a few loud channels, as deep models have
    loud = 1.0 + 9.0 * (torch.rand(D, generator=gen, device=dev) < 0.01)
    x = (torch.randn((B, T, D), generator=gen, device=dev) * loud + 0.1).to(res)
    if case["view"] == "half":
        y = normal((B, T, 2 * D), 0.7, 0.05, blk)[..., :D]
    else:
        y = normal((B, T, D), 0.7, 0.05, blk)
    # conditioned norms have their parameters per sample
    shape = (B, D) if case["gate"] == "sample" else (D,)
    mean = 1.0 - case["offset"]
    a = {"gate": None, "post_weight": None, "post_bias": None}
    if case["gate"] != "none":
        a["gate"] = normal((B, T, D) if case["gate"] == "full" else shape, 0.2, 0.5,
                           blk if case["gate"] == "full" else par)
    if case["post"] != "none":
        a["post_weight"] = normal((D,), 0.1, mean, par)
        if case["bias"]:
            a["post_bias"] = normal((D,), 0.1, 0.0, par)
    a["pre_weight"] = normal(shape, 0.1, mean, par)
    a["pre_bias"] = normal(shape, 0.1, 0.0, par) if case["bias"] else None
    state = {"case": case, "x": x, "y": y, "args": a}
    if case["op"] != "forward":
        state["g_x"] = normal((B, T, D), 0.5, 0.0, res)
        state["g_u"] = normal((B, T, D), 0.5, 0.0, blk)
    if case["op"] == "backward":
        # what the forward leaves for the backward: mean and 1/deviation of each row
        state["stats"] = _forward(state)[2]
    if case["op"] == "train":
        for t in [x, y, *a.values()]:
            if t is not None:
                t.requires_grad_(True)
    return state


def prepare(case, seed):
    if case["op"] in ("norm", "clip"):
        return _prepare_tensors(case, seed)
    return _prepare_rows(case, seed)


# ------------------------------------------------------- the plain forms, in float32

def _per_row(p):
    """[D] and [B, T, D] as they are, [B, D] over the tokens."""
    if p is None:
        return None
    p = p.detach().float()
    return p[:, None, :] if p.dim() == 2 else p


def _statistics(v, kind):
    if kind == "none":
        one = torch.ones_like(v[..., :1])
        return torch.zeros_like(one), one
    mean = v.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(v[..., :1])
    return mean, 1.0 / torch.sqrt(((v - mean) ** 2).mean(-1, keepdim=True) + EPS)


def _forward(state):
    case = state["case"]
    p = {k: _per_row(v) for k, v in state["args"].items()}
    x, y = state["x"].detach().float(), state["y"].detach().float()
    mean1, rstd1 = _statistics(y, case["post"])
    z = (y - mean1) * rstd1
    if p["post_weight"] is not None:
        z = z * (p["post_weight"] + case["offset"])
    if p["post_bias"] is not None:
        z = z + p["post_bias"]
    if p["gate"] is not None:
        z = z * p["gate"]
    x_out = case["scale"] * x + z
    mean2, rstd2 = _statistics(x_out, case["pre"])
    u = (x_out - mean2) * rstd2 * (p["pre_weight"] + case["offset"])
    if p["pre_bias"] is not None:
        u = u + p["pre_bias"]
    stats = torch.cat([mean1, rstd1, mean2, rstd2], -1)
    return x_out, u, stats


def _to_shape(grad, param):
    """A gradient over all rows, summed to the shape of what it belongs to."""
    if param.dim() == 1:
        return grad.sum((0, 1)).to(param.dtype)
    return (grad.sum(1) if param.dim() == 2 else grad).to(param.dtype)


def _backward(state):
    case, args = state["case"], state["args"]
    p = {k: _per_row(v) for k, v in args.items()}
    x, y = state["x"].detach().float(), state["y"].detach().float()
    g_x, g_u = state["g_x"].float(), state["g_u"].float()
    mean1, rstd1 = _statistics(y, case["post"])
    yh = (y - mean1) * rstd1
    w1 = p["post_weight"] + case["offset"] if p["post_weight"] is not None else None
    z = yh if w1 is None else yh * w1
    z = z if p["post_bias"] is None else z + p["post_bias"]
    x_out = case["scale"] * x + (z if p["gate"] is None else z * p["gate"])
    mean2, rstd2 = _statistics(x_out, case["pre"])
    xh = (x_out - mean2) * rstd2
    out = {"pre_weight": _to_shape(g_u * xh, args["pre_weight"])}
    if args["pre_bias"] is not None:
        out["pre_bias"] = _to_shape(g_u, args["pre_bias"])
    dxh = g_u * (p["pre_weight"] + case["offset"])
    t = dxh - xh * (dxh * xh).mean(-1, keepdim=True)
    if case["pre"] == "layer":
        t = t - dxh.mean(-1, keepdim=True)
    t = g_x + rstd2 * t
    out["x"] = (case["scale"] * t).to(state["x"].dtype)
    if args["gate"] is not None:
        out["gate"] = _to_shape(t * z, args["gate"])
        t = t * p["gate"]
    if args["post_bias"] is not None:
        out["post_bias"] = _to_shape(t, args["post_bias"])
    if w1 is not None:
        out["post_weight"] = _to_shape(t * yh, args["post_weight"])
        t = t * w1
    if case["post"] != "none":
        d = t - yh * (t * yh).mean(-1, keepdim=True)
        if case["post"] == "layer":
            d = d - t.mean(-1, keepdim=True)
        t = rstd1 * d
    out["y"] = t.to(state["y"].dtype)
    return out


def _plain(state):
    case = state["case"]
    if case["op"] in ("norm", "clip"):
        grads = state["grads"]
        norm = torch.stack([(g.float() * g.float()).sum() for g in grads]).sum().sqrt()
        if case["op"] == "norm":
            return norm
        coef = torch.clamp(case["max_norm"] / (norm + 1e-6), max=1.0)
        torch._foreach_copy_(state["out"], [g.float() * coef for g in grads])
        return {"norm": norm, "out": state["flat_out"]}
    if case["op"] == "backward":
        return _backward(state)
    x_out, u, _ = _forward(state)
    out = {"x_out": x_out.to(state["x"].dtype), "u": u.to(state["y"].dtype)}
    if case["op"] == "train":
        out["grads"] = _backward(state)
    return out


# ------------------------------------------------------------ the package's calls

_NAMES = ("x", "y", "gate", "post_weight", "post_bias", "pre_weight", "pre_bias")


def _own(state):
    import differentiable_image_quality_gb300 as pkg

    case = state["case"]
    if case["op"] == "norm":
        return pkg.grad_norm(state["grads"])
    if case["op"] == "clip":
        norm = pkg.clip_grads(state["grads"], case["max_norm"], out=state["out"])
        return {"norm": norm, "out": state["flat_out"]}
    how = {"post_norm": None if case["post"] == "none" else case["post"], "pre_norm": case["pre"],
           "residual_scale": case["scale"], "weight_offset": case["offset"], "eps": EPS}
    x, y, args = state["x"], state["y"], state["args"]
    if case["op"] == "forward":
        x_out, u, _ = pkg.residual_norm_fwd(x, y, **args, **how)
        return {"x_out": x_out, "u": u}
    if case["op"] == "backward":
        grads = pkg.residual_norm_bwd(state["g_x"], state["g_u"], x, y, state["stats"], **args,
                                      **how)
        return {k: g for k, g in zip(_NAMES, grads) if g is not None}
    x_out, u = pkg.fused_residual_norm(x, y, **args, **how)
    wanted = [(k, t) for k, t in zip(_NAMES, [x, y] + [args[n] for n in _NAMES[2:]])
              if t is not None]
    grads = torch.autograd.grad((x_out, u), [t for _, t in wanted], (state["g_x"], state["g_u"]))
    return {"x_out": x_out.detach(), "u": u.detach(),
            "grads": {k: g for (k, _), g in zip(wanted, grads)}}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------ the least a pass costs

_BYTES = {torch.float32: 4, torch.bfloat16: 2, torch.float16: 2}


def work(case):
    if case["op"] in ("norm", "clip"):
        sizes, types = _sizes(case), _types(case)
        read = sum(n * _BYTES[t] for n, t in zip(sizes, types))
        if case["op"] == "norm":
            return {"bytes": read + 4, "flops": 2 * sum(sizes)}
        write = read if case["out"] == "same" else 4 * sum(sizes)
        return {"bytes": read + write + 4, "flops": 3 * sum(sizes)}
    rows = case["batch"] * case["tokens"]
    n = rows * case["dim"]
    res, blk, par = (_BYTES[TYPES[case[k]]] for k in ("res", "blk", "par"))
    per = case["dim"] * par * (case["batch"] if case["gate"] == "sample" else 1)
    params = per * (2 if case["bias"] else 1)
    if case["post"] != "none":
        params += case["dim"] * par * (2 if case["bias"] else 1)
    if case["gate"] == "full":
        params += n * blk
    elif case["gate"] != "none":
        params += per
    forward, backward = 2 * n * (res + blk) + params, 3 * n * (res + blk) + 2 * params + 16 * rows
    if case["op"] == "forward":
        return {"bytes": forward, "flops": 20 * n}
    if case["op"] == "backward":
        return {"bytes": backward, "flops": 45 * n}
    return {"bytes": 4 * n * (res + blk) + 2 * params, "flops": 65 * n}


# ------------------------------------------------------------ in 64 bits, by definition

def _norm64(v, kind, weight, bias, offset):
    if kind == "layer":
        v = v - v.sum(-1, keepdim=True) / v.shape[-1]
    if kind != "none":
        v = v / (v.square().sum(-1, keepdim=True) / v.shape[-1] + EPS).sqrt()
    if weight is not None:
        v = v * (weight.unsqueeze(1) if weight.dim() == 2 else weight).add(offset)
    if bias is not None:
        v = v + (bias.unsqueeze(1) if bias.dim() == 2 else bias)
    return v


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] in ("norm", "clip"):
        total = math.sqrt(math.fsum(float(g.double().square().sum()) for g in state["grads"]))
        norm = torch.tensor(total, dtype=torch.float64)
        if case["op"] == "norm":
            return norm
        coef = min(1.0, case["max_norm"] / (total + 1e-6))
        wide = {b.dtype: torch.zeros(b.numel(), dtype=torch.float64, device=b.device)
                for b in state["flat_out"]}
        at = {b.dtype: b.data_ptr() for b in state["flat_out"]}
        for g, o in zip(state["grads"], state["out"]):
            first = (o.data_ptr() - at[o.dtype]) // o.element_size()
            wide[o.dtype][first:first + o.numel()] = g.double() * coef
        return {"norm": norm, "out": [wide[b.dtype] for b in state["flat_out"]]}
    # the gradients by differentiating the definition, not by the backward's formulas
    wants = case["op"] != "forward"
    wide = {k: state["args"][k].detach().double().requires_grad_(wants)
            for k in _NAMES[2:] if state["args"][k] is not None}
    x = state["x"].detach().double().requires_grad_(wants)
    y = state["y"].detach().double().requires_grad_(wants)
    z = _norm64(y, case["post"], wide.get("post_weight"), wide.get("post_bias"), case["offset"])
    if "gate" in wide:
        z = z * (wide["gate"].unsqueeze(1) if wide["gate"].dim() == 2 else wide["gate"])
    x_out = x * case["scale"] + z
    u = _norm64(x_out, case["pre"], wide["pre_weight"], wide.get("pre_bias"), case["offset"])
    out = {"x_out": x_out.detach(), "u": u.detach()}
    if not wants:
        return out
    asked = {"x": x, "y": y, **wide}
    got = torch.autograd.grad((x_out, u), list(asked.values()),
                              (state["g_x"].double(), state["g_u"].double()))
    grads = dict(zip(asked, got))
    return grads if case["op"] == "backward" else dict(out, grads=grads)
