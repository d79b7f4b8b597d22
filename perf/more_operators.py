"""Cases of the operators between the tokens of a transformer block: rotary
positions with several axes, attention (forward, one token against a long cache
included), attention's backward, and both under autograd.

With ``own`` false, run() evaluates the operators from elementary torch
operations in float32, each operator's outputs rounded once (angles in float64,
where far positions need it); with ``own`` true it calls the package.
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BASE = 10000.0


def _rotary(op, batch, tokens, heads, kv_heads, dim, pairs, dtype, layout="half",
            positions="int", far=False, view="whole"):
    return {"op": op, "batch": batch, "tokens": tokens, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "pairs": pairs, "type": dtype, "layout": layout, "positions": positions,
            "far": far, "view": view}


def _attention(op, batch, q, k, heads, kv_heads, dim, dtype, causal=False, ragged="none",
               view="whole", pairs=""):
    return {"op": op, "batch": batch, "q": q, "k": k, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "type": dtype, "causal": causal, "ragged": ragged, "view": view,
            "pairs": pairs}


def listed():
    return [
        # a small denoiser on 64 x 64 crops in patches of 8: what counts is the call's own time
        dict(_rotary("rotary", 8, 64, 8, 8, 32, "8,8", "bf16"), name="rotary 8x64 tokens bf16"),
        # sixteen frames of 512 x 512 in patches of 8: time, height, width; shared key heads,
        # q and k as they lie in one product
        dict(_rotary("rotary", 1, 65536, 16, 4, 128, "16,24,24", "bf16", "half", "int", True,
                     "product"), name="rotary video 65536 tokens bf16"),
        # gradients of a 1080 x 1920 image in patches of 8, positions at fractions of the
        # training size's, neighbouring pairs, eight columns of a head without a position
        dict(_rotary("inverse", 1, 32400, 12, 12, 88, "20,20", "f32", "adjacent", "float"),
             name="rotary gradient 32400 tokens f32"),
        # the small denoiser's attention
        dict(_attention("forward", 8, 64, 64, 8, 8, 32, "bf16"), name="forward 8x64 bf16"),
        # one token of a model that writes its image patch by patch, 65536 patches written
        dict(_attention("forward", 1, 1, 65536, 32, 8, 128, "bf16", True),
             name="forward one token over 65536 bf16"),
        # eight 512 x 512 images in 16 x 16 patches
        dict(_attention("forward", 8, 1024, 1024, 16, 16, 72, "f16", False, "none", "product"),
             name="forward 8x1024 f16"),
        # a long prompt
        dict(_attention("forward", 1, 16384, 16384, 16, 4, 128, "bf16", True),
             name="forward causal 16384 bf16"),
        # crops of 64 x 64
        dict(_attention("backward", 8, 64, 64, 8, 8, 32, "bf16"), name="backward 8x64 bf16"),
        # images of many sizes one behind the other
        dict(_attention("backward", 24, 1500, 1500, 16, 16, 64, "f16", False, "packed"),
             name="backward packed 24 images f16"),
        # the largest: two long sequences, shared key heads
        dict(_attention("backward", 2, 8192, 8192, 16, 4, 128, "bf16", True),
             name="backward causal 2x8192 bf16"),
        # a conditioned block's positions and attention under autograd
        dict(_attention("train", 8, 1024, 1024, 16, 16, 72, "bf16", False, "none", "product",
                        "18,18"), name="train 8x1024 bf16"),
        # patches that attend to a padded batch of reference tokens
        dict(_attention("train", 4, 4096, 2333, 16, 8, 128, "bf16", False, "lengths", "whole",
                        "16,24,24"), name="train across 4x4096x2333 bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _pairs(rng, dim):
    """How many pairs each of one to three axes turns; what is left of a head stays."""
    axes = rng.choice([1, 2, 2, 3])
    most = dim // 2 // axes
    n = [max(1, rng.choice([most, most, most - 1, most // 2])) for _ in range(axes)]
    return ",".join(str(v) for v in n)


def draw(rng):
    op = rng.choice(["rotary", "inverse", "forward", "forward", "backward", "backward", "train"])
    dim = rng.choice([16, 32, 40, 64, 64, 72, 80, 96, 128, 128, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 8, 8])
    heads = kv_heads * rng.choice([1, 1, 2, 3, 4, 8] if kv_heads < 8 else [1, 1, 2, 4])
    view = rng.choice(["whole", "product"])
    batch = rng.choice([1, 1, 2, 3, 8])
    if op in ("rotary", "inverse"):
        most = 160_000_000 // ((heads + kv_heads) * dim * batch)
        return _rotary(op, batch, _log_int(rng, 1, min(100_000, most)), heads, kv_heads, dim,
                       _pairs(rng, dim), rng.choice(["f32", "bf16", "f16"]),
                       rng.choice(["half", "adjacent"]), rng.choice(["int", "int", "float"]),
                       rng.random() < 0.3, view)
    ragged = rng.choice(["none", "none", "lengths", "packed"])
    if ragged != "none":
        batch = rng.choice([2, 5, 16])
    scores = (4.2e9 if op == "forward" else 2.1e9) / (batch * heads)
    k = _log_int(rng, 1, min(16384, int(math.sqrt(scores))))
    q = k
    if ragged != "packed" and rng.random() < 0.4:
        # another number of queries: few beside what was kept, or another picture's
        q = rng.choice([1, 1, 7, _log_int(rng, 1, min(16384, int(math.sqrt(scores))))])
        if op == "forward" and q <= 7:
            k = _log_int(rng, 1, 131_072 // batch)
    return _attention(op, batch, q, k, heads, kv_heads, dim, rng.choice(["bf16", "bf16", "f16"]),
                      rng.random() < 0.5, ragged, view if q == k else "whole",
                      _pairs(rng, dim) if op == "train" else "")


# ------------------------------------------------------------------ inputs

def _lengths(case):
    """Per sequence how many keys it has, by the case alone: log-spread, and one sequence
    without any where there are enough."""
    n, most = case["batch"], case["k"]
    rng = random.Random(1_000_003 * n + most)
    out = [_log_int(rng, max(1, most // 8), most) for _ in range(n)]
    out[rng.randrange(n)] = most
    if n > 4:
        out[n // 2] = 0
    return out


def _sequences(case):
    """(queries, keys) of every sequence."""
    if case["ragged"] == "none":
        return [(case["q"], case["k"])] * case["batch"]
    if case["ragged"] == "lengths":
        return [(case["q"], n) for n in _lengths(case)]
    return [(n, n) for n in _lengths(case)]


TAIL = 5  # rows of a packed batch behind its last sequence


def _grid_positions(axes, tokens, far, fractions, gen, dev):
    """Coordinates of a picture's or a film's patches, from a corner that the seed sets."""
    side = max(1, round(tokens ** (1.0 / axes)))
    i = torch.arange(tokens, device=dev)
    pos = torch.stack([i // side ** a % side if a < axes - 1 else i // side ** a
                       for a in reversed(range(axes))], -1)
    corner = torch.randint(0, 1_000_000 if far else 64, (axes,), generator=gen, device=dev)
    pos = pos + corner
    return (pos * 0.375 + 0.125).float() if fractions else pos


def _heads(case, shape, counts, gen, dev, std=1.0):
    """One tensor [*shape, n, dim] for each n: apart, or side by side in one product."""
    dim, dtype = case["dim"], TYPES[case["type"]]

    def normal(width):
        return (torch.randn((*shape, width), generator=gen, device=dev) * std).to(dtype)

    if case["view"] == "product":
        parts = normal(sum(counts) * dim).split([n * dim for n in counts], -1)
    else:
        parts = [normal(n * dim) for n in counts]
    return [p.unflatten(-1, (n, dim)) for p, n in zip(parts, counts)]


def _frequencies(pairs, dev):
    """Per axis base^(-i / n) for its n pairs, in float64."""
    return torch.cat([BASE ** (-torch.arange(n, dtype=torch.float64, device=dev) / n)
                      for n in pairs])


def _split(pairs):
    return [int(n) for n in pairs.split(",")]


def _prepare_rotary(case, gen, dev):
    pairs = _split(case["pairs"])
    q, k = _heads(case, (case["batch"], case["tokens"]), [case["heads"], case["kv_heads"]], gen,
                  dev)
    pos = _grid_positions(len(pairs), case["tokens"], case["far"], case["positions"] == "float",
                          gen, dev)
    return {"case": case, "q": q, "k": k, "positions": pos, "pairs": pairs,
            "frequencies": _frequencies(pairs, dev)}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    if case["op"] in ("rotary", "inverse"):
        return _prepare_rotary(case, gen, dev)
    H, K, B = case["heads"], case["kv_heads"], case["batch"]
    state = {"case": case, "scale": case["dim"] ** -0.5, "kv_lengths": None, "offsets": None}
    if case["ragged"] == "packed":
        n = _lengths(case)
        ends = [sum(n[:i]) for i in range(B + 1)]
        state["offsets"] = torch.tensor(ends, dtype=torch.int32, device=dev)
        shape_q = shape_k = (ends[-1] + TAIL,)
    else:
        shape_q, shape_k = (B, case["q"]), (B, case["k"])
        if case["ragged"] == "lengths":
            state["kv_lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device=dev)
    if shape_q == shape_k:
        q, k, v = _heads(case, shape_q, [H, K, K], gen, dev)
    else:
        q, = _heads(case, shape_q, [H], gen, dev)
        k, v = _heads(case, shape_k, [K, K], gen, dev)
    # an eighth of a head's columns louder than the others, so that scores spread as trained
    # models' do
    k[..., :case["dim"] // 8] *= 2.0
    state.update(q=q, k=k, v=v)
    if case["op"] != "forward":
        state["g"] = (torch.randn(q.shape, generator=gen, device=dev) * 0.1).to(q.dtype)
    if case["op"] == "backward":
        # what the forward leaves for the backward: its output and each row's log-sum
        out, state["lse"] = _attend(state, q, k, v)
        state["out"] = out.to(q.dtype)
    if case["op"] == "train":
        state["pairs"] = _split(case["pairs"])
        state["frequencies"] = _frequencies(state["pairs"], dev)
        axes = len(state["pairs"])
        state["positions"] = _grid_positions(axes, shape_q[-1], False, False, gen, dev)
        state["k_positions"] = state["positions"] if case["q"] == case["k"] else \
            _grid_positions(axes, shape_k[-1], False, False, gen, dev)
        state["leaves"] = [t.detach().requires_grad_(True) for t in (q, k, v)]
    return state


# ------------------------------------------------------- the plain forms, in float32

def _turn(x, positions, frequencies, pairs, layout, inverse):
    """x [..., tokens, heads, dim] turned by its tokens' positions; float32, not rounded."""
    axis = torch.repeat_interleave(torch.arange(len(pairs), device=x.device),
                                   torch.tensor(pairs, device=x.device),
                                   output_size=sum(pairs))
    angle = (positions.double()[..., axis] * frequencies)[..., None, :]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    sin = -sin if inverse else sin
    n = sum(pairs)
    x = x.float()
    if layout == "half":
        a, b = x[..., :n], x[..., n:2 * n]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([turned, x[..., 2 * n:]], -1)


def _padded(state, t):
    """A packed tensor's sequences as the samples of a batch; others as they are."""
    if state["offsets"] is None:
        return t
    at, _ = _places(state)
    return t[at]


def _places(state):
    """Per sequence and token the row of the packed tensors, and whether there is one."""
    start, n = state["offsets"][:-1, None], state["offsets"].diff()[:, None]
    i = torch.arange(state["case"]["k"], device=n.device)[None]
    there = i < n
    return torch.where(there, start + i, 0).long(), there


def _packed(state, t, like):
    """Back from samples to packed rows, zeros behind the last sequence."""
    if state["offsets"] is None:
        return t
    at, there = _places(state)
    out = torch.zeros(like.shape[0], *t.shape[2:], dtype=t.dtype, device=t.device)
    out[at[there]] = t[there]
    return out


def _hidden(state, q, k):
    """True where a query does not see a key, [batch, 1, 1, queries, keys]; None: sees all."""
    case, hidden = state["case"], None
    i = torch.arange(q, device=state["q"].device)[:, None]
    j = torch.arange(k, device=state["q"].device)[None, :]
    if case["causal"]:
        hidden = (j > i + (k - q))[None, None, None]
    n = state["kv_lengths"]
    if state["offsets"] is not None:
        n = state["offsets"].diff()
    if n is not None:
        behind = (j[None] >= n[:, None, None])[:, None, None]
        hidden = behind if hidden is None else hidden | behind
    return hidden


def _grouped(t, kv_heads):
    """[batch, tokens, heads, dim] -> [batch, kv_heads, group * tokens, dim], float32."""
    t = t.float().unflatten(2, (kv_heads, -1)).permute(0, 2, 3, 1, 4)
    return t.flatten(2, 3)


def _ungrouped(t, group):
    return t.unflatten(2, (group, -1)).permute(0, 3, 1, 2, 4).flatten(2, 3)


def _probabilities(state, q, k):
    """Softmax of the scores [batch, kv_heads, group, queries, keys], and its log-sums."""
    case = state["case"]
    group = case["heads"] // case["kv_heads"]
    s = _grouped(q, case["kv_heads"]) @ _grouped(k, case["kv_heads"]).transpose(-1, -2)
    s = s.unflatten(2, (group, -1)).mul_(state["scale"])
    hidden = _hidden(state, q.shape[1], k.shape[1])
    if hidden is not None:
        s.masked_fill_(hidden, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(torch.where(total == 0, 1.0, total))
    return p, (top + torch.log(total)).squeeze(-1)


def _attend(state, q, k, v):
    """(output like q, log-sums [batch, heads, queries] or [heads, rows]), float32."""
    case = state["case"]
    group = case["heads"] // case["kv_heads"]
    p, lse = _probabilities(state, _padded(state, q), _padded(state, k))
    o = p.flatten(2, 3) @ _grouped(_padded(state, v), case["kv_heads"])
    lse = lse.flatten(1, 2)
    if state["offsets"] is not None:
        at, there = _places(state)
        flat = torch.full((case["heads"], q.shape[0]), -math.inf, device=q.device)
        flat[:, at[there]] = lse.permute(1, 0, 2)[:, there]
        lse = flat
    return _packed(state, _ungrouped(o, group), q), lse


def _attend_backward(state, g, q, k, v):
    case = state["case"]
    kv_heads, group = case["kv_heads"], case["heads"] // case["kv_heads"]
    pq, pk = _padded(state, q), _padded(state, k)
    p, _ = _probabilities(state, pq, pk)
    p = p.flatten(2, 3)
    do = _grouped(_padded(state, g), kv_heads)
    if state["offsets"] is not None:  # rows that are no sequence's have no gradient
        there = _places(state)[1][:, None, None, :, None]
        do = (do.unflatten(2, (group, -1)) * there).flatten(2, 3)
    dv = p.transpose(-1, -2) @ do
    dp = do @ _grouped(_padded(state, v), kv_heads).transpose(-1, -2)
    ds = dp.sub_((p * dp).sum(-1, keepdim=True)).mul_(p).mul_(state["scale"])
    dq = ds @ _grouped(pk, kv_heads)
    dk = ds.transpose(-1, -2) @ _grouped(pq, kv_heads)
    return (_packed(state, _ungrouped(dq, group), q), _packed(state, _ungrouped(dk, 1), k),
            _packed(state, _ungrouped(dv, 1), v))


def _plain(state):
    case = state["case"]
    dtype = TYPES[case["type"]]
    if case["op"] in ("rotary", "inverse"):
        how = (state["positions"], state["frequencies"], state["pairs"], case["layout"],
               case["op"] == "inverse")
        return {"q": _turn(state["q"], *how).to(dtype), "k": _turn(state["k"], *how).to(dtype)}
    if case["op"] == "forward":
        return _attend(state, state["q"], state["k"], state["v"])[0].to(dtype)
    if case["op"] == "backward":
        dq, dk, dv = _attend_backward(state, state["g"], state["q"], state["k"], state["v"])
        return {"q": dq.to(dtype), "k": dk.to(dtype), "v": dv.to(dtype)}
    q, k, v = (t.detach() for t in state["leaves"])
    at_q = (state["positions"], state["frequencies"], state["pairs"], "half")
    at_k = (state["k_positions"], *at_q[1:])
    q, k = _turn(q, *at_q, False).to(dtype), _turn(k, *at_k, False).to(dtype)
    out = _attend(state, q, k, v)[0].to(dtype)
    dq, dk, dv = _attend_backward(state, state["g"], q, k, v)
    return {"out": out, "q": _turn(dq.to(dtype), *at_q, True).to(dtype),
            "k": _turn(dk.to(dtype), *at_k, True).to(dtype), "v": dv.to(dtype)}


# ------------------------------------------------------------ the package's calls

def _own(state):
    import differentiable_image_quality_gb300 as pkg

    case = state["case"]
    if case["op"] in ("rotary", "inverse"):
        q, k = pkg.rotary(state["q"], state["k"], state["positions"], state["frequencies"],
                          state["pairs"], layout=case["layout"], inverse=case["op"] == "inverse")
        return {"q": q, "k": k}
    how = {"causal": case["causal"], "scale": state["scale"], "kv_lengths": state["kv_lengths"],
           "offsets": state["offsets"]}
    if case["op"] == "forward":
        return pkg.attention_fwd(state["q"], state["k"], state["v"], **how)[0]
    if case["op"] == "backward":
        dq, dk, dv = pkg.attention_bwd(state["g"], state["q"], state["k"], state["v"],
                                       state["out"], state["lse"], **how)
        return {"q": dq, "k": dk, "v": dv}
    q, k, v = state["leaves"]
    at = (state["frequencies"], state["pairs"])
    if case["q"] == case["k"]:
        q, k = pkg.fused_rotary(q, k, state["positions"], *at)
    else:
        q, _ = pkg.fused_rotary(q, None, state["positions"], *at)
        k, _ = pkg.fused_rotary(k, None, state["k_positions"], *at)
    out = pkg.fused_attention(q, k, v, **how)
    grads = torch.autograd.grad(out, state["leaves"], state["g"])
    return {"out": out.detach(), "q": grads[0], "k": grads[1], "v": grads[2]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------ the least a pass costs

_BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def work(case):
    size, dim = _BYTES[case["type"]], case["dim"]
    if case["op"] in ("rotary", "inverse"):
        n = case["batch"] * case["tokens"] * (case["heads"] + case["kv_heads"]) * dim
        axes = len(_split(case["pairs"]))
        pos = case["tokens"] * axes * (4 if case["positions"] == "float" else 8)
        return {"bytes": 2 * n * size + pos, "flops": 3 * n}
    H, K = case["heads"], case["kv_heads"]
    seen = rows = keys = 0
    for q, k in _sequences(case):
        if case["causal"]:
            # query i sees the first i + 1 + (width - queries) keys, as far as there are any
            shift = (k if case["ragged"] == "packed" else case["k"]) - q
            first, last = max(0, -shift), max(0, min(q, k - shift))
            part = max(0, last - first)
            seen += part * (first + last - 1 + 2 * (shift + 1)) // 2 + (q - max(last, first)) * k
        else:
            seen += q * k
        rows += q
        keys += k
    q_bytes, kv_bytes = rows * H * dim * size, 2 * keys * K * dim * size
    if case["op"] == "forward":
        return {"bytes": 2 * q_bytes + kv_bytes, "flops": 4 * seen * H * dim}
    if case["op"] == "backward":
        return {"bytes": 4 * q_bytes + 2 * kv_bytes + 4 * rows * H, "flops": 10 * seen * H * dim}
    # the leaves and the output's gradient in; the output and the leaves' gradients out
    return {"bytes": 4 * q_bytes + 2 * kv_bytes, "flops": 14 * seen * H * dim}


# ------------------------------------------------------------ in 64 bits, by definition

def _turn64(x, positions, frequencies, pairs, layout, sign):
    """As a product of complex numbers."""
    n = sum(pairs)
    turns = torch.cat([p[..., None] * f for p, f in
                       zip(positions.double().unbind(-1), frequencies.split(pairs))], -1)
    turn = torch.polar(torch.ones_like(turns), sign * turns).unsqueeze(-2)
    head, rest = x[..., :2 * n], x[..., 2 * n:]
    if layout == "half":
        z = torch.complex(head[..., :n], head[..., n:]) * turn
        return torch.cat([z.real, z.imag, rest], -1)
    z = torch.view_as_complex(head.unflatten(-1, (n, 2)).contiguous()) * turn
    return torch.cat([torch.view_as_real(z).flatten(-2), rest], -1)


def _one_head64(q, k, v, causal, scale, width):
    """One head of one sequence, [queries, dim] and [keys, dim]; `width`: the keys that the
    causal diagonal ends at."""
    if k.shape[0] == 0 or q.shape[0] == 0:
        return q * 0
    s = q @ k.T * scale
    if causal:
        seen = torch.ones(s.shape, dtype=torch.bool, device=s.device).tril(width - q.shape[0])
        s = torch.where(seen, s, -math.inf)
    lse = torch.logsumexp(s, -1, keepdim=True)
    return torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)) @ v


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] in ("rotary", "inverse"):
        how = (state["positions"], state["frequencies"], state["pairs"], case["layout"],
               -1.0 if case["op"] == "inverse" else 1.0)
        return {"q": _turn64(state["q"].double(), *how), "k": _turn64(state["k"].double(), *how)}
    train, wants = case["op"] == "train", case["op"] != "forward"
    leaves = [state[n].detach() for n in ("q", "k", "v")]
    group = case["heads"] // case["kv_heads"]
    out = torch.zeros(leaves[0].shape, dtype=torch.float64, device=leaves[0].device)
    grads = [torch.zeros(t.shape, dtype=torch.float64, device=t.device) for t in leaves]
    at = 0
    for b, (nq, nk) in enumerate(_sequences(case)):
        if case["ragged"] == "packed":
            rows, keys, width = slice(at, at + nq), slice(at, at + nk), nk
            at += nq
        else:
            rows, keys, width = (b, slice(0, nq)), (b, slice(0, nk)), case["k"]
        where = [rows, keys, keys]
        for h in range(case["heads"]):
            kh = h // group
            # one head at a time, the gradients by differentiating the definition
            q, k, v = (t[w][:, i].double().requires_grad_(wants)
                       for t, w, i in zip(leaves, where, (h, kh, kh)))
            tq, tk = q, k
            if train:
                how = (state["frequencies"], state["pairs"], "half", 1.0)
                pos, kpos = state["positions"], state["k_positions"]
                pos = pos[rows] if case["ragged"] == "packed" else pos[:nq]
                kpos = kpos[keys] if case["ragged"] == "packed" else kpos[:nk]
                tq = _turn64(q[:, None], pos, *how)[:, 0]
                tk = _turn64(k[:, None], kpos, *how)[:, 0]
            o = _one_head64(tq, tk, v, case["causal"], state["scale"], width)
            out[rows][:, h] = o.detach()
            if wants and nq and nk:
                got = torch.autograd.grad(o, (q, k, v), state["g"][rows][:, h].double())
                for sum_, w, i, g in zip(grads, where, (h, kh, kh), got):
                    sum_[w][:, i] += g
    found = dict(zip("qkv", grads))
    if not wants:
        return out
    return found if case["op"] == "backward" else {"out": out, **found}
