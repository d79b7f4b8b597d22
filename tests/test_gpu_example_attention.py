"""The example's model with attention between its patches: that it runs, and its gradients."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from differentiable_image_quality_gb300 import _build

    _build.build()
    spec = importlib.util.spec_from_file_location(
        "train_denoiser", os.path.join(ROOT, "examples", "train_denoiser.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_trains(example):
    losses = example.train(steps=3, mixing="attention", report=lambda line: None)
    assert len(losses) == 3 and all(v == v for v in losses)


def test_gradients(example, monkeypatch):
    """Against the same model with attention and positions in plain float32 operations: the
    two differ by the roundings of q, k, v, the probabilities and their gradients to
    bfloat16, 2^-8 at most each, in both of the two blocks, forward and back: 5 of them,
    2 blocks, 2 directions, 2^-8 sqrt(20) = 1.8 % of a gradient where they are
    independent, twice that allowed."""
    import torch

    def rotary(q, k, at, f, pairs):
        angle = (at.double()[:, [0] * pairs[0] + [1] * pairs[1]] * f)[:, None].float()
        n = sum(pairs)

        def turn(t):
            a, b = t.float()[..., :n], t.float()[..., n:]
            return torch.cat([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()], -1)

        return turn(q), turn(k)

    def attention(q, k, v):
        s = torch.einsum("bihd,bjhd->bhij", q, k) * q.shape[-1] ** -0.5
        return torch.einsum("bhij,bjhd->bihd", s.softmax(-1), v.float()).to(v.dtype)

    def gradients():
        torch.manual_seed(0)
        model = example.Denoiser(64, 2, "attention").cuda()
        torch.nn.init.normal_(model.head.weight, std=0.05)
        clean, noisy, strength = next(example.batches(4))
        (model(noisy, strength) - clean).square().mean().backward()
        return {n: p.grad for n, p in model.named_parameters()}

    ours = gradients()
    monkeypatch.setattr(example, "fused_rotary", rotary)
    monkeypatch.setattr(example, "fused_attention", attention)
    plain = gradients()
    assert any("qkv" in n for n in ours)
    for name, ref in plain.items():
        assert ref.norm() > 0 or "head" not in name
        assert (ours[name] - ref).norm() <= 0.036 * ref.norm() + 1e-12, name
