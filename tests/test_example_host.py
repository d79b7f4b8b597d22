"""The example's model on the CPU, with a stand-in for the operator."""
import importlib.util
import os

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_norms_start_with_a_gain_of_one(monkeypatch):
    spec = importlib.util.spec_from_file_location(
        "train_denoiser", os.path.join(ROOT, "examples", "train_denoiser.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    gains = []

    def norm(x, y=None, gate=None, *, post_weight=None, weight_offset=0.0, **how):
        if post_weight is not None:
            gains.append(post_weight.detach() + weight_offset)
        return x, x.to(torch.bfloat16)

    monkeypatch.setattr(example, "fused_residual_norm", norm)
    model = example.Denoiser(16, 2)
    model(torch.rand(2, 3, example.SIZE, example.SIZE), torch.rand(2))
    assert len(gains) == 4 and all(torch.equal(g, torch.ones(16)) for g in gains)
