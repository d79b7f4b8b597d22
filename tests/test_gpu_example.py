"""The example's training step: the operators together, learning something."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_denoiser_learns():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from differentiable_image_quality_gb300 import _build

    _build.build()
    spec = importlib.util.spec_from_file_location(
        "train_denoiser", os.path.join(ROOT, "examples", "train_denoiser.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses = example.train(report=lambda line: None)
    assert all(v == v for v in losses)
    first, last = sum(losses[:5]) / 5, sum(losses[-5:]) / 5
    # the noisy image is where it starts; it has to have come a good part of the way
    assert last < 0.7 * first, (first, last)
