"""GPU: the training example runs all operators together, learns, and its
gradient is the loss's: a step along it lowers the loss as it says."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
m = pytest.importorskip("maxsim_scoring_02_gb300")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("train_encoder", os.path.join(ROOT, "examples", "train_encoder.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    m.load_library()
    return mod


def test_training_lowers_the_loss(example):
    losses = example.train()
    assert all(l == l for l in losses)
    assert sum(losses[-3:]) < 0.9 * sum(losses[:3]), losses


def test_gradient_is_the_losses(example):
    """The loss along the gradient: a step of s * g / |g| changes it by about
    s * |g| (to 25 %: the forward rounds to bf16, and curvature is left out)."""
    data = example.batch(32, 16, 100, 256, seed=5)
    e = example.Encoder(256, 4, 64, seed=3)
    before = [w.clone() for w in (e.w_qkv, e.w_out)]
    loss, norm = example.step(e, data, lr=0.0, max_norm=1e9)
    moved = []
    for s in (0.4, -0.4):
        e.w_qkv, e.w_out = (w.clone() for w in before)
        example.step(e, data, lr=s / norm.item(), max_norm=1e9)
        moved.append(example.step(e, data, lr=0.0)[0].item())
    assert abs((moved[1] - moved[0]) / (0.8 * norm.item()) - 1) <= 0.25, (moved, norm.item())
