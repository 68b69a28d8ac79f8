"""The expert layer, its gradients and the orthogonalised step as one training
step uses them (examples/train_experts.py)."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_experts.py")
    spec = importlib.util.spec_from_file_location("train_experts", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_a_steps_gradients_are_autograds(example):
    tower = example.ExpertTower(64, 96, 40, 6, 2, seed=1)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x = torch.randn(150, 64, generator=g, device="cuda")
    grad_logit = torch.randn(150, generator=g, device="cuda")
    logit = tower.forward(x)
    grad_x, grad_router, grad_head, grad_w = tower.backward(grad_logit)

    ids = tower.kept[1]
    leaves = [t.double().requires_grad_() for t in (x, tower.router, tower.head, tower.w16[0], tower.w16[1])]
    xd, router, head, w1, w2 = leaves
    weights = torch.softmax((xd @ router.t()).gather(1, ids), dim=1)
    y = torch.einsum("tjoh,tjh->tjo", w2[ids], torch.relu(torch.einsum("tjhi,ti->tjh", w1[ids], xd)))
    ref = (weights[:, :, None] * y).sum(1) @ head
    ref.backward(grad_logit.double())
    # a chain of at most eight roundings to bf16 (2^-9 each on average over a norm, and a ReLU's sign that one of them flips)
    bound = 8 * 2.0 ** -8
    assert (logit - ref).norm() <= bound * ref.norm()
    for got, leaf in zip((grad_x, grad_router, grad_head, *grad_w), leaves):
        assert (got.double() - leaf.grad).norm() <= bound * leaf.grad.norm()


def test_training_learns(example):
    losses = example.train(40, report=lambda *_: None)
    assert losses[0] > 0.6 and sum(losses[-5:]) / 5 < 0.8 * losses[0]
