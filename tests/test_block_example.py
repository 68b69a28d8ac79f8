"""Layer norm, dropout and the expert layer of a few tokens as one tower uses them with the
other expert calls (examples/train_experts.py)."""
import importlib.util
import os

import pytest
import torch

import dlrm_sparse_embedding_gb300 as emb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_experts.py")
    spec = importlib.util.spec_from_file_location("train_experts", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def tower_and_batch(example, tokens, dropout):
    tower = example.ExpertTower(64, 96, 40, 6, 2, seed=1, norm=True, dropout=dropout)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    tower.norm[0] += 0.2 * r(64)
    tower.norm[1] += 0.2 * r(64)
    return tower, 3 * r(tokens, 64) + r(64), r(tokens)


E = 2.0 ** -24      # fp32's half step


@pytest.mark.parametrize("dropout", [0.0, 0.25])
def test_norm_and_dropout_in_a_step(example, dropout):
    """The tower with its norm is the tower without one on normalised tokens, and takes that
    one's gradient back through the norm; the dropped part of its answer has no gradient."""
    T, out_width = 150, 40
    tower, x, grad_logit = tower_and_batch(example, T, dropout)
    inner = example.ExpertTower(64, 96, out_width, 6, 2, seed=1, dropout=dropout)     # the same weights
    logit = tower.forward(x)
    grad_x, *grads = tower.backward(grad_logit)
    tokens, out = tower.kept[0], tower.kept[7]
    assert torch.equal(inner.forward(tokens), logit)
    grad_tokens, *inner_grads = inner.backward(grad_logit)
    for a, b in zip((*grads[:2], *grads[2]), (*inner_grads[:2], *inner_grads[2])):
        assert torch.equal(a, b)

    xd, gain, shift = (t.double().requires_grad_() for t in (x, *tower.norm))
    normed = (xd - xd.mean(1, keepdim=True)) / (xd.var(1, correction=0, keepdim=True) + 1e-5).sqrt()
    h = normed * gain + shift
    # 64 wide: an element is off by at most 100 roundings of 1 + its own size, a gradient's by 400 of the row's
    assert ((tokens.double() - h).abs() <= 100 * E * (1 + normed.abs()) * (gain.abs() + shift.abs())).all()
    h.backward(grad_tokens.double())
    row = grad_tokens.double().norm(dim=1, keepdim=True) * gain.abs().max() / xd.std(1, correction=0, keepdim=True)
    assert ((grad_x.double() - xd.grad).abs() <= 400 * E * row * (1 + normed.abs())).all()
    for got, want, terms in zip(tower.norm_grad, (gain.grad, shift.grad), ((grad_tokens * normed).abs(), grad_tokens.double().abs())):
        assert ((got.double() - want).abs() <= 400 * E * (terms.sum(0) + grad_tokens.double().abs().sum(0))).all()

    # the same step without dropout, masked by hand
    kept = emb.dropout(torch.ones(T, out_width, device="cuda"), dropout, tower.seed, tower.steps)
    whole = example.ExpertTower(64, 96, out_width, 6, 2, seed=1)
    whole.forward(tokens)
    assert ((whole.kept[7] * kept).double() - out.double()).abs().max() <= 4 * E * out.abs().max()
    _, _, weights, plan, _, _, y, _ = tower.kept
    grad_y, grad_weights = emb.expert_combine_grad(plan, emb.dropout_grad(grad_logit[:, None] * tower.head, dropout, tower.seed, tower.steps), y, weights)
    by_hand, by_hand_weights = emb.expert_combine_grad(plan, grad_logit[:, None] * tower.head * kept, y, weights)
    # one rounding of the scale more, which a rounding to bf16 may carry a step further
    assert ((grad_y.double() - by_hand.double()).abs() <= 2.0 ** -7 * by_hand.double().abs()).all()
    assert ((grad_weights - by_hand_weights).abs() <= 400 * E * by_hand_weights.abs().max()).all()


@pytest.mark.parametrize("tokens", [1, 7, 150])
def test_a_few_samples_are_served_as_they_were_trained(example, tokens):
    tower, x, _ = tower_and_batch(example, tokens, 0.0)
    # both round hidden to bf16, the one its products' rows as well
    got, ref = tower.predict(x), tower.forward(x)
    scale = tower.kept[7].norm(dim=1) * tower.head.norm()
    assert ((got - ref).abs() <= 4 * 2.0 ** -8 * scale).all()


def test_the_example_runs(example):
    said = []
    losses = example.train(5, report=said.append, norm=True, dropout=0.1)
    assert len(losses) == 5 and all(l == l for l in losses) and said[-1].startswith("served")
