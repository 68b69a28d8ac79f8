"""A recommender's training step with experts: pooled embeddings, k of E expert
networks a sample, one logit, and every weight stepped.

    python examples/train_experts.py [--steps 60]

The embedding layer's output (fp32) is each sample's token.  A router gives k
experts and their weights; expert_sort plans the batch, expert_dispatch brings
the rows into expert order in bf16, two expert_linear calls with a ReLU between
them are the experts' networks, expert_combine adds their answers up.  The
gradients take the same calls' gradients back to grad_out of the layer's
backward_update.  The experts' weights, [E, out, in], are stepped with
orthogonalised momentum (the Muon optimiser), the router and the last layer with
plain SGD.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import ctr_inputs as ci  # noqa: E402
import dlrm_sparse_embedding_gb300 as emb  # noqa: E402


class ExpertTower:
    """logit[b] = <head, sum_j w[b, j] W2[e] relu(W1[e] x[b])> over sample b's k experts e."""

    def __init__(self, width: int, hidden: int, out: int, experts: int, k: int, seed: int = 0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def normal(*shape):
            return torch.randn(*shape, generator=g, device="cuda") / shape[-1] ** 0.5

        self.experts, self.k = experts, k
        self.router, self.head = normal(experts, width), normal(out)
        # fp32 weights with the bf16 copies that the products read, and their momentum
        self.w = [normal(experts, hidden, width), normal(experts, out, hidden)]
        self.w16 = [w.bfloat16() for w in self.w]
        self.momentum = [torch.zeros_like(w) for w in self.w]

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        scores, ids = torch.topk(x @ self.router.t(), self.k, dim=1)
        weights = torch.softmax(scores, dim=1)
        plan = emb.expert_sort(ids, self.experts)
        rows = emb.expert_dispatch(plan, x, dtype=torch.bfloat16)
        hidden = torch.relu_(emb.expert_linear(plan, rows, self.w16[0]))
        y = emb.expert_linear(plan, hidden, self.w16[1])
        out = emb.expert_combine(plan, y, weights, dtype=torch.float32)
        self.kept = (x, ids, weights, plan, rows, hidden, y, out)
        return out @ self.head

    def backward(self, grad_logit: torch.Tensor):
        """Gradients of x, the router, the head and the experts' weights."""
        x, ids, weights, plan, rows, hidden, y, out = self.kept
        grad_out = grad_logit[:, None] * self.head
        grad_y, grad_weights = emb.expert_combine_grad(plan, grad_out, y, weights)
        grad_hidden, grad_w2 = emb.expert_linear_grad(plan, grad_y, hidden, self.w16[1])
        grad_hidden.mul_(hidden > 0)
        grad_rows, grad_w1 = emb.expert_linear_grad(plan, grad_hidden, rows, self.w16[0])
        grad_x = emb.expert_dispatch_grad(plan, grad_rows, dtype=torch.float32)
        # the softmax over the chosen scores
        grad_scores = weights * (grad_weights - (weights * grad_weights).sum(1, keepdim=True))
        grad_router_out = torch.zeros(x.shape[0], self.experts, device=x.device).scatter_(1, ids, grad_scores)
        return (grad_x + grad_router_out @ self.router, grad_router_out.t() @ x, grad_logit @ out, [grad_w1, grad_w2])

    def step(self, grad_router, grad_head, grad_w, lr: float, momentum: float = 0.9) -> None:
        self.router -= lr * grad_router
        self.head -= lr * grad_head
        for w, w16, m, g in zip(self.w, self.w16, self.momentum, grad_w):
            m.mul_(momentum).add_(g)
            update = emb.orthogonalize(m)      # every expert's matrix by itself
            rows, cols = w.shape[1:]
            w.sub_(update, alpha=0.1 * lr * max(1.0, rows / cols) ** 0.5)
            w16.copy_(w)


def train(steps: int, batch: int = 1024, experts: int = 8, k: int = 2, lr: float = 0.1, report=print):
    """Learns whether the first table's key is in the upper half; returns the losses."""
    tables = [ci.TableSpec(2000, 32, "f32", "sum", "adagrad", lr=0.05) for _ in range(8)]
    w = ci.Workload("experts", tuple(tables), batch, "fixed", 1, 1, "uniform")
    layer = emb.EmbeddingLayer(tables, batch, batch * len(tables))
    losses = []
    try:
        layer.init_uniform(0, -0.5, 0.5)
        tower = ExpertTower(layer.total_dim, 512, 64, experts, k)
        for step in range(steps):
            b = ci.make_batch(w, seed=step)
            label = torch.from_numpy((b.keys[:batch] >= 1000).astype("float32")).cuda()
            x = layer.forward(torch.from_numpy(b.keys).cuda(), torch.from_numpy(b.offsets).cuda(),
                              torch.from_numpy(b.table_ids).cuda(), batch)
            logit = tower.forward(x)
            loss = torch.nn.functional.binary_cross_entropy_with_logits(logit, label)
            grad_x, grad_router, grad_head, grad_w = tower.backward((torch.sigmoid(logit) - label) / batch)
            layer.backward_update(grad_x, "reduction")
            tower.step(grad_router, grad_head, grad_w, lr)
            losses.append(loss.item())
            if step % 10 == 0 or step == steps - 1:
                report("step %3d  loss %.4f" % (step, losses[-1]))
        if layer.sync_status() != emb.EMB_OK or emb.dense_status() != emb.EMB_OK:
            raise RuntimeError("a call reported an error")
    finally:
        layer.close()
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    train(ap.parse_args().steps)
