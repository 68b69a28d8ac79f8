"""What all calls of the dense side share: the device's status word, the current
device, gradients."""
import threading

import pytest
import torch

import dlrm_sparse_embedding_gb300 as emb
from dlrm_sparse_embedding_gb300 import experts

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("callers", [2, 8, 100])
def test_of_many_callers_one_gets_the_status(callers):
    ids = torch.tensor([[0], [9]], dtype=torch.int32, device="cuda")
    streams = [torch.cuda.Stream() for _ in range(callers)]
    for _ in range(200 if callers < 100 else 10):
        emb.expert_sort(ids, 4)
        torch.cuda.synchronize()
        begin, got = threading.Barrier(callers), [None] * callers

        def ask(i):
            begin.wait()
            got[i] = emb.dense_status(streams[i])

        threads = [threading.Thread(target=ask, args=(i,)) for i in range(callers)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert sorted(got) == sorted([emb.EMB_ERR_KEY_RANGE] + [emb.EMB_OK] * (callers - 1))


def test_a_device_that_is_not_the_current_one_is_refused(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    with pytest.raises(ValueError, match="current device"):
        experts._stream(torch.device("cuda", 1))


@gpu
def test_every_call_refuses_tensors_of_another_device(monkeypatch):
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    ids, w, weights, stream = z(6, 2, dtype=torch.int32), z(4, 16, 24), z(6, 2, dtype=torch.float32), torch.cuda.Stream()
    plan = emb.expert_sort(ids, 4)
    calls = [
        lambda: emb.expert_sort(ids, 4), lambda: emb.expert_dispatch(plan, z(6, 8)), lambda: emb.expert_dispatch_grad(plan, z(12, 8)),
        lambda: emb.expert_combine(plan, z(12, 8), weights), lambda: emb.expert_combine_grad(plan, z(6, 8), z(12, 8), weights),
        lambda: emb.expert_linear(plan, z(12, 24), w), lambda: emb.expert_linear_grad(plan, z(12, 16), z(12, 24), w),
        lambda: emb.expert_linear_grad(plan, z(12, 16), z(12, 24), w, need_rows=False), lambda: emb.orthogonalize(z(4, 4)),
        lambda: emb.dense_status(stream),
    ]
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)      # nothing is launched: the tensors are on 0
    for i, call in enumerate(calls):
        with pytest.raises(ValueError, match="current device"):
            call()
            pytest.fail("call %d was taken" % i)
    monkeypatch.undo()
    for call in calls:
        call()


@gpu
def test_results_require_no_gradient():
    # the backward pass is explicit: inputs that require gradients are read, and nothing joins autograd's graph
    r = lambda *s, dtype=torch.bfloat16: torch.randn(*s, device="cuda").to(dtype).requires_grad_()  # noqa: E731
    plan = emb.expert_sort(torch.randint(0, 4, (6, 2), device="cuda"), 4)
    x, rows, y, w, weights, g = r(6, 24), r(12, 24), r(12, 16), r(4, 16, 24), r(6, 2, dtype=torch.float32), r(6, 16)
    got = [emb.expert_dispatch(plan, x), emb.expert_dispatch_grad(plan, rows), emb.expert_linear(plan, rows, w),
           emb.expert_combine(plan, y, weights), emb.orthogonalize(w), *emb.expert_linear_grad(plan, y, rows, w),
           *emb.expert_combine_grad(plan, g, y, weights)]
    assert not any(t.requires_grad for t in got)
    assert torch.equal(got[2], emb.expert_linear(plan, rows.detach(), w.detach()))


@gpu
def test_a_function_of_autograd_takes_the_calls():
    class Expert(torch.autograd.Function):
        @staticmethod
        def forward(ctx, plan, x, w, weights):
            rows = emb.expert_dispatch(plan, x, torch.float16)
            y = emb.expert_linear(plan, rows, w)
            ctx.plan = plan
            ctx.save_for_backward(rows, w, y, weights)
            return emb.expert_combine(plan, y, weights, torch.float32)

        @staticmethod
        def backward(ctx, grad):
            rows, w, y, weights = ctx.saved_tensors
            grad_y, grad_weights = emb.expert_combine_grad(ctx.plan, grad.contiguous(), y, weights)
            grad_rows, grad_w = emb.expert_linear_grad(ctx.plan, grad_y, rows, w)
            return None, emb.expert_dispatch_grad(ctx.plan, grad_rows, torch.float32), grad_w, grad_weights

    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    ids = torch.randint(0, 3, (20, 2), generator=g, device="cuda")
    # small whole numbers: exact in every type
    ints = lambda *s, dtype=torch.float32: torch.randint(-2, 3, s, generator=g, device="cuda").to(dtype).requires_grad_()  # noqa: E731
    x, w, weights = ints(20, 16), ints(3, 8, 16, dtype=torch.float16), ints(20, 2)
    Expert.apply(emb.expert_sort(ids, 3), x, w, weights).sum().backward()
    xr, wr, sr = (t.detach().double().requires_grad_() for t in (x, w, weights))
    (torch.einsum("tjoi,ti->tjo", wr[ids], xr) * sr[:, :, None]).sum().backward()
    for t, ref in ((x, xr), (w, wr), (weights, sr)):
        assert torch.equal(t.grad.double(), ref.grad)
