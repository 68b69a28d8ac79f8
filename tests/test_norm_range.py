"""layer_norm's eps over the whole range that its contract gives."""
import pytest
import torch

import dlrm_sparse_embedding_gb300 as emb
from dlrm_sparse_embedding_gb300 import norm

LARGEST = torch.finfo(torch.float32).max


def test_eps_up_to_the_largest_number_is_taken():
    for eps in (1e-24, 1.0, 1e30, 1.1e30, 1e38, LARGEST):
        assert norm._eps(eps) == eps
    for eps in (0.0, -1.0, 9e-25, LARGEST * 1.001, float("inf"), float("nan")):
        with pytest.raises(ValueError, match="eps"):
            norm._eps(eps)


@pytest.mark.gpu
@pytest.mark.parametrize("width", [40, 1000, 3328, 9000])
@pytest.mark.parametrize("eps", [1e31, LARGEST])
@pytest.mark.parametrize("size", [1.0, 2.0 ** 60])
def test_a_large_eps(width, eps, size):
    g = torch.Generator(device="cuda")
    g.manual_seed(width)
    x, gy = (torch.randn(20, width, generator=g, device="cuda") for _ in range(2))
    x *= size
    y, (dx, dw, db) = emb.layer_norm(x, eps=eps), emb.layer_norm_grad(gy, x, eps=eps)
    xd, gd = x.double(), gy.double()
    c = xd - xd.mean(1, keepdim=True)
    rstd = 1 / (c.square().mean(1, keepdim=True) + eps).sqrt()
    h = c * rstd
    ref = rstd * (gd - gd.mean(1, keepdim=True) - h * (gd * h).mean(1, keepdim=True))
    # chains of at most 73 roundings (widths to 9000), some ten operations more, of terms no larger than the row's largest
    # element; the squares' sum likewise, of which the root takes half
    off = 100 * 2.0 ** -24
    large, grad = xd.abs().amax(1, keepdim=True) * rstd, gd.abs().amax(1, keepdim=True)
    assert ((y.double() - h).abs() <= off * large).all()
    assert ((dx.double() - ref).abs() <= 4 * off * rstd * grad * (1 + large) ** 2).all()
    assert ((dw.double() - (gd * h).sum(0)).abs() <= 2 * off * 20 * (grad * large).amax()).all()
    assert ((db.double() - gd.sum(0)).abs() <= off * 20 * grad.amax()).all()
