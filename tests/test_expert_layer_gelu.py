"""expert_layer's gelu where its value is far smaller than its argument.

A token with one element and a `down` of ones on its diagonal show hidden as it is: the activation of an
exact argument, rounded once.  The error allowed is that rounding's half step and, relative to the value, of
v / 2 erfc(-v / sqrt 2): some 16 roundings e = 2^-24 of erfc, the products and the argument's own, 2 e
at most, which erfc's slope makes at most v^2 + 1 times as large."""
import pytest
import torch

import dlrm_sparse_embedding_gb300 as emb
from test_expert_layer import LARGE, HALF_ULP, TINY
from test_expert_layer_ways import tiles

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
E24 = 2.0 ** -24


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,E,D,H,N", [(1, 1, 1, 8, 200, 200), (5, 2, 3, 16, 208, 200), (64, 2, 4, 16, 200, 208), LARGE[0], (65, 6, 3, 1000, 1000, 1000)])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("xt", [None, F32])
def test_small_values_keep_their_digits(T, k, E, D, H, N, dtype, xt):
    assert tiles(T, k, E, D, H, N, "gelu", xt or dtype) == (D > 500)
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    v = (torch.arange(H, device="cuda") % 200 - 150).double() / 12.5        # -12 .. 3.92
    v = v.to(dtype)
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda")
    x = torch.zeros(T, D, dtype=xt or dtype, device="cuda")
    x[:, 0] = 1
    up, down = torch.zeros(E, H, D, dtype=dtype, device="cuda"), torch.zeros(E, N, H, dtype=dtype, device="cuda")
    up[:, :, 0] = v
    n = min(N, H)
    down[:, range(n), range(n)] = 1
    weights = torch.zeros(T, k, device="cuda")
    weights[:, 0] = 1
    out = emb.expert_layer(ids, x, up, down, weights, "gelu", F32)[:, :n].double()
    z = v[:n].double()
    ref = 0.5 * z * torch.special.erfc(-z * 0.5 ** 0.5)
    off = ref.abs() * (16 + 2 * (z * z + 1)) * E24
    bound = off + HALF_ULP[dtype] * (ref.abs() + off) + TINY[dtype]
    assert ((out - ref).abs() <= bound).all(), ((out - ref).abs() - bound).max().item()
