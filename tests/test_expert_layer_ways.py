"""Which of its two ways expert_layer takes, as the library tells it and as its workspace shows it."""
import ctypes

import pytest
import torch

import dlrm_sparse_embedding_gb300 as emb
from dlrm_sparse_embedding_gb300._lib import ACTIVATIONS
from test_expert_layer import LARGE, SMALL, case, check

gpu = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
CODE = {F32: 0, HF: 1, BF: 2}


def tiles(T, k, E, D, H, N, act="relu", xt=BF) -> bool:
    way = ctypes.c_int32(-1)
    assert emb.lib.emb_expert_layer_tiles(T, k, E, CODE[xt], D, H, N, ACTIVATIONS[act], ctypes.byref(way)) == emb.EMB_OK
    return {0: False, 1: True}[way.value]


def test_the_calls_refusals():
    way = ctypes.c_int32()
    ok = [4, 2, 8, 2, 64, 32, 24, 0, ctypes.byref(way)]
    assert emb.lib.emb_expert_layer_tiles(*ok) == emb.EMB_OK and way.value == 0
    assert emb.lib.emb_expert_layer_tiles(0, *ok[1:]) == emb.EMB_OK and way.value == 0
    for i, v in ((0, -1), (0, 257), (1, 0), (1, 65), (2, 0), (2, 1025), (3, 3), (3, -1), (4, 12), (5, 0), (6, 2 ** 25), (7, 4), (7, -1), (8, None)):
        args = list(ok)
        args[i] = v
        assert emb.lib.emb_expert_layer_tiles(*args) == emb.EMB_ERR_INVALID_ARG, (i, v)


def test_the_lists_of_the_layers_tests_reach_both_ways():
    # small: warps but for some, large: tiles but for some, by a wide margin of sizes whatever the rule's constants
    for xt in (BF, F32):
        for act in ("relu", "silu", "gelu", "swiglu"):
            assert sum(tiles(*c, act, xt) for c in LARGE) >= len(LARGE) - 1
            assert sum(tiles(*c, act, xt) for c in SMALL) <= 1


def workspace_used(args, act):
    """Whether the call brings the tokens' rows to its workspace, which the tiles' way alone does first."""
    ids, x, up, down, weights = args
    (T, k), (E, _, D), (_, N, H) = ids.shape, up.shape, down.shape
    n = ctypes.c_size_t()
    assert emb.lib.emb_expert_layer_workspace(T, k, D, H, N, ctypes.byref(n)) == emb.EMB_OK
    ws = torch.full((n.value,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.empty(T, N, dtype=up.dtype, device="cuda")
    at = lambda t: t.data_ptr()  # noqa: E731
    assert emb.lib.emb_expert_layer(at(ids), ids.element_size(), T, k, E, at(x), CODE[x.dtype], x.stride(0), D, at(up), at(down), CODE[up.dtype], H, N,
                                    ACTIVATIONS[act], at(weights), at(out), CODE[up.dtype], at(ws), n.value,
                                    torch.cuda.current_stream().cuda_stream) == emb.EMB_OK
    check(args, act, out=out)
    return bool((ws[:T * k * D * 2] != 0xA5).any())


@gpu
@pytest.mark.parametrize("act,xt", [("relu", BF), ("swiglu", BF), ("gelu", F32)])
@pytest.mark.parametrize("c", SMALL + LARGE)
def test_the_call_takes_the_way_it_tells(c, act, xt):
    args = case(sum(c), *c, BF, xt, act)
    assert workspace_used(args, act) == tiles(*c, act, xt)


# one group of every size, in tiles: k's other assignments are to nobody
IN_TILES = [(1, 64), (15, 32), (16, 32), (17, 30), (31, 16), (32, 16), (33, 15), (63, 8), (64, 8), (65, 7), (127, 4), (128, 4), (129, 3), (255, 2)]


def test_the_groups_below_are_in_tiles():
    for n, k in IN_TILES:
        assert tiles(n, k, 64, 1024, 1544, 1032)


@gpu
@pytest.mark.parametrize("n,k", IN_TILES)
@pytest.mark.parametrize("act", ["relu", "swiglu"])
def test_groups_of_every_size_in_tiles(n, k, act):
    ids, x, up, down, weights = case(n, n, k, 64, 1024, 1544, 1032, BF, BF, act)
    ids[:] = -1
    ids[:, k // 2] = 2
    weights[:, k // 2] = 0.75
    if n > 20:
        ids[3, 0], ids[9, 1] = 63, 0
    check((ids, x, up, down, weights), act)
