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
    # small: warps but for two at the most, large: tiles but for one
    for xt in (BF, F32):
        for act in ("relu", "silu", "gelu", "swiglu"):
            assert sum(tiles(*c, act, xt) for c in LARGE) >= len(LARGE) - 1
            assert sum(tiles(*c, act, xt) for c in SMALL) <= 2


# both ways measured, in us: shapes near where they cross, with 1, 2, 4 and more assignments a group, and with many tokens
MEASURED = [
    (76, 4, 153, 512, 512, 512, "relu", BF, 33.7, 32.7),
    (105, 4, 210, 512, 512, 512, "relu", BF, 38.4, 39.6),
    (28, 2, 14, 1024, 2048, 1024, "relu", BF, 30.0, 32.2),
    (52, 2, 26, 1024, 2048, 1024, "relu", BF, 50.3, 46.2),
    (18, 2, 18, 3328, 1024, 1024, "relu", BF, 30.5, 36.3),
    (68, 4, 34, 3328, 1024, 1024, "relu", BF, 77.4, 60.2),
    (20, 2, 5, 4096, 1024, 4096, "relu", BF, 31.7, 37.5),
    (14, 2, 7, 4096, 1024, 4096, "relu", BF, 28.7, 39.0),
    (10, 2, 10, 4096, 1024, 4096, "relu", BF, 32.0, 39.4),
    (16, 2, 32, 2048, 1408, 2048, "swiglu", BF, 68.0, 65.2),
    (48, 4, 64, 1024, 2048, 1024, "silu", HF, 88.4, 80.2),
    (64, 4, 16, 3328, 2048, 1024, "relu", BF, 96.2, 59.1),
    (1, 2, 16, 3328, 1024, 1024, "relu", F32, 14.2, 24.5),
    (16, 2, 16, 3328, 1024, 1024, "relu", BF, 28.1, 34.2),
    (64, 8, 8, 2048, 2048, 2048, "relu", BF, 67.2, 45.7),
    (512, 1, 1, 4096, 4096, 4096, "relu", BF, 249.2, 130.7),
    (128, 4, 16, 1024, 2048, 1024, "relu", BF, 64.0, 39.7),
    (114, 1, 95, 808, 2360, 624, "gelu", F32, 77.5, 65.5),
    (2, 8, 132, 256, 1464, 2224, "relu", F32, 29.7, 31.6),
    (182, 2, 25, 832, 304, 2312, "relu", F32, 39.2, 26.5),
    (66, 1, 16, 840, 2736, 1352, "relu", F32, 58.9, 48.6),
    (3, 2, 68, 1440, 1872, 2656, "swiglu", BF, 30.0, 32.7),
    (35, 1, 18, 4328, 1152, 720, "silu", BF, 49.3, 43.1),
    (68, 1, 19, 696, 1600, 1352, "swiglu", F32, 46.4, 39.6),
    (3, 4, 133, 1192, 3008, 672, "relu", F32, 32.0, 39.0),
    (89, 2, 2, 464, 3096, 1456, "swiglu", F32, 63.8, 44.4),
    (72, 2, 341, 1272, 536, 1912, "relu", BF, 73.4, 68.0),
    (1, 5, 5, 680, 5232, 4816, "gelu", BF, 61.0, 56.8),
    (80, 1, 67, 2736, 968, 2176, "silu", F32, 73.8, 65.1),
    (169, 2, 178, 360, 344, 1376, "relu", F32, 45.4, 43.4),
]


def test_the_rule_takes_the_faster_way():
    # or one within 3 % of it, on all but three; of 740 shapes measured the worst choice was 20 % behind
    behind = []
    for T, k, E, D, H, N, act, xt, warps, in_tiles in MEASURED:
        taken = in_tiles if tiles(T, k, E, D, H, N, act, xt) else warps
        behind.append(taken / min(warps, in_tiles) - 1)
    assert max(behind) <= 0.2 and sum(b > 0.03 for b in behind) <= 3, behind


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
