"""The expert layer of a few tokens against a plain implementation in 64 bits.

Tolerances.  u is half the spacing of the weights' type (2^-11 fp16, 2^-8 bf16), e = 2^-24.  A
product's sum of n terms adds exact products in fp32, which the tensor cores may cut
off where others round: z is off by dz = n 2^-23 sum |up x|.  The activations' slopes are at
most 1.13; evaluating one is off by 8 e of |z| (gelu's 1 + erf loses nothing relative to z).
hidden is rounded to the type: dh = 1.13 dz + 8 e |z| + u (|h| + those) + half the type's
smallest number; a gated one's two factors each bring their own, the gate's times the other.
y is off by |down| dh and by H 2^-23 |down| (|h| + dh), the weighted sum of k by (k + 1) e of
its terms' magnitudes, and the output is rounded once.
"""
import ctypes
import math

import pytest
import torch

import dlrm_sparse_embedding_gb300 as emb

gpu = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
HALF_ULP = {F32: 2.0 ** -24, HF: 2.0 ** -11, BF: 2.0 ** -8}
TINY = {F32: 2.0 ** -149, HF: 2.0 ** -25, BF: 2.0 ** -133}
E24, E23 = 2.0 ** -24, 2.0 ** -23


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def case(seed, T, k, E, D, H, N, dtype, xt, act="relu", dropped=0.0, ids_dtype=torch.int32):
    g = gen(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda")       # an expert may come twice
    if dropped:
        ids[torch.rand(T, k, generator=g, device="cuda") < dropped] = -1
    x = r(T, D).to(xt)
    up = (r(E, H * (2 if act == "swiglu" else 1), D) / D ** 0.5).to(dtype)
    down = (r(E, N, H) / H ** 0.5).to(dtype)
    weights = torch.rand(T, k, generator=g, device="cuda") - 0.25
    weights[ids < 0] = float("nan")     # not used
    return ids.to(ids_dtype), x, up, down, weights


def act_of(act, z, dz, H):
    """The activation and its error's bound before rounding."""
    s = lambda v: v * torch.sigmoid(v)  # noqa: E731
    if act == "swiglu":
        g, u = z[:, :H], z[:, H:]
        dg, du = dz[:, :H], dz[:, H:]
        sg, dsg = s(g), 1.13 * dg + 8 * E24 * g.abs()
        return sg * u, dsg * (u.abs() + du) + sg.abs() * du + E24 * (sg * u).abs()
    h = {"relu": torch.relu, "silu": s, "gelu": lambda v: v * torch.special.ndtr(v)}[act](z)
    return h, 1.13 * dz + 8 * E24 * z.abs()


def check(args, act, dtype=None, out=None):
    ids, x, up, down, weights = args
    T, k = ids.shape
    H, N = down.shape[2], down.shape[1]
    got = emb.expert_layer(ids, x, up, down, weights, act, dtype) if out is None else out
    assert got.dtype == (dtype or up.dtype) and got.shape == (T, N) and got.is_contiguous()
    xd = x.to(up.dtype).double()
    ref = torch.zeros(T, N, dtype=torch.float64, device="cuda")
    off, size = torch.zeros_like(ref), torch.zeros_like(ref)
    for e in ids.unique().tolist():
        if not 0 <= e < up.shape[0]:
            continue
        t, j = torch.nonzero(ids == e, as_tuple=True)
        W1, W2, w = up[e].double(), down[e].double(), weights[t, j].double()[:, None]
        z, dz = xd[t] @ W1.t(), up.shape[2] * E23 * (xd[t].abs() @ W1.abs().t())
        h, dh = act_of(act, z, dz, H)
        dh = dh + HALF_ULP[up.dtype] * (h.abs() + dh) + TINY[up.dtype]
        y = h @ W2.t()
        dy = dh @ W2.abs().t() + H * E23 * ((h.abs() + dh) @ W2.abs().t())
        ref.index_add_(0, t, w * y)
        off.index_add_(0, t, w.abs() * dy)
        size.index_add_(0, t, (w * y).abs() + w.abs() * dy)
    off += (k + 1) * E24 * size
    bound = off + HALF_ULP[got.dtype] * (ref.abs() + off) + TINY[got.dtype]
    assert torch.isfinite(got).all()
    over = (got.double() - ref).abs() - bound
    assert over.numel() == 0 or over.max().item() <= 0, "off by %g over the bound" % over.max().item()
    return got


# the second list's weights are read in tiles on the tensor cores: few or no tokens an expert, up to 64, 128, 512 of one expert
SMALL = [(1, 1, 1, 8, 8, 8), (1, 2, 16, 3328, 1024, 1024), (2, 1, 3, 16, 24, 40), (3, 4, 5, 40, 72, 8), (7, 3, 12, 1032, 776, 520),
         (8, 8, 1000, 128, 64, 128), (16, 2, 32, 512, 264, 256), (64, 4, 16, 256, 512, 136), (64, 8, 8, 96, 200, 64), (512, 1, 3, 72, 48, 56),
         (100, 5, 1, 64, 32, 24), (8, 64, 7, 64, 56, 72), (33, 2, 1024, 64, 40, 16), (1, 64, 200, 2048, 128, 32), (5, 2, 4, 16, 8, 4104),
         (64, 8, 1000, 16, 24, 40), (512, 1, 1024, 8, 16, 8), (2, 16, 4, 40, 24, 16), (3, 11, 9, 64, 32, 24)]
LARGE = [(64, 8, 8, 520, 1032, 536), (128, 4, 4, 512, 1032, 520), (512, 1, 1, 520, 1160, 512), (8, 4, 32, 1024, 1544, 1032),
         (60, 4, 40, 1032, 776, 1048), (65, 5, 3, 1000, 1000, 1000)]


def in_tiles(T, k, E, D, H, N, act):
    """The library's rule of when tiles are faster, by megabytes of weights and assignments a group."""
    groups = min(T * k, E)
    return groups * H * (D * (2 if act == "swiglu" else 1) + N) * 2e-6 * (0.028 + 0.006 * T * k / groups) > 6


def test_the_lists_are_of_both_kinds():
    for act in ("relu", "swiglu"):
        assert all(in_tiles(*c, act) for c in LARGE) and not any(in_tiles(*c, act) for c in SMALL)


@gpu
@pytest.mark.parametrize("T,k,E,D,H,N", SMALL + LARGE)
@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("dtype,xt", [(BF, F32), (BF, BF), (HF, HF), (HF, F32)])
def test_the_layer(T, k, E, D, H, N, act, dtype, xt):
    out = [None, F32, HF, BF][(T + k + E) % 4]
    check(case(T * k + D, T, k, E, D, H, N, dtype, xt, act, 0.2 if T > 4 else 0.0, [torch.int32, torch.int64][D % 16 // 8]), act, out)
    assert emb.dense_status() == emb.EMB_OK


@gpu
def test_groups_of_every_size():
    # 1 to 70 members of one expert: every number of eights, and one chunk more than a chunk
    for n in list(range(1, 34)) + [40, 63, 64, 65, 70, 128, 129, 200]:
        ids, x, up, down, weights = case(n, n, 2, 4, 64, 32, 24, BF, BF)
        ids[:, 0], ids[:, 1] = 2, -1
        check((ids, x, up, down, weights), "relu")


@gpu
def test_groups_of_every_size_in_tiles():
    for n in [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 255]:
        ids, x, up, down, weights = case(n, n, 2, 64, 1024, 1544, 1032, BF, BF)
        ids[:, 0], ids[:, 1] = 2, -1
        if n > 20:
            ids[3, 1], ids[9, 1] = 63, 0
            weights[3, 1] = weights[9, 1] = 0.5
        assert in_tiles(n, 2, 64, 1024, 1544, 1032, "relu") == (n >= 15)
        check((ids, x, up, down, weights), "relu")


@gpu
@pytest.mark.parametrize("extra", [8, 24])
@pytest.mark.parametrize("T,k,E,D,H,N", [(6, 2, 4, 128, 64, 64), LARGE[0]])
@pytest.mark.parametrize("xt", [F32, BF])
def test_rows_of_any_stride(extra, T, k, E, D, H, N, xt):
    ids, x, up, down, weights = case(1, T, k, E, D, H, N, BF, xt)
    big = torch.full((T, D + extra), float("nan"), device="cuda", dtype=xt)
    big[:, :D] = x
    assert torch.equal(check((ids, big[:, :D], up, down, weights), "gelu"), emb.expert_layer(ids, x, up, down, weights, "gelu"))


@gpu
def test_tokens_without_experts_and_nothing_at_all():
    for T, k, E, D, H, N in ((5, 3, 4, 64, 32, 24), (40, 3, 4, 64, 32, 24), (64, 8, 8, 512, 1024, 2056)):
        ids, x, up, down, weights = case(2, T, k, E, D, H, N, HF, HF)
        ids[T // 2] = -1
        x[T // 2] = float("nan")       # not read
        weights[T // 2] = float("nan")
        assert not check((ids, x, up, down, weights), "silu")[T // 2].any()
        ids[:] = -1
        assert not emb.expert_layer(ids, x * float("nan"), up, down, weights * float("nan")).any()
    none = emb.expert_layer(ids[:0], x[:0], up, down, weights[:0])
    assert none.shape == (0, 2056)


@gpu
@pytest.mark.parametrize("bad", [7, -2, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("T,D,H,N", [(5, 64, 32, 24), (50, 64, 32, 24), (256, 512, 1032, 520)])
def test_ids_out_of_range_are_dropped_and_reported(bad, T, D, H, N):
    ids, x, up, down, weights = case(3, T, 2, 7, D, H, N, BF, BF)
    assert in_tiles(T, 2, 7, D, H, N, "relu") == (T == 256)
    ids[2, 1] = bad
    weights[2, 1] = float("nan")
    got = check((ids, x, up, down, weights), "relu")
    assert emb.dense_status() == emb.EMB_ERR_KEY_RANGE and emb.dense_status() == emb.EMB_OK
    wide = ids.long()
    wide[2, 1] = 2 ** 40 + 3               # its low 32 bits are a valid id
    assert torch.equal(emb.expert_layer(wide, x, up, down, weights), got)
    assert emb.dense_status() == emb.EMB_ERR_KEY_RANGE


@gpu
@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("D,H,N", [(128, 64, 40), (4096, 4096, 4096)])
def test_a_tokens_infinities_and_nans_stay_its_own(act, D, H, N):
    ids, x, up, down, weights = case(4, 20, 2, 3, D, H, N, BF, BF, act)
    assert in_tiles(20, 2, 3, D, H, N, act) == (D == 4096)
    clean = emb.expert_layer(ids, x, up, down, weights, act)
    x[11, 5] = float("nan")
    got = emb.expert_layer(ids, x, up, down, weights, act)
    others = torch.arange(20, device="cuda") != 11
    assert torch.equal(got[others], clean[others]) and torch.isnan(got[11]).all()
    up[:] = torch.where(torch.arange(3, device="cuda")[:, None, None] == 1, float("inf"), up)     # an expert's, those of its tokens
    got = emb.expert_layer(ids, x, up, down, weights, act)
    free = others & (ids != 1).all(1)
    assert free.any() and torch.equal(got[free], clean[free])


@gpu
@pytest.mark.parametrize("T,k,E,D,H,N", [(1, 2, 16, 3328, 1024, 1024), (48, 4, 64, 256, 512, 256), (64, 8, 8, 96, 200, 64)] + LARGE[:3])
def test_results_repeat(T, k, E, D, H, N):
    args = case(5, T, k, E, D, H, N, BF, F32, "swiglu")
    first = emb.expert_layer(*args, "swiglu")
    for _ in range(20):
        assert torch.equal(emb.expert_layer(*args, "swiglu"), first)


@gpu
def test_weights_past_32_bits():
    # 1000 experts of 2200 x 2048: the last one's weights begin past 2^32 elements
    E, D, H, N = 1000, 2048, 2200, 8
    up = torch.zeros(E, H, D, dtype=BF, device="cuda")
    ids = torch.tensor([[E - 1, 0], [E - 1, 1]], device="cuda")
    _, x, part, small, weights = case(6, 2, 2, 2, D, H, N, BF, BF)
    up[-1] = part[0]
    down = torch.zeros(E, N, H, dtype=BF, device="cuda")
    down[-1] = small[0]
    check((ids, x, up, down, weights), "relu", F32)


@gpu
@pytest.mark.parametrize("T,D,H,N", [(16, 256, 128, 64), (40, 256, 128, 64), (256, 512, 1032, 520)])
def test_streams_and_graphs(T, D, H, N):
    args = case(7, T, 2, 8, D, H, N, HF, HF, "gelu")
    assert in_tiles(T, 2, 8, D, H, N, "gelu") == (T == 256)
    ref = emb.expert_layer(*args, "gelu")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = emb.expert_layer(*args, "gelu", stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, ref)
    graphs = []
    for seed in (8, 9):
        a = case(seed, T, 2, 8, D, H, N, HF, HF, "gelu")
        emb.expert_layer(*a, "gelu")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = emb.expert_layer(*a, "gelu")
            again = emb.expert_layer(*a, "silu")
        graphs.append((graph, a, out, again))
    for turn in range(4):
        for graph, a, out, again in graphs:
            a[0].copy_(torch.randint(-1, 8, (T, 2), generator=gen(turn), device="cuda"))
            a[4].uniform_()
            graph.replay()
            assert torch.equal(out, emb.expert_layer(*a, "gelu")) and torch.equal(again, emb.expert_layer(*a, "silu"))


@gpu
@pytest.mark.parametrize("T,k,E,D,H,N", [SMALL[1], (4, 2, 4, 256, 256, 256), (40, 3, 8, 256, 128, 64), LARGE[0], LARGE[1]])
def test_weights_and_ids_that_change_between_calls(T, k, E, D, H, N):
    # the second kernel's first weights and the groups are read before the first kernel's end:
    # what stood in the stream before the call has to be seen, be it a copy or a kernel that lets the next one begin early
    args = [case(40 + i, T, k, E, D, H, N, BF, BF) for i in range(3)]
    refs = [emb.expert_layer(*a) for a in args]
    ids, x, up, down, weights = (t.clone() for t in args[0])

    def put(i):
        for to, t in zip((ids, x, up, down, weights), args[i]):
            to.copy_(t)

    for turn in range(60):
        put(turn % 3)
        assert torch.equal(emb.expert_layer(ids, x, up, down, weights), refs[turn % 3]), turn
    put(0)
    graph, at = torch.cuda.CUDAGraph(), torch.zeros(1, dtype=torch.int64, device="cuda")
    several = [torch.stack([a[j] for a in args]) for j in range(5)]
    with torch.cuda.graph(graph):
        for to, t in zip((ids, x, up, down, weights), several):
            to.copy_(torch.index_select(t, 0, at)[0])
        out = emb.expert_layer(ids, x, up, down, weights)
    for turn in range(30):
        at.fill_(turn % 3)
        graph.replay()
        assert torch.equal(out, refs[turn % 3]), turn


@gpu
def test_weights_straight_from_a_call():
    T, k, E, D, H, N = 4, 2, 4, 256, 256, 128
    ids, x, up, down, weights = case(50, T, k, E, D, H, N, BF, BF)
    for turn in range(20):
        update = torch.randn(E, N, H, generator=gen(turn), device="cuda")
        got = emb.expert_layer(ids, x, up, emb.orthogonalize(update), weights)
        torch.cuda.synchronize()
        assert torch.equal(got, emb.expert_layer(ids, x, up, emb.orthogonalize(update).clone(), weights)), turn


@gpu
@pytest.mark.parametrize("T,k,E,D,H,N", [(8, 4, 16, 1024, 1024, 512), (32, 4, 16, 512, 512, 512), LARGE[0], LARGE[1]])
def test_calls_on_two_streams_at_once(T, k, E, D, H, N):
    jobs = []
    for seed in range(2):
        args = case(20 + seed, T, k, E, D, H, N, BF, F32)
        jobs.append((torch.cuda.Stream(), args, emb.expert_layer(*args)))
    torch.cuda.synchronize()
    got = [[emb.expert_layer(*args, stream=s) for s, args, _ in jobs] for _ in range(20)]
    torch.cuda.synchronize()
    for outs in got:
        for out, (_, _, ref) in zip(outs, jobs):
            assert torch.equal(out, ref)


@gpu
@pytest.mark.parametrize("T,k,E,D,H,N", [(1, 2, 16, 3328, 1024, 1024), (64, 4, 16, 512, 1024, 256), LARGE[1]])
def test_it_is_the_plans_calls_at_once(T, k, E, D, H, N):
    ids, x, up, down, weights = args = case(10, T, k, E, D, H, N, BF, F32, dropped=0.1)
    plan = emb.expert_sort(ids, E)
    hidden = torch.relu(emb.expert_linear(plan, emb.expert_dispatch(plan, x, BF), up))
    out = emb.expert_combine(plan, emb.expert_linear(plan, hidden, down), weights, F32)
    got = check(args, "relu", F32)
    # two roundings of hidden (each of a sum of its own), one of y: 2^-8 of each
    assert (out - got).norm() <= 3 * 2.0 ** -8 * got.norm()


@gpu
def test_a_block_of_the_dense_side():
    # x + dropout(experts(layer_norm(x))): the calls in a row, against 64 bits
    ids, x, up, down, weights = case(11, 40, 2, 8, 256, 128, 256, BF, F32, "swiglu")
    w, b = torch.randn(256, generator=gen(1), device="cuda"), torch.randn(256, generator=gen(2), device="cuda")
    normed = emb.layer_norm(x, w, b)
    y = emb.expert_layer(ids, normed, up, down, weights, "swiglu", dtype=F32)
    check((ids, normed, up, down, weights), "swiglu", F32, out=y)
    z = emb.dropout(y, 0.25, 3, residual=x)
    kept = emb.dropout(torch.ones_like(y), 0.25, 3) != 0
    ref = torch.where(kept, y.double() / 0.75, 0.0) + x.double()
    assert ((z.double() - ref).abs() <= 3 * E24 * (y.double().abs() * 2 + ref.abs())).all()
    assert emb.dense_status() == emb.EMB_OK


@gpu
def test_inputs_that_require_gradients_and_tensors_of_another_device(monkeypatch):
    ids, x, up, down, weights = case(12, 3, 2, 4, 64, 32, 24, BF, F32)
    weights = torch.rand(3, 2, device="cuda").requires_grad_()
    out = emb.expert_layer(ids, x.requires_grad_(), up.requires_grad_(), down.requires_grad_(), weights)
    assert not out.requires_grad
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)      # nothing is launched: the tensors are on 0
    with pytest.raises(ValueError, match="current device"):
        emb.expert_layer(ids, x, up, down, weights)


@gpu
def test_calls_of_several_threads():
    import threading
    jobs = []
    for i, c in enumerate([SMALL[1], (40, 3, 8, 256, 128, 64), LARGE[0], LARGE[1]]):
        args = case(30 + i, *c, BF, F32)
        jobs.append((torch.cuda.Stream(), args, emb.expert_layer(*args)))
    torch.cuda.synchronize()
    wrong = []

    def work(stream, args, ref):
        for _ in range(30):
            out = emb.expert_layer(*args, stream=stream)
            stream.synchronize()
            wrong.extend([] if torch.equal(out, ref) else [1])

    threads = [threading.Thread(target=work, args=job) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@gpu
def test_inputs_freed_while_another_stream_reads_them():
    args = case(13, 40, 2, 8, 1024, 1024, 512, BF, F32)
    ref = emb.expert_layer(*args)
    stream = torch.cuda.Stream()
    for _ in range(20):
        x, ids = args[1].clone(), args[0].clone()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            torch.cuda._sleep(200000)
        out = emb.expert_layer(ids, x, *args[2:], stream=stream)
        del x, ids
        torch.full((40, 1024), float("nan"), device="cuda")      # takes their memory, if it is to be had
        torch.full((40, 2), 5, dtype=torch.int32, device="cuda")
        torch.cuda.current_stream().wait_stream(stream)
        assert torch.equal(out, ref)


def test_refusals_without_a_gpu():
    x, w, up = torch.zeros(3, 16), torch.zeros(3, 2), torch.zeros(4, 8, 16, dtype=BF)
    with pytest.raises(ValueError, match="CUDA"):
        emb.expert_layer(torch.zeros(3, 2, dtype=torch.int32), x, up, up, w)
    n, bad = ctypes.c_size_t(), emb.EMB_ERR_INVALID_ARG
    size = lambda *a: emb.lib.emb_expert_layer_workspace(*a, ctypes.byref(n))  # noqa: E731
    assert size(64, 8, 16, 16, 16) == emb.EMB_OK and n.value % 256 == 0 and n.value >= 512 * 16 * 6
    assert size(0, 8, 16, 16, 16) == emb.EMB_OK and n.value > 0
    for a in ((65, 8, 8, 16, 16), (-1, 1, 8, 16, 16), (1, 0, 8, 16, 16), (1, 65, 8, 16, 16), (1, 1, 8, 12, 16), (1, 1, 8, 16, 0),
              (2 ** 40, 2, 8, 16, 16), (1, 1, 4, 16, 16)):
        assert size(*a) == bad, a
    at = 0x10000
    ok = [at, 4, 3, 2, 4, at, 2, 16, 16, at, at, 2, 8, 16, 0, at, at, 2, at, 1 << 20, None]
    for i, v in ((0, None), (0, at + 2), (1, 2), (2, -1), (2, 300), (3, 0), (4, 0), (4, 1025), (5, at + 8), (5, None), (6, 1), (7, 8), (7, 17),
                 (8, 12), (9, at + 2), (10, None), (11, 0), (12, 4), (13, 4), (14, 4), (14, -1), (15, at + 2), (16, at + 8), (17, 3), (18, None),
                 (18, at + 16), (19, 64)):
        args = list(ok)
        args[i] = v
        assert emb.lib.emb_expert_layer(*args) == bad, (i, v)


REFUSALS = [
    ("int32 or int64", lambda a: dict(ids=a["ids"].float())),
    ("tensors", lambda a: dict(x=a["x"].cpu().numpy())),
    ("activation", lambda a: dict(activation="tanh")),
    ("dtype", lambda a: dict(dtype=torch.float64)),
    ("assignments", lambda a: dict(ids=torch.zeros(257, 2, dtype=torch.int32, device="cuda"))),
    ("up", lambda a: dict(up=a["up"].float())),
    ("down", lambda a: dict(down=a["down"].transpose(1, 2))),
    ("belong", lambda a: dict(down=a["down"].half())),
    ("belong", lambda a: dict(down=a["down"][:3].contiguous())),
    ("belong", lambda a: dict(activation="swiglu")),
    ("multiples of 8", lambda a: dict(down=torch.zeros(4, 12, 8, dtype=BF, device="cuda"))),
    ("x must", lambda a: dict(x=a["x"][:2])),
    ("x must", lambda a: dict(x=a["x"].half())),
    ("x is on", lambda a: dict(x=a["x"].cpu())),
    ("contiguous rows", lambda a: dict(x=torch.zeros(16, 3, device="cuda").t())),
    ("16 bytes", lambda a: dict(x=torch.zeros(3, 17, device="cuda")[:, :16])),
    ("16-byte", lambda a: dict(x=torch.zeros(3, 20, device="cuda")[:, 1:17])),
    ("weights must", lambda a: dict(weights=a["weights"].half())),
    ("weights is on", lambda a: dict(weights=a["weights"].cpu())),
    ("16-byte", lambda a: dict(up=torch.zeros(4 * 8 * 16 + 1, dtype=BF, device="cuda")[1:].reshape(4, 8, 16))),
]


@gpu
@pytest.mark.parametrize("i", range(len(REFUSALS)))
def test_refusals(i):
    what, change = REFUSALS[i]
    args = dict(ids=torch.zeros(3, 2, dtype=torch.int32, device="cuda"), x=torch.zeros(3, 16, device="cuda"),
                up=torch.zeros(4, 8, 16, dtype=BF, device="cuda"), down=torch.zeros(4, 16, 8, dtype=BF, device="cuda"),
                weights=torch.zeros(3, 2, device="cuda"))
    emb.expert_layer(**args)
    args.update(change(args))
    with pytest.raises(ValueError, match=what):
        emb.expert_layer(**args)
