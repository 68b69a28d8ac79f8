"""The expert layer against plain implementations in 64 bits.

Tolerances.  u is half the spacing of the output type relative to 1 (2^-24 fp32,
2^-11 fp16, 2^-8 bf16; fp16 results below 2^-14 are off by 2^-25 at most).  A
result is rounded once, so it is within u |ref| of the fp32 value, and an fp32
sum of n terms in any order is within (n - 1) 2^-24 S of the exact one, where S
is the sum of the terms' magnitudes.  The tensor cores add exact products of
16-bit numbers in fp32 and may truncate where others round: n 2^-23 S.
"""
import ctypes

import numpy as np
import pytest
import torch

import dlrm_sparse_embedding_gb300 as emb
from dlrm_sparse_embedding_gb300._lib import EmbExpertPlan

gpu = pytest.mark.gpu
HALF_ULP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133}
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def make_ids(g, T, k, E, dropped=0.0, dtype=torch.int32):
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda")
    if dropped:
        ids[torch.rand(T, k, generator=g, device="cuda") < dropped] = -1
    return ids.to(dtype)


def plain_plan(ids, E):
    flat = ids.cpu().numpy().reshape(-1).astype(np.int64)
    ok = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(ok, flat, E), kind="stable")
    kept = int(ok.sum())
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[ok], minlength=E))])
    pos = np.full(flat.size, -1)
    pos[order[:kept]] = np.arange(kept)
    src = np.full(flat.size, -1)
    src[:kept] = order[:kept]
    return offsets, src, pos.reshape(ids.shape)


def check_close(got, ref, bound):
    """|got - ref| <= bound, all finite, in 64 bits."""
    got, ref = got.double(), ref.double()
    assert got.shape == ref.shape
    assert torch.isfinite(got).all()
    off = (got - ref).abs() - bound
    assert off.numel() == 0 or off.max().item() <= 0, "off by %g over the bound" % off.max().item()


def out_bound(ref, dtype, total, n, per=2.0 ** -24):
    return HALF_ULP[dtype] * (ref.double().abs() + n * per * total) + n * per * total + TINY[dtype]


# --------------------------------------------------------------------------- #
# the plan
# --------------------------------------------------------------------------- #
PLANS = [(0, 2, 4, 0.0), (1, 1, 1, 0.0), (1, 2, 16, 0.0), (3, 4, 3, 0.5), (37, 8, 64, 0.1), (1000, 3, 7, 0.3),
         (511, 2, 1000, 0.0), (1025, 1, 1024, 0.02), (4096, 2, 32, 0.0), (4097, 2, 33, 0.02), (30000, 4, 64, 0.05),
         (70001, 1, 1, 0.0), (9000, 64, 5, 0.01), (1300001, 2, 130, 0.1), (2000, 2, 8, 1.0)]


@gpu
@pytest.mark.parametrize("T,k,E,dropped", PLANS)
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort_is_the_stable_one(T, k, E, dropped, dtype):
    ids = make_ids(gen(T + k), T, k, E, dropped, dtype)
    plan = emb.expert_sort(ids, E)
    offsets, src, pos = plain_plan(ids, E)
    assert np.array_equal(plan.offsets.cpu().numpy(), offsets)
    assert np.array_equal(plan.src.cpu().numpy(), src)
    assert np.array_equal(plan.pos.cpu().numpy(), pos)
    assert emb.dense_status() == emb.EMB_OK


@gpu
def test_one_expert_takes_everything_and_runs_of_one_expert():
    for E, ids in ((8, torch.full((9000, 2), 5)), (3, torch.arange(3).repeat_interleave(7000).reshape(-1, 1))):
        ids = ids.int().cuda()
        plan = emb.expert_sort(ids, E)
        for got, ref in zip((plan.offsets, plan.src, plan.pos), plain_plan(ids, E)):
            assert np.array_equal(got.cpu().numpy(), ref)


@gpu
@pytest.mark.parametrize("bad", [7, 8, -2, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("T", [5, 20000])
def test_ids_out_of_range_are_dropped_and_reported(bad, T):
    ids = make_ids(gen(3), T, 2, 7)
    ids[T // 2, 1] = bad
    plan = emb.expert_sort(ids, 7)
    for got, ref in zip((plan.offsets, plan.src, plan.pos), plain_plan(ids, 7)):
        assert np.array_equal(got.cpu().numpy(), ref)
    assert emb.dense_status() == emb.EMB_ERR_KEY_RANGE
    assert emb.dense_status() == emb.EMB_OK      # cleared
    if bad > 0:
        wide = ids.long()
        wide[T // 2, 1] = 2 ** 40 + 3            # its low 32 bits are a valid id
        plan = emb.expert_sort(wide, 7)
        assert plan.pos[T // 2, 1].item() == -1
        assert emb.dense_status() == emb.EMB_ERR_KEY_RANGE


# --------------------------------------------------------------------------- #
# dispatch and combine
# --------------------------------------------------------------------------- #
ROWS = [(1, 1, 1, 8, 0.0), (1, 2, 4, 3328, 0.0), (5, 3, 4, 1, 0.2), (37, 4, 8, 777, 0.1), (64, 8, 16, 64, 0.0),
        (200, 2, 5, 2056, 0.3), (1000, 5, 64, 136, 0.1), (33, 64, 3, 40, 0.2), (6, 2, 3, 48, 1.0), (3000, 2, 9, 30, 0.0)]


def routed(seed, T, k, E, dropped):
    g = gen(seed)
    ids = make_ids(g, T, k, E, dropped)
    if T > 1 and dropped:
        ids[T // 2] = -1     # a token without experts
    plan = emb.expert_sort(ids, E)
    _, src, pos = plain_plan(ids, E)
    return g, plan, torch.from_numpy(src).cuda(), torch.from_numpy(pos).cuda(), int(plan.offsets[-1])


def padded(t, extra, fill=float("nan")):
    """The same matrix with a row stride `extra` elements longer, `fill` between the rows."""
    big = torch.full((t.shape[0], t.shape[1] + extra), fill, dtype=t.dtype, device=t.device)
    big[:, :t.shape[1]] = t
    return big[:, :t.shape[1]]


@gpu
@pytest.mark.parametrize("T,k,E,width,dropped", ROWS)
@pytest.mark.parametrize("xt,rt", [(F32, BF), (BF, BF), (HF, HF), (F32, F32), (F32, HF), (BF, F32)])
@pytest.mark.parametrize("extra", [0, 8, 5])
def test_dispatch_and_its_gradient(T, k, E, width, dropped, xt, rt, extra):
    g, plan, src, pos, kept = routed(T * k, T, k, E, dropped)
    x = padded(normal(g, T, width, dtype=xt), extra)
    rows = emb.expert_dispatch(plan, x, dtype=rt)
    ref = torch.zeros(T * k, width, dtype=rt, device="cuda")
    ref[:kept] = x[src[:kept] // k].to(rt)      # a copy, or one rounding to nearest even
    assert torch.equal(rows, ref)
    dr = padded(normal(g, T * k, width, dtype=rt), extra)
    dr[kept:] = float("nan")                    # not read
    dx = emb.expert_dispatch_grad(plan, dr, dtype=xt)
    picked = torch.where((pos >= 0)[:, :, None], dr.double()[pos.clamp(min=0)], 0.0)
    check_close(dx, picked.sum(1), out_bound(picked.sum(1), xt, picked.abs().sum(1), k))


@gpu
@pytest.mark.parametrize("T,k,E,width,dropped", ROWS)
@pytest.mark.parametrize("rt,ot", [(BF, BF), (HF, HF), (F32, F32), (BF, F32), (HF, BF)])
@pytest.mark.parametrize("extra", [0, 8, 3])
def test_combine_and_its_gradients(T, k, E, width, dropped, rt, ot, extra):
    g, plan, src, pos, kept = routed(T * k + 1, T, k, E, dropped)
    rows = padded(normal(g, T * k, width, dtype=rt), extra)
    rows[kept:] = float("nan")                  # not read
    w = torch.rand(T, k, generator=g, device="cuda") - 0.25
    w[pos < 0] = float("nan")                   # the weight of an assignment without an expert is not used
    out = emb.expert_combine(plan, rows, w, dtype=ot)
    has = (pos >= 0)[:, :, None]
    y = torch.where(has, rows.double()[pos.clamp(min=0)], 0.0)
    wd = torch.where(pos >= 0, w.double(), 0.0)
    terms = y * wd[:, :, None]
    check_close(out, terms.sum(1), out_bound(terms.sum(1), ot, terms.abs().sum(1), k))
    go = padded(normal(g, T, width, dtype=ot), extra)
    drows, dw = emb.expert_combine_grad(plan, go, rows, w)
    assert drows.dtype == rt and dw.dtype == F32
    ref = torch.zeros(T * k, width, dtype=torch.float64, device="cuda")
    at = src[:kept]
    ref[:kept] = go.double()[at // k] * wd.reshape(-1)[at][:, None]
    check_close(drows, ref, out_bound(ref, rt, ref.abs(), 1))
    dots = y * go.double()[:, None, :]
    check_close(dw, dots.sum(2), out_bound(dots.sum(2), F32, dots.abs().sum(2), width))


@gpu
@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_gradients_are_the_differences(dtype):
    # small whole numbers: every product and sum is exact, and so is a central
    # difference of these functions, each linear in each argument
    g, plan, src, pos, kept = routed(8, 40, 3, 5, 0.1)
    ints = lambda *shape: torch.randint(-3, 4, shape, generator=g, device="cuda").to(dtype)  # noqa: E731
    x, dx, gr = ints(40, 24), ints(40, 24), ints(120, 24)
    gr[kept:] = 0
    f = lambda v: emb.expert_dispatch(plan, v).double()  # noqa: E731
    assert ((f(x + dx) - f(x - dx)) / 2 * gr.double()).sum() == (emb.expert_dispatch_grad(plan, gr, dtype=F32).double() * dx.double()).sum()
    rows, drows, go = ints(120, 24), ints(120, 24), ints(40, 24)
    rows[kept:], drows[kept:] = 0, 0
    w, dw = ints(40, 3).float(), ints(40, 3).float()
    gw_rows, gw = emb.expert_combine_grad(plan, go, rows, w)
    c = lambda r, v: emb.expert_combine(plan, r, v, dtype=F32).double()  # noqa: E731
    assert ((c(rows + drows, w) - c(rows - drows, w)) / 2 * go.double()).sum() == (gw_rows.double() * drows.double()).sum()
    assert ((c(rows, w + dw) - c(rows, w - dw)) / 2 * go.double()).sum() == (gw.double() * dw.double()).sum()


# --------------------------------------------------------------------------- #
# the products
# --------------------------------------------------------------------------- #
LINEAR = [(1, 1, 1, 8, 8, 0.0), (1, 2, 16, 3328, 1024, 0.0), (2, 2, 4, 200, 136, 0.0), (9, 4, 64, 256, 512, 0.0),
          (48, 4, 64, 1024, 264, 0.1), (127, 1, 1, 64, 64, 0.0), (129, 1, 2, 72, 520, 0.0), (300, 2, 3, 1032, 776, 0.3),
          (700, 2, 40, 128, 256, 0.02), (2000, 1, 5, 512, 384, 0.0), (1500, 3, 4, 264, 1040, 0.1), (40, 2, 8, 64, 64, 1.0)]


def linear_case(T, k, E, K, N, dropped, dtype, extra=0, skew=False):
    g = gen(T + K)
    ids = make_ids(g, T, k, E, dropped)
    if skew:
        ids[(ids >= 0) & (torch.rand(T, k, generator=g, device="cuda") < 0.7)] = E // 2
        ids[ids == 0] = E - 1      # expert 0 is left without rows
    plan = emb.expert_sort(ids, E)
    off = plan.offsets.tolist()
    x = padded(normal(g, T * k, K, dtype=dtype), extra)
    gy = padded(normal(g, T * k, N, dtype=dtype), extra)
    w = normal(g, E, N, K, dtype=dtype)
    x[off[-1]:], gy[off[-1]:] = float("nan"), float("inf")    # not read
    return plan, off, x, gy, w


@gpu
@pytest.mark.parametrize("T,k,E,K,N,dropped", LINEAR)
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("extra,skew", [(0, False), (8, False), (0, True)])
def test_linear_and_its_gradients(T, k, E, K, N, dropped, dtype, extra, skew):
    plan, off, x, gy, w = linear_case(T, k, E, K, N, dropped, dtype, extra, skew)
    y = emb.expert_linear(plan, x, w)
    dx, dw = emb.expert_linear_grad(plan, gy, x, w)
    assert emb.dense_status() == emb.EMB_OK
    per = 2.0 ** -23
    for e in range(E):
        a, b = off[e], off[e + 1]
        xe, ge, we = x[a:b].double(), gy[a:b].double(), w[e].double()
        for got, p, q, n in ((y[a:b], xe, we.t(), K), (dx[a:b], ge, we, N), (dw[e], ge.t(), xe, b - a)):
            ref, total = p @ q, p.abs() @ q.abs()
            check_close(got, ref, out_bound(ref, dtype, total, n, per))
    assert not y[off[-1]:].any() and not dx[off[-1]:].any()


@gpu
@pytest.mark.parametrize("T,k,E,K,N", [(20000, 1, 3, 136, 2056), (9000, 2, 7, 1032, 776), (30000, 2, 200, 72, 264), (3, 2, 1024, 64, 4096)])
def test_linear_in_many_tiles(T, k, E, K, N):
    # pairs and single CTAs, several rounds of tiles, last rounds of halves
    plan, off, x, gy, w = linear_case(T, k, E, K, N, 0.05, BF, skew=E < 100)
    y = emb.expert_linear(plan, x, w)
    dx, dw = emb.expert_linear_grad(plan, gy, x, w)
    for e in range(0, E, max(1, E // 7)):
        a, b = off[e], off[e + 1]
        xe, ge, we = x[a:b].double(), gy[a:b].double(), w[e].double()
        for got, p, q, n in ((y[a:b], xe, we.t(), K), (dx[a:b], ge, we, N), (dw[e], ge.t(), xe, b - a)):
            ref, total = p @ q, p.abs() @ q.abs()
            check_close(got, ref, out_bound(ref, BF, total, n, 2.0 ** -23))
    assert not y[off[-1]:].any() and not dx[off[-1]:].any()
    assert emb.dense_status() == emb.EMB_OK


@gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T", [6, 500])
def test_linear_keeps_groups_apart_whatever_they_hold(dtype, T):
    # 16-bit rows of one expert, infinite and NaN, beside the others'
    plan, off, x, gy, w = linear_case(T, 2, 3, 128, 72, 0.0, dtype)
    clean_x, clean_g = x.clone(), gy.clone()
    x[off[1]:off[2]] = float("nan")
    gy[off[1]:off[2]] = float("inf")
    y, yc = emb.expert_linear(plan, x, w), emb.expert_linear(plan, clean_x, w)
    (dx, dw), (dxc, dwc) = emb.expert_linear_grad(plan, gy, x, w), emb.expert_linear_grad(plan, clean_g, clean_x, w)
    keep = torch.ones(2 * T, dtype=torch.bool, device="cuda")
    keep[off[1]:off[2]] = False
    assert torch.equal(y[keep], yc[keep]) and torch.equal(dx[keep], dxc[keep])
    assert torch.equal(dw[0], dwc[0]) and torch.equal(dw[2], dwc[2])
    assert off[1] == off[2] or (torch.isnan(y[~keep]).all() and torch.isnan(dw[1]).all())


@gpu
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T,E", [(3, 2), (300, 4)])
def test_linear_gradients_are_the_differences(dtype, T, E):
    g = gen(5)
    plan = emb.expert_sort(make_ids(g, T, 2, E, 0.1), E)
    ints = lambda *shape: torch.randint(-1, 2, shape, generator=g, device="cuda").to(dtype)  # noqa: E731
    kept = int(plan.offsets[-1])
    x, dx, gy, w, dw = ints(2 * T, 64), ints(2 * T, 64), ints(2 * T, 72), ints(E, 72, 64), ints(E, 72, 64)
    for t in (x, dx, gy):
        t[kept:] = 0
    # sums of up to 64 (72, 256) products of at most 2 in magnitude are whole and at most 256: exact in both types
    grad_x, grad_w = emb.expert_linear_grad(plan, gy, x, w)
    f = lambda r, v: emb.expert_linear(plan, r, v).double()  # noqa: E731
    if T <= 128 or dtype == HF:
        assert ((f(x, w + dw) - f(x, w - dw)) / 2 * gy.double()).sum() == (grad_w.double() * dw.double()).sum()
    assert ((f(x + dx, w) - f(x - dx, w)) / 2 * gy.double()).sum() == (grad_x.double() * dx.double()).sum()


@gpu
def test_calls_repeat_bit_for_bit_and_run_on_other_streams():
    plan, off, x, gy, w = linear_case(900, 2, 6, 512, 264, 0.05, BF)
    x[off[-1]:], gy[off[-1]:] = 0, 0
    g = gen(1)
    tokens, weights = normal(g, 900, 512), torch.rand(900, 2, generator=g, device="cuda")

    def everything(stream=None):
        q = emb.expert_sort(make_ids(gen(2), 900, 2, 6, 0.1), 6, stream=stream)
        rows = emb.expert_dispatch(q, tokens, BF, stream=stream)
        y = emb.expert_linear(q, rows, w, stream=stream)
        out = emb.expert_combine(q, y, weights, stream=stream)
        dy, dwt = emb.expert_combine_grad(q, out, y, weights, stream=stream)
        dr, dw = emb.expert_linear_grad(q, dy, rows, w, stream=stream)
        return out, dwt, dw, emb.expert_dispatch_grad(q, dr, F32, stream=stream)

    first = everything()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):       # the ids are made on the stream that sorts them
        second = everything()
    other.synchronize()
    third = everything()
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)


@gpu
def test_a_graph_captures_the_layer():
    plan, off, x, gy, w = linear_case(600, 2, 6, 256, 136, 0.0, BF)
    ids = make_ids(gen(9), 600, 2, 6)
    tokens, weights = normal(gen(1), 600, 256), torch.rand(600, 2, device="cuda")

    def step():
        q = emb.expert_sort(ids, 6)
        rows = emb.expert_dispatch(q, tokens, BF)
        y = emb.expert_linear(q, rows, w)
        return emb.expert_combine(q, y, weights), emb.expert_linear_grad(q, y, rows, w)[1]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    ids.copy_(make_ids(gen(10), 600, 2, 6))      # another routing in the same graph
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, step()):
        assert torch.equal(a, b)


@gpu
def test_rows_past_32_bits_of_elements():
    # 2.2e9 elements: row offsets do not fit 32 bits
    T, width = 70000, 31500
    ids = torch.arange(T, device="cuda").flip(0).remainder(2).int().reshape(T, 1)
    plan = emb.expert_sort(ids, 2)
    x = torch.empty(T, width, dtype=BF, device="cuda")
    x[:] = (torch.arange(T, device="cuda") % 251).to(BF)[:, None]
    rows = emb.expert_dispatch(plan, x)
    back = emb.expert_combine(plan, rows, torch.ones(T, 1, device="cuda"))
    assert torch.equal(rows[:, -1], x[plan.src.long(), 0])
    assert torch.equal(back[-3:], x[-3:]) and torch.equal(back[:, 0], x[:, 0])


# --------------------------------------------------------------------------- #
# refusals
# --------------------------------------------------------------------------- #
def meta(*shape, dtype=torch.int32):
    return torch.empty(*shape, dtype=dtype)


@pytest.mark.parametrize("ids,E,match", [
    (meta(3, 2, dtype=torch.int16), 4, "ids"), (meta(6), 4, "ids"), ([[0]], 4, "ids"),
    (meta(2, 3).t(), 4, "contiguous"), (meta(3, 2), 4, "CUDA"),
])
def test_sort_refuses(ids, E, match):
    with pytest.raises(ValueError, match=match):
        emb.expert_sort(ids, E)


@pytest.mark.parametrize("offsets,src,pos,match", [
    (meta(5, dtype=torch.int64), meta(6), meta(3, 2), "offsets"), (meta(5), meta(6), meta(6), "pos"),
    (meta(5), meta(6), meta(3, 2), "CUDA"),
])
def test_a_plan_refuses(offsets, src, pos, match):
    with pytest.raises(ValueError, match=match):
        emb.ExpertPlan(offsets, src, pos)


@gpu
def test_calls_refuse_what_does_not_fit():
    plan = emb.expert_sort(make_ids(gen(0), 6, 2, 4), 4)
    z = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    w, wt = z(4, 16, 24), z(6, 2, dtype=F32)
    bad = [
        lambda: emb.expert_sort(z(6, 2, dtype=torch.int32), 0), lambda: emb.expert_sort(z(6, 2, dtype=torch.int32), 1025),
        lambda: emb.expert_sort(z(6, 65, dtype=torch.int32), 4), lambda: emb.expert_sort(z(6, 0, dtype=torch.int32), 4),
        lambda: emb.ExpertPlan(plan.offsets, plan.src[:-1], plan.pos),
        lambda: emb.expert_dispatch(plan, z(5, 8)), lambda: emb.expert_dispatch(plan, z(6, 8, dtype=torch.float64)),
        lambda: emb.expert_dispatch(plan, z(6, 8), dtype=torch.int32), lambda: emb.expert_dispatch(plan, z(8, 6).t()),
        lambda: emb.expert_dispatch(plan, z(8).expand(6, 8)), lambda: emb.expert_dispatch(plan, z(6, 0)),
        lambda: emb.expert_dispatch(plan, torch.zeros(6, 8)), lambda: emb.expert_dispatch("plan", z(6, 8)),
        lambda: emb.expert_dispatch_grad(plan, z(6, 8)),
        lambda: emb.expert_combine(plan, z(12, 8), z(6, 2)), lambda: emb.expert_combine(plan, z(12, 8), wt[:5]),
        lambda: emb.expert_combine(plan, z(11, 8), wt), lambda: emb.expert_combine(plan, z(12, 8), wt.t().contiguous().t()),
        lambda: emb.expert_combine_grad(plan, z(6, 7), z(12, 8), wt), lambda: emb.expert_combine_grad(plan, z(12, 8), z(12, 8), wt),
        lambda: emb.expert_linear(plan, z(12, 24), z(3, 16, 24)), lambda: emb.expert_linear(plan, z(12, 23), w),
        lambda: emb.expert_linear(plan, z(12, 24, dtype=HF), w), lambda: emb.expert_linear(plan, z(12, 25)[:, 1:], w),
        lambda: emb.expert_linear(plan, z(12, 24, dtype=F32), z(4, 16, 24, dtype=F32)),
        lambda: emb.expert_linear(plan, z(12, 20), z(4, 16, 20)), lambda: emb.expert_linear(plan, z(12, 24), z(4, 12, 24)),
        lambda: emb.expert_linear(plan, z(12, 24), z(4, 24, 16).transpose(1, 2)),
        lambda: emb.expert_linear(plan, z(11, 24), w), lambda: emb.expert_linear_grad(plan, z(12, 24), z(12, 24), w),
        lambda: emb.expert_linear_grad(plan, z(12, 16), z(12, 16), w), lambda: emb.expert_linear_grad(plan, z(12, 16), None, w),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail("call %d was taken" % i)
    # one gradient alone
    dx, dw = emb.expert_linear_grad(plan, z(12, 16), None, w, need_weight=False)
    assert dw is None and dx.shape == (12, 24)


def _no_cuda():
    return not torch.cuda.is_available()


# The addresses below are of no allocation: the host checks reject each call
# before anything is enqueued, and the test runs only where there is no GPU.
@pytest.mark.skipif(not _no_cuda(), reason="host-only check: runs where no GPU is present")
def test_the_library_refuses_on_the_host():
    L, bad = emb.lib, emb.EMB_ERR_INVALID_ARG
    n = ctypes.c_size_t()
    for T, k, E in ((-1, 2, 4), (4, 0, 4), (4, 65, 4), (4, 2, 0), (4, 2, 1025), (2 ** 30, 2, 4)):
        assert L.emb_expert_sort_workspace(T, k, E, ctypes.byref(n)) == bad
    assert L.emb_expert_sort_workspace(4, 2, 4, None) == bad
    sizes = []
    for T in (0, 1, 5000, 100000, 2 ** 30 - 1):
        assert L.emb_expert_sort_workspace(T, 2, 64, ctypes.byref(n)) == emb.EMB_OK
        sizes.append(n.value)
    assert sizes == sorted(sizes) and all(s % 256 == 0 and s > 0 for s in sizes)
    ok = dict(offsets=0x1000, src=0x2000, pos=0x3000, tokens=4, k=2, experts=4)
    plan = lambda **over: ctypes.byref(EmbExpertPlan(*dict(ok, **over).values()))  # noqa: E731
    p = plan()
    for over in (dict(offsets=0), dict(src=0), dict(pos=0), dict(offsets=0x1002), dict(pos=0x3001), dict(tokens=-1), dict(k=0),
                 dict(experts=0), dict(tokens=2 ** 31)):
        assert L.emb_expert_dispatch(plan(**over), 0x4000, 0, 8, 8, 0x5000, 0, None) == bad, over
    assert L.emb_expert_sort(0x4000, 2, p, 0x10000, 4096, None) == bad
    assert L.emb_expert_sort(0x4002, 4, p, 0x10000, 4096, None) == bad
    assert L.emb_expert_sort(0x4000, 4, p, 0x10010, 4096, None) == bad
    assert L.emb_expert_sort(0x4000, 4, p, 0x10000, 255, None) == bad
    assert L.emb_expert_sort(None, 4, p, 0x10000, 4096, None) == bad
    assert L.emb_expert_dispatch(p, 0x4000, 3, 8, 8, 0x5000, 0, None) == bad       # type
    assert L.emb_expert_dispatch(p, 0x4000, 0, 7, 8, 0x5000, 0, None) == bad       # stride below the width
    assert L.emb_expert_dispatch(p, 0x4000, 0, 8, 0, 0x5000, 0, None) == bad       # no width
    assert L.emb_expert_dispatch(p, 0x4002, 0, 8, 8, 0x5000, 0, None) == bad       # misaligned
    assert L.emb_expert_dispatch_grad(p, None, 0, 8, 8, 0x5000, 0, None) == bad
    assert L.emb_expert_combine(p, 0x4000, 1, 8, None, 8, 0x5000, 1, None) == bad
    assert L.emb_expert_combine_grad(p, 0x4000, 1, 8, 0x6000, 1, 8, 0x7000, 8, 0x8000, None, None) == bad
    for args in ((p, 0x4000, 24, 0x5000, 24, 16, 0, 0x6000), (p, 0x4000, 24, 0x5000, 20, 16, 1, 0x6000),
                 (p, 0x4000, 24, 0x5000, 24, 12, 1, 0x6000), (p, 0x4008, 24, 0x5000, 24, 16, 1, 0x6000),
                 (p, 0x4000, 25, 0x5000, 24, 16, 1, 0x6000), (p, 0x4000, 24, 0x5008, 24, 16, 1, 0x6000),
                 (p, 0x4000, 24, None, 24, 16, 1, 0x6000), (None, 0x4000, 24, 0x5000, 24, 16, 1, 0x6000)):
        assert L.emb_expert_linear(*args, None) == bad, args
    assert L.emb_expert_linear_grad_rows(p, 0x4000, 16, 0x5000, 24, 16, 2, 0x6004, None) == bad
    assert L.emb_expert_linear_grad_weight(p, 0x4000, 16, 0x5000, 20, 24, 16, 2, 0x6000, None) == bad


@gpu
def test_inputs_freed_while_another_stream_still_reads_them():
    g = gen(77)
    E, side = 4, torch.cuda.Stream()
    ids, x = make_ids(g, 700, 2, E), normal(g, 700, 264, dtype=BF)
    update = normal(g, 200, 136)
    ref, orthogonal = emb.expert_dispatch(emb.expert_sort(ids, E), x), emb.orthogonalize(update)
    for _ in range(2):                                # the first time, kernels are loaded
        copies = [ids.clone(), x.clone(), update.clone()]
        plan = emb.expert_sort(copies[0], E)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)
        again = emb.expert_sort(copies[0], E, stream=side)
        rows = emb.expert_dispatch(plan, copies[1], stream=side)
        result = emb.orthogonalize(copies[2], stream=side)
        shapes = [(t.shape, t.dtype) for t in copies + [plan.offsets, plan.src, plan.pos]]
        del copies, plan
        keep = [torch.full(shape, 1, dtype=dtype, device="cuda") for shape, dtype in shapes for _ in range(8)]
        torch.cuda.synchronize()
        assert len(keep) == 8 * len(shapes)
        assert torch.equal(rows, ref) and torch.equal(result, orthogonal)
        assert torch.equal(emb.expert_dispatch(again, x), ref)


@gpu
@pytest.mark.parametrize("width", [32, 56, 64, 65, 120, 128, 136, 200, 256, 264, 519, 1025, 2064])
@pytest.mark.parametrize("k", [1, 2, 6])
@pytest.mark.parametrize("T", [50, 1500])
def test_rows_of_many_widths(T, k, width):
    for extra in (0, 8, 3):
        test_dispatch_and_its_gradient(T, k, 7, width, 0.1, F32, BF, extra)
        test_combine_and_its_gradients(T, k, 7, width, 0.1, HF, F32, extra)


@gpu
@pytest.mark.parametrize("T,width", [(600011, 9), (2200003, 8), (600011, 40)])   # more than blocks take at once
def test_very_many_short_rows(T, width):
    test_dispatch_and_its_gradient(T, 1, 3, width, 0.01, BF, BF, 0)
    test_combine_and_its_gradients(T, 1, 3, width, 0.01, BF, BF, 0)


@gpu
@pytest.mark.parametrize("width", [2, 34, 130, 514, 1026, 2058])
@pytest.mark.parametrize("types", [(F32, BF), (HF, HF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("k", [1, 2, 3])
def test_rows_of_even_widths(width, types, k):
    for extra in (0, 2, 5):
        test_dispatch_and_its_gradient(700, k, 7, width, 0.1, *types, extra)
        test_combine_and_its_gradients(700, k, 7, width, 0.1, types[1], types[0], extra)


@gpu
@pytest.mark.parametrize("T,k,E,K,N", [(1777, 2, 12, 1032, 776), (9000, 2, 7, 1032, 776), (2000, 1, 5, 512, 384)])
def test_weight_gradients_of_ragged_groups_repeat_bit_for_bit(T, k, E, K, N):
    # pairs of CTAs zero the rows past a group, each its own half, before one of them multiplies both
    plan, off, x, gy, w = linear_case(T, k, E, K, N, 0.05, BF, skew=True)
    first = emb.expert_linear_grad(plan, gy, x, w, need_rows=False)[1]
    for _ in range(30):
        assert torch.equal(emb.expert_linear_grad(plan, gy, x, w, need_rows=False)[1], first)
    for e in range(E):
        a, b = off[e], off[e + 1]
        p, q = gy[a:b].double().t(), x[a:b].double()
        check_close(first[e], p @ q, out_bound(p @ q, BF, p.abs() @ q.abs(), b - a, 2.0 ** -23))
    assert emb.dense_status() == emb.EMB_OK


@gpu
@pytest.mark.parametrize("P", [4096, 65536, 262144])
def test_long_sums_of_one_sign(P):
    # a cut after every 16 products, below fp32's last bit of the running sum (2^-23 of it), then one rounding
    g = gen(P)
    plan = emb.expert_sort(torch.zeros(P, 1, dtype=torch.int32, device="cuda"), 1)
    x, gy = ((torch.rand(P, n, generator=g, device="cuda") * (4 / P) ** 0.5).to(HF) for n in (136, 264))
    got = emb.expert_linear_grad(plan, gy, x, torch.zeros(1, 264, 136, dtype=HF, device="cuda"), need_rows=False)[1][0]
    ref = gy.double().t() @ x.double()
    check_close(got, ref, out_bound(ref, HF, ref, P / 16, 2.0 ** -23))
