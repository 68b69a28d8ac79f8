"""Orthogonalised updates against Newton-Schulz steps in 64 bits.

Tolerance.  The output is bf16: its rounding alone is 1.7e-3 of the result's
2-norm (2^-8 / sqrt(12) over the mean of a significand).  Between the steps A
and B are rounded to fp16; the same steps in 64 bits with exactly those
roundings put in are at most 1.3e-3 off, over flat, power-law and
low-rank-plus-noise spectra.  Together 2.1e-3; the bound is twice that, for
sizes and spectra that were not emulated.  fp32 sums add far less.
"""
import ctypes

import pytest
import torch

import dlrm_sparse_embedding_gb300 as emb

gpu = pytest.mark.gpu
BOUND = 4.2e-3
ABC = (3.4445, -4.7750, 2.0315)
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def plain(G, steps=5, abc=ABC, eps=1e-7):
    a, b, c = abc
    out = []
    for M in G.double():
        X = M / (torch.linalg.norm(M) + eps)
        for _ in range(steps):
            if X.shape[0] <= X.shape[1]:
                A = X @ X.T
                X = a * X + (b * A + c * A @ A) @ X
            else:
                A = X.T @ X
                X = a * X + X @ (b * A + c * A @ A)
        out.append(X)
    return torch.stack(out)


def matrices(seed, batch, rows, cols, kind, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    if kind == "flat":
        G = r(batch, rows, cols)
    elif kind == "decay":
        n = min(rows, cols)
        G = r(batch, rows, n) * torch.arange(1, n + 1, device="cuda").float().pow(-1.0) @ r(batch, n, cols)
    else:                                        # a few directions over noise
        n = min(rows, cols, 8)
        G = r(batch, rows, n) @ r(batch, n, cols) + 0.05 * r(batch, rows, cols)
    return (G * 1e-2).to(dtype)


def off(got, ref):
    assert got.dtype == BF and torch.isfinite(got).all()
    return ((got.double() - ref).norm() / ref.norm()).item()


SIZES = [(1, 1, 1), (1, 1, 9), (2, 7, 1), (3, 5, 5), (2, 64, 64), (2, 65, 63), (1, 128, 256), (5, 100, 333), (1, 519, 177),
         (2, 256, 1024), (1, 700, 700), (3, 129, 130), (1, 1030, 260), (1, 40, 5000)]


@gpu
@pytest.mark.parametrize("batch,rows,cols", SIZES)
@pytest.mark.parametrize("kind", ["flat", "decay", "lowrank"])
@pytest.mark.parametrize("dtype", [BF, F32, HF])
def test_against_64_bits(batch, rows, cols, kind, dtype):
    G = matrices(rows + cols, batch, rows, cols, kind, dtype)
    got = emb.orthogonalize(G)
    assert got.shape == G.shape and got.is_contiguous()
    ref = plain(G)
    for i in range(batch):
        assert off(got[i], ref[i]) <= BOUND, i
    assert emb.dense_status() == emb.EMB_OK


@gpu
@pytest.mark.parametrize("batch,rows,cols", [(24, 300, 500), (12, 1024, 2600), (2, 2600, 700), (40, 130, 65), (300, 20, 90)])
def test_many_tiles_at_once(batch, rows, cols):
    # several rounds of tiles of each width, matrices that run into each other's products
    G = matrices(batch, batch, rows, cols, "decay", BF)
    got, ref = emb.orthogonalize(G), plain(G)
    assert max(off(got[i], ref[i]) for i in range(batch)) <= BOUND
    assert torch.equal(got, emb.orthogonalize(G))      # and the same again
    assert emb.dense_status() == emb.EMB_OK


@gpu
def test_a_graph_captures_the_steps():
    for rows, cols in ((100, 300), (300, 200)):
        G = matrices(1, 2, rows, cols, "flat", F32)
        emb.orthogonalize(G)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = emb.orthogonalize(G)
        G.copy_(matrices(2, 2, rows, cols, "decay", F32))
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, emb.orthogonalize(G))


@gpu
@pytest.mark.parametrize("steps", [1, 2, 3, 8])
@pytest.mark.parametrize("rows,cols", [(96, 200), (200, 96)])
def test_steps_and_coefficients(steps, rows, cols):
    G = matrices(1, 2, rows, cols, "decay", BF)
    assert off(emb.orthogonalize(G, steps=steps), plain(G, steps)) <= BOUND
    abc = (1.875, -1.25, 0.375)                  # the convergent quintic
    assert off(emb.orthogonalize(G, steps=steps, coefficients=abc), plain(G, steps, abc)) <= BOUND
    assert off(emb.orthogonalize(G, steps=steps, eps=0.5), plain(G, steps, eps=0.5)) <= BOUND


@gpu
def test_singular_values_end_near_one():
    s = torch.linalg.svdvals(emb.orthogonalize(matrices(3, 1, 256, 512, "flat", BF))[0].double())
    assert 0.6 < s.min() and s.max() < 1.3


@gpu
@pytest.mark.parametrize("dtype,scale", [(F32, 1e-18), (F32, 1e-6), (F32, 1e15), (F32, 1e30), (BF, 1e-6), (BF, 1e30), (HF, 1e3)])
def test_size_does_not_matter(dtype, scale):
    G = (matrices(4, 2, 64, 96, "decay", F32) * scale).to(dtype)
    assert off(emb.orthogonalize(G, eps=0.0), plain(G, eps=0.0)) <= BOUND


@gpu
def test_zero_and_broken_matrices_stay_by_themselves():
    G = matrices(5, 4, 72, 40, "flat", BF)
    clean = emb.orthogonalize(G)
    G[1] = 0
    G[2, 3, 5] = float("inf")
    G[3, 0, 0] = float("nan")
    got = emb.orthogonalize(G)
    assert torch.equal(got[0], clean[0])
    assert not got[1].any()
    assert torch.isnan(got[2]).all() and torch.isnan(got[3]).all()
    assert torch.isnan(emb.orthogonalize(torch.zeros(1, 4, 4, device="cuda"), eps=0.0)).all()   # 0 / 0, as the formula says


@gpu
def test_strides_streams_and_out():
    big = matrices(6, 3, 80, 160, "flat", F32)
    view = big[::2, 3:70, 5:90]
    ref = emb.orthogonalize(view.contiguous())
    assert torch.equal(emb.orthogonalize(view), ref)
    one = emb.orthogonalize(view[1])
    assert torch.equal(one, ref[1])
    out = torch.empty(2, 67, 85, dtype=BF, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert emb.orthogonalize(view, out=out, stream=side) is out
    side.synchronize()
    assert torch.equal(out, ref)
    assert emb.orthogonalize(big[:0]).shape == (0, 80, 160)


@gpu
def test_refusals():
    z = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    bad = [lambda: emb.orthogonalize(z(4)), lambda: emb.orthogonalize(z(4, 4, dtype=torch.float64)),
           lambda: emb.orthogonalize(z(4, 6).t()), lambda: emb.orthogonalize(z(6).expand(4, 6)),
           lambda: emb.orthogonalize(z(0, 4)), lambda: emb.orthogonalize(z(4, 4), steps=0),
           lambda: emb.orthogonalize(z(4, 4), steps=33), lambda: emb.orthogonalize(z(4, 4), coefficients=(1.0, 2.0)),
           lambda: emb.orthogonalize(z(4, 4), eps=-1.0), lambda: emb.orthogonalize(z(4, 4), eps=float("nan")),
           lambda: emb.orthogonalize(z(4, 4), out=z(4, 4, dtype=F32)), lambda: emb.orthogonalize(z(4, 4), out=z(4, 5)),
           lambda: emb.orthogonalize(torch.zeros(4, 4))]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail("call %d was taken" % i)


@pytest.mark.skipif(torch.cuda.is_available(), reason="host-only check: runs where no GPU is present")
def test_the_library_refuses_on_the_host():
    L, bad = emb.lib, emb.EMB_ERR_INVALID_ARG
    n = ctypes.c_size_t()
    for b, r, c in ((-1, 4, 4), (1, 0, 4), (1, 4, 0), (1, 65537, 4), (65536, 4, 4)):
        assert L.emb_orthogonalize_workspace(b, r, c, ctypes.byref(n)) == bad
    assert L.emb_orthogonalize_workspace(1, 4, 4, None) == bad
    assert L.emb_orthogonalize_workspace(2, 40, 30, ctypes.byref(n)) == emb.EMB_OK and n.value % 256 == 0
    ok = dict(update=0x1000, dtype=2, bs=1200, rs=30, batch=2, rows=40, cols=30, steps=5, a=1.0, b=1.0, c=1.0, eps=0.0,
              out=0x9000, ws=0x10000, bytes=n.value, stream=None)
    for over in (dict(dtype=3), dict(rs=29), dict(steps=0), dict(steps=33), dict(eps=-1.0), dict(update=0x1001), dict(out=0x9001),
                 dict(ws=0x10010), dict(bytes=n.value - 1), dict(update=None), dict(out=None), dict(ws=None)):
        assert L.emb_orthogonalize(*dict(ok, **over).values()) == bad, over
