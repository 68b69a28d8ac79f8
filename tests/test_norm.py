"""Layer norm and dropout against plain implementations in 64 bits.

Tolerances.  u is half the spacing of the output type relative to 1 (2^-24 fp32,
2^-11 fp16, 2^-8 bf16), e = 2^-24.  An fp32 sum of n terms is added up by at least 32
threads or in chains of at most 16 + 16 + 32 (a row of n: 64 + n / 1024 covers every way):
within L e of the terms' magnitudes, L that chain's length.

Layer norm.  Let h be exact, S = mean |x - mean| rstd <= 1 (by Cauchy-Schwarz).  The
centred element (x - m) - d takes two roundings (of x - m, which is at most |x - mean| +
|d|, and of the difference) and d's own error: d is a sum of the centred elements, off by
L e mean |x - m|.  m itself is whatever it is, d corrects it, but d is at most m's error,
(L + 1) e mean |x|, so with M = mean |x| rstd the centred element times rstd is off by
2 e |h| + (L + 2) e S + (L + 1)^2 e^2 M.  The variance is a mean of squares: relatively off by
(L + 6) e and, by d^2, (L + 1)^2 e^2 M^2; rstd by half of that and 2 e.  Together
|h' - h| <= |h| ((L / 2 + 8) e + (L + 1)^2 e^2 M^2) + (L + 2) e + (L + 1)^2 e^2 M.
y = h w + b is one rounding more, then the output's.
"""
import math

import numpy as np
import pytest
import torch

import dlrm_sparse_embedding_gb300 as emb

gpu = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
HALF_ULP = {F32: 2.0 ** -24, HF: 2.0 ** -11, BF: 2.0 ** -8}
TINY = {F32: 2.0 ** -149, HF: 2.0 ** -25, BF: 2.0 ** -133}
E = 2.0 ** -24


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def padded(t, extra, fill=float("nan")):
    """The same matrix with a row stride `extra` elements longer, `fill` between the rows."""
    big = torch.full((t.shape[0], t.shape[1] + extra), fill, dtype=t.dtype, device=t.device)
    big[:, :t.shape[1]] = t
    return big[:, :t.shape[1]]


def check_close(got, ref, bound, what=""):
    got = got.double()
    assert got.shape == ref.shape
    assert torch.isfinite(got).all()
    off = (got - ref).abs() - bound
    assert off.numel() == 0 or off.max().item() <= 0, "%s off by %g over the bound" % (what, off.max().item())


def chain(width):
    return 64 + width / 1024


def rounded(ref, dtype, bound):
    """The bound after the output's rounding."""
    return bound + HALF_ULP[dtype] * (ref.abs() + bound) + TINY[dtype]


def plain(x, w, b, eps):
    """h, rstd, y and the bound of h's error, in 64 bits."""
    x = x.double()
    mean = x.mean(1, keepdim=True)
    c = x - mean
    rstd = 1 / (c.square().mean(1, keepdim=True) + eps).sqrt()
    h = c * rstd
    L, M = chain(x.shape[1]), x.abs().mean(1, keepdim=True) * rstd
    off = (L + 1) ** 2 * E * E
    return h, rstd, h * w + b, h.abs() * ((L / 2 + 8) * E + off * M * M) + (L + 2) * E + off * M


def check_norm(x, w, b, eps, dtype):
    y = emb.layer_norm(x, w, b, eps, dtype)
    assert y.dtype == dtype and y.is_contiguous()
    wd = 1.0 if w is None else w.double()
    bd = 0.0 if b is None else b.double()
    h, rstd, ref, dh = plain(x, wd, bd, eps)
    dh = dh * (wd if w is None else wd.abs())
    check_close(y, ref, rounded(ref, dtype, dh + E * (ref.abs() + dh)), "y")


def check_grad(g, x, w, eps):
    """The gradients' bounds follow from h's: the means over a row of g w and g w h are sums like
    the ones above; a column's sum goes over at most rows / 100 + 300 terms one after another,
    or all of them where there are fewer rows."""
    dx, dw, db = emb.layer_norm_grad(g, x, w, eps)
    assert dx.dtype == x.dtype and dw.dtype == db.dtype == (F32 if w is None else w.dtype)
    wd = torch.ones(x.shape[1], dtype=torch.float64, device="cuda") if w is None else w.double()
    h, rstd, _, dh = plain(x, wd, 0.0, eps)
    gd = g.double()
    gw = gd * wd
    mean = lambda t: t.mean(1, keepdim=True)  # noqa: E731
    along = mean(gw * h)
    ref = rstd * (gw - mean(gw) - h * along)
    L = chain(x.shape[1])
    d_mean = (L + 3) * E * mean(gw.abs())
    d_along = mean(gw.abs() * dh) + (L + 8) * E * mean(gw.abs() * (h.abs() + 1))
    inner = 4 * E * (gw.abs() + mean(gw.abs()) + (h * along).abs()) + d_mean + dh * along.abs() + (h.abs() + dh) * d_along
    rel = (L / 2 + 8) * E + (L + 1) ** 2 * E * E * (x.double().abs().mean(1, keepdim=True) * rstd) ** 2
    inner = rstd * inner * (1 + rel) + ref.abs() * rel
    check_close(dx, ref, rounded(ref, x.dtype, inner), "dx")
    n = x.shape[0]
    n = min(n, n / 100 + 300)
    for got, terms, off in ((dw, gd * h, gd.abs() * dh), (db, gd, torch.zeros_like(gd))):
        ref = terms.sum(0)
        bound = off.sum(0) + (n + 2) * E * (terms.abs() + off).sum(0)
        check_close(got, ref, rounded(ref, got.dtype, bound), "parameters")


SIZES = [(1, 1), (3, 1), (1, 8), (5, 7), (300, 3), (1000, 16), (37, 64), (2000, 100), (513, 128), (9, 255), (70, 256), (31, 257),
         (400, 264), (1, 3328), (700, 3328), (5, 4096), (7, 4097), (11, 4104), (160, 6400), (3, 8191), (6, 8192), (3, 8193), (9, 8200),
         (2, 20000), (40, 33000), (500, 16384), (7, 32768), (5, 32776), (3, 65536), (3, 65541), (2, 131072), (3, 140000)]
TYPES = [(F32, BF), (BF, BF), (HF, HF), (F32, F32), (HF, F32), (BF, HF)]


@gpu
@pytest.mark.parametrize("rows,width", SIZES)
@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("extra", [0, 8, 3])
def test_norm_and_its_gradients(rows, width, xt, yt, extra):
    g = gen(rows * 7 + width)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = padded(((r(rows, width) + 0.5 * r(width)) * torch.exp(r(rows, 1))).to(xt), extra)
    pt = [F32, yt, BF][(rows + extra) % 3]
    w, b = (1 + 0.3 * r(width)).to(pt), (0.5 * r(width)).to(pt)
    check_norm(x, w, b, 1e-5, yt)
    check_grad(padded(r(rows, width).to(yt), extra), x, w, 1e-5)


@gpu
@pytest.mark.parametrize("width", [5, 40, 129, 520, 1000, 3328, 9000])
@pytest.mark.parametrize("first", [1, 3, 8])
@pytest.mark.parametrize("xt,yt", [(F32, BF), (BF, BF), (HF, F32)])
def test_rows_that_begin_anywhere(width, first, xt, yt):
    # columns of a wider matrix: neighbours are read at most, never used
    g = gen(width + first)
    rows = 37
    big = torch.randn(rows, width + 16, generator=g, device="cuda").to(xt)
    wide = torch.randn(rows, width + 24, generator=g, device="cuda").to(yt)
    for t in (big, wide):
        t[:, :first], t[:, first + width:] = float("nan"), float("inf")
    x, gy = big[:, first:first + width], wide[:, first:first + width]
    w = torch.randn(width + 1, generator=g, device="cuda")[1:]      # a parameter off a vector's boundary
    check_norm(x, w, w, 1e-5, yt)
    check_grad(gy, x, w, 1e-5)
    check_grad(gy.contiguous(), x, w, 1e-5)
    check_grad(gy, x.contiguous(), w, 1e-5)
    assert torch.equal(emb.dropout(gy, 0.5, 3, residual=gy), emb.dropout(gy.contiguous(), 0.5, 3, residual=gy.contiguous()))


@gpu
def test_calls_of_several_threads():
    import threading
    jobs = []
    for i in range(4):
        g = gen(i)
        x, w = torch.randn(500 + i, 700 + 100 * i, generator=g, device="cuda"), torch.randn(700 + 100 * i, generator=g, device="cuda")
        jobs.append((torch.cuda.Stream(), x, w, (emb.layer_norm(x, w), *emb.layer_norm_grad(x, x, w), emb.dropout(x, 0.3, i))))
    torch.cuda.synchronize()
    wrong = []

    def work(seed, stream, x, w, ref):
        for _ in range(30):
            with torch.cuda.stream(stream):
                got = emb.layer_norm(x, w), *emb.layer_norm_grad(x, x, w), emb.dropout(x, 0.3, seed)
            stream.synchronize()
            wrong.extend(1 for a, b in zip(got, ref) if not torch.equal(a, b))

    threads = [threading.Thread(target=work, args=(i, *job)) for i, job in enumerate(jobs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@gpu
def test_weight_and_bias_may_be_left_out():
    g = gen(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    for rows, width in ((40, 96), (3, 9000)):
        x, w, b, gy = r(rows, width), r(width), r(width), r(rows, width)
        check_norm(x, None, None, 1e-5, F32)
        check_norm(x, w, None, 1e-5, BF)
        check_norm(x, None, b, 1e-5, HF)
        check_grad(gy, x, None, 1e-5)
        whole = emb.layer_norm_grad(gy, x, w)
        alone, nothing, none = emb.layer_norm_grad(gy, x, w, need_weight=False)
        assert nothing is None and none is None and torch.equal(alone, whole[0])
        nothing, dw, db = emb.layer_norm_grad(gy, x, w, need_x=False)
        assert nothing is None and torch.equal(dw, whole[1]) and torch.equal(db, whole[2])
        assert emb.layer_norm_grad(gy, x, w, need_x=False, need_weight=False) == (None, None, None)


@gpu
@pytest.mark.parametrize("rows,width", [(33, 100), (9, 3328), (5, 8192), (3, 9001)])
@pytest.mark.parametrize("kind", ["far from zero", "large", "huge", "small", "constant", "one large element"])
def test_rows_of_any_size(rows, width, kind):
    g = gen(5)
    x = torch.randn(rows, width, generator=g, device="cuda")
    eps = 1e-5
    if kind == "far from zero":
        x += 3000
    elif kind == "large":
        x *= 2.0 ** 60
    elif kind == "huge":
        x = x.clamp(-4, 4) * 2.0 ** 125
    elif kind == "small":
        x, eps = x * 1e-9, 1e-24
    elif kind == "constant":
        x = torch.full_like(x, -7.25)
    else:
        x[:, width // 2] = 1e4
    w, b, gy = (torch.randn(*s, generator=g, device="cuda") for s in ((width,), (width,), (rows, width)))
    check_norm(x, w, b, eps, F32)
    check_grad(gy, x, w, eps)


@gpu
@pytest.mark.parametrize("width", [40, 100, 3328, 9000])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_rows_infinities_and_nans_stay_its_own(width, bad):
    g = gen(2)
    x, gy, w = (torch.randn(*s, generator=g, device="cuda") for s in ((40, width), (40, width), (width,)))
    clean = emb.layer_norm(x, w), emb.layer_norm_grad(gy, x, w)
    x[17, width // 3] = bad
    y, (dx, dw, db) = emb.layer_norm(x, w), emb.layer_norm_grad(gy, x, w)
    others = torch.arange(40, device="cuda") != 17
    assert torch.isnan(y[17]).all() and torch.isnan(dx[17]).all()
    assert torch.equal(y[others], clean[0][others]) and torch.equal(dx[others], clean[1][0][others])
    assert torch.isnan(dw).all() and torch.equal(db, clean[1][2])


@gpu
@pytest.mark.parametrize("width", [513, 1024, 1288, 1301, 1536, 1700, 2048, 2049])
@pytest.mark.parametrize("rows", [4, 803])
@pytest.mark.parametrize("t", [F32, BF])
def test_gradients_of_rows_that_share_a_block(rows, width, t):
    g = gen(rows + width)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, gy, w = r(rows, width).to(t), r(rows, width).to(t), (1 + 0.3 * r(width)).to(t)
    check_grad(gy, x, w, 1e-5)
    clean = emb.layer_norm_grad(gy, x, w)
    x[2] = (x[2].float() * 2.0 ** 80).to(t)     # a row that is taken twice, beside rows that are not
    dx, _, db = emb.layer_norm_grad(gy, x, w)
    others = torch.arange(rows, device="cuda") != 2
    assert torch.equal(dx[others], clean[0][others]) and torch.equal(db, clean[2])


@gpu
@pytest.mark.parametrize("width", [24, 3328, 10000])
def test_norm_gradients_are_the_differences(width):
    g = gen(3)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, w, gy, along = r(6, width), r(width), r(6, width), r(6, width)
    dx, dw, db = emb.layer_norm_grad(gy, x, w, 1e-5)

    def f(v):      # the formula, in 64 bits
        return (plain(v, w.double(), 0.0, 1e-5)[2] * gy.double()).sum()

    step = 1e-4
    slope = (f(x.double() + step * along.double()) - f(x.double() - step * along.double())) / (2 * step)
    # the difference is off by step^2 times a third derivative, 1e-8 of the terms; dx by roundings, 1e-5 of them
    terms = (dx.double() * along.double()).abs().sum()
    assert (slope - (dx.double() * along.double()).sum()).abs() <= 1e-4 * terms
    h = plain(x, w.double(), 0.0, 1e-5)[0]
    assert (dw.double() - (gy.double() * h).sum(0)).abs().max() <= 1e-4 and (db.double() - gy.double().sum(0)).abs().max() <= 1e-5


@gpu
def test_no_rows():
    for width in (8, 9000):
        x, w = torch.empty(0, width, device="cuda"), torch.ones(width, device="cuda", dtype=BF)
        assert emb.layer_norm(x, w).shape == (0, width)
        dx, dw, db = emb.layer_norm_grad(x, x, w)
        assert dx.shape == (0, width) and not dw.any() and not db.any()
        assert emb.dropout(x, 0.1, 1).shape == (0, width)


@gpu
@pytest.mark.parametrize("rows,width", [(2000, 100), (300, 3328), (40, 20000)])
def test_results_repeat(rows, width):
    g = gen(4)
    x, gy, w = (torch.randn(*s, generator=g, device="cuda") for s in ((rows, width), (rows, width), (width,)))
    a = emb.layer_norm_grad(gy, x, w)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(a, emb.layer_norm_grad(gy, x, w)))


# --------------------------------------------------------------------------- #
# dropout
# --------------------------------------------------------------------------- #
def mask(n, rate, seed, offset):
    """Elements kept: Philox4x32 with 7 rounds in Python's whole numbers where n is small."""
    u = np.uint64
    low, half = u(0xFFFFFFFF), u(32)
    ctr = np.arange((n + 7) // 8, dtype=np.uint64)
    c = [ctr & low, ctr >> half, np.full_like(ctr, offset & 0xFFFFFFFF), np.full_like(ctr, offset >> 32 & 0xFFFFFFFF)]
    k = [seed & 0xFFFFFFFF, seed >> 32 & 0xFFFFFFFF]
    for _ in range(7):
        p, q = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(q >> half) ^ c[1] ^ u(k[0]), q & low, (p >> half) ^ c[3] ^ u(k[1]), p & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    bits = np.stack([c[0] & u(0xFFFF), c[0] >> u(16), c[1] & u(0xFFFF), c[1] >> u(16),
                     c[2] & u(0xFFFF), c[2] >> u(16), c[3] & u(0xFFFF), c[3] >> u(16)], 1).reshape(-1)[:n]
    return bits >= round(rate * 65536)


def test_the_masks_generator():
    # ten rounds of the same steps give the known answers of Philox4x32-10 (Random123's kat_vectors)
    def philox(c, k, rounds):
        for _ in range(rounds):
            p, q = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
            c = [(q >> 32) ^ c[1] ^ k[0], q & 0xFFFFFFFF, (p >> 32) ^ c[3] ^ k[1], p & 0xFFFFFFFF]
            k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
        return c

    assert philox([0] * 4, [0] * 2, 10) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert philox([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, 10) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    seed, offset = 0x123456789ABCDEF0, 0xFEDCBA9876543210
    for group in (0, 5):
        words = philox([group, 0, offset & 0xFFFFFFFF, offset >> 32], [seed & 0xFFFFFFFF, seed >> 32], 7)
        bits = [h for w in words for h in (w & 0xFFFF, w >> 16)]
        for rate in (0.1, 0.5, 0.9):
            assert mask(48, rate, seed, offset)[group * 8:group * 8 + 8].tolist() == [b >= round(rate * 65536) for b in bits]


DROPS = [(1, 1), (1, 7), (3, 5), (2, 8), (17, 13), (5, 255), (9, 256), (7, 257), (300, 24), (1, 5000), (77, 777), (1000, 128), (2, 100003),
         (70000, 8)]


@gpu
@pytest.mark.parametrize("rows,width", DROPS)
@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("extra", [0, 8, 3])
@pytest.mark.parametrize("residual", [False, True])
def test_dropout_and_its_gradient(rows, width, xt, yt, extra, residual):
    rate, seed, offset = [(0.1, 5, 0), (0.5, -3, 2 ** 40 + 1), (0.25, 2 ** 63 + 11, 7)][(rows + width + extra) % 3]
    g = gen(rows + width)
    x, gy, res = (padded(torch.randn(rows, width, generator=g, device="cuda").to(t), extra) for t in (xt, yt, yt))
    keep = torch.from_numpy(mask(rows * width, rate, seed & 2 ** 64 - 1, offset)).cuda().reshape(rows, width)
    x[~keep] = float("nan")       # what is dropped is not used
    gy[~keep] = float("inf")
    scale = 1 / (1 - round(rate * 65536) / 65536)
    y = emb.dropout(x, rate, seed, offset, res if residual else None, yt)
    dx = emb.dropout_grad(gy, rate, seed, offset, xt)
    assert y.dtype == yt and dx.dtype == xt
    for got, v, add in ((y, x, res if residual else None), (dx, gy, None)):
        term = torch.where(keep, v.double(), 0.0) * scale
        ref = term if add is None else term + add.double()
        # the scale's rounding, one of the sum in fp32, the output's
        check_close(got, ref, rounded(ref, got.dtype, E * (2 * term.abs() + ref.abs())))
        if add is None:
            assert not got[~keep].any()
        else:
            assert torch.equal(got[~keep], add[~keep])


@gpu
def test_the_kept_share_and_unrelated_uses():
    x = torch.ones(1000, 1000, device="cuda")
    n = x.numel()
    masks = []
    for rate in (0.0, 0.1, 0.5, 0.9, 1.0):
        y = emb.dropout(x, rate, 17, 3)
        kept = (y != 0).sum().item()
        assert abs(kept - n * (1 - rate)) <= 6 * math.sqrt(n * rate * (1 - rate)) + n * 2 ** -16   # six standard deviations, the rate's step
        if rate in (0.0, 1.0):
            assert kept == n * (1 - rate)
    for seed, offset in ((17, 3), (18, 3), (17, 4), (17, 3 + 2 ** 32), (17 + 2 ** 32, 3)):
        masks.append(emb.dropout(x, 0.5, seed, offset) != 0)
    for i in range(len(masks)):
        for j in range(i):
            same = (masks[i] == masks[j]).sum().item()
            assert abs(same - n / 2) <= 6 * math.sqrt(n) / 2


@gpu
def test_the_mask_does_not_depend_on_layout_or_type():
    x = torch.ones(50, 264, device="cuda")
    ref = emb.dropout(x, 0.3, 9) != 0
    shifted = torch.ones(50 * 264 + 1, device="cuda")[1:].reshape(50, 264)     # 4 bytes past a vector's boundary
    for v in (x.bfloat16(), padded(x, 8), padded(x, 1), shifted, padded(x.half(), 2)):
        assert torch.equal(emb.dropout(v, 0.3, 9) != 0, ref)


@gpu
def test_a_captured_seed_is_read_at_every_replay():
    x = torch.randn(64, 200, device="cuda")
    seed = torch.tensor([4], device="cuda")
    emb.dropout(x, 0.5, seed, 1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = emb.dropout(x, 0.5, seed, 1)
        dx = emb.dropout_grad(y, 0.5, seed, 1)
    for s in (4, 5, -6):
        seed.fill_(s)
        graph.replay()
        assert torch.equal(y, emb.dropout(x, 0.5, s, 1)) and torch.equal(dx, emb.dropout_grad(y, 0.5, s, 1))


@gpu
def test_more_elements_than_32_bits():
    # the last rows of a matrix of 2^32 + elements: offsets and counters past 32 bits
    rows, width = 2 ** 21 + 40, 2048 + 8
    x = torch.ones(rows, width, dtype=BF, device="cuda")
    y = emb.dropout(x, 0.5, 3)
    first = rows * width - 2 ** 20
    first -= first % 8
    u = np.uint64
    ctr = np.arange(first // 8, rows * width // 8, dtype=np.uint64)
    low, half = u(0xFFFFFFFF), u(32)
    c = [ctr & low, ctr >> half, np.zeros_like(ctr), np.zeros_like(ctr)]
    k = [3, 0]
    for _ in range(7):
        p, q = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(q >> half) ^ c[1] ^ u(k[0]), q & low, (p >> half) ^ c[3] ^ u(k[1]), p & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    bits = np.stack([w >> u(s) & u(0xFFFF) for w in c for s in (0, 16)], 1).reshape(-1)
    assert np.array_equal((y.reshape(-1)[first:] != 0).cpu().numpy(), bits >= 32768)
    del y
    w = torch.ones(width, device="cuda")
    x[-1] = torch.arange(width, device="cuda") % 7
    y = emb.layer_norm(x, w)
    assert torch.equal(y[-1:], emb.layer_norm(x[-1:].clone(), w)) and not y[:-1].any()


# --------------------------------------------------------------------------- #
# streams, graphs, refusals
# --------------------------------------------------------------------------- #
@gpu
def test_on_another_stream():
    x, w = torch.randn(500, 1024, device="cuda"), torch.randn(1024, device="cuda")
    ref = emb.layer_norm(x, w), emb.layer_norm_grad(x, x, w), emb.dropout(x, 0.1, 2, residual=x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = emb.layer_norm(x, w, stream=s), emb.layer_norm_grad(x, x, w, stream=s), emb.dropout(x, 0.1, 2, residual=x, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[2], ref[2])
    assert all(torch.equal(a, b) for a, b in zip(got[1], ref[1]))


@gpu
def test_two_graphs_replayed_in_turn():
    x, w = torch.randn(3000, 512, device="cuda"), torch.randn(512, device="cuda")
    graphs = []
    for scale in (1.0, 2.0):
        gy = x * scale
        emb.layer_norm_grad(gy, x, w)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = emb.layer_norm_grad(gy, x, w)
        graphs.append((graph, out, gy))
    for _ in range(3):
        for graph, out, gy in graphs:
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(out, emb.layer_norm_grad(gy, x, w)))


@gpu
def test_inputs_that_require_gradients_and_tensors_of_another_device(monkeypatch):
    x, w = torch.randn(5, 40, device="cuda").requires_grad_(), torch.randn(40, device="cuda").requires_grad_()
    calls = [lambda: emb.layer_norm(x, w, w), lambda: emb.layer_norm_grad(x, x, w), lambda: emb.dropout(x, 0.1, 1, residual=x),
             lambda: emb.dropout_grad(x, 0.1, 1)]
    for call in calls:
        got = call()
        assert not any(t.requires_grad for t in (got if isinstance(got, tuple) else (got,)))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)      # nothing is launched: the tensors are on 0
    for call in calls:
        with pytest.raises(ValueError, match="current device"):
            call()


@gpu
def test_under_autograd():
    # the explicit gradients in a torch.autograd.Function
    class Block(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, b):
            ctx.save_for_backward(x, w)
            return emb.dropout(emb.layer_norm(x, w, b), 0.25, 5, residual=x)

        @staticmethod
        def backward(ctx, grad):
            x, w = ctx.saved_tensors
            grad = grad.contiguous()
            dx, dw, db = emb.layer_norm_grad(emb.dropout_grad(grad, 0.25, 5), x, w)
            return dx + grad, dw, db

    g = gen(9)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, w, b, gy = r(300, 264).requires_grad_(), r(264).requires_grad_(), r(264).requires_grad_(), r(300, 264)
    keep = (emb.dropout(torch.ones(300, 264, device="cuda"), 0.25, 5) != 0).double() / 0.75
    leaves = [t.detach().double().requires_grad_() for t in (x, w, b)]
    xd, wd, bd = leaves
    h = (xd - xd.mean(1, keepdim=True)) / (xd.var(1, correction=0, keepdim=True) + 1e-5).sqrt()
    ref = torch.autograd.grad(((h * wd + bd) * keep + xd).mul(gy.double()).sum(), leaves)
    got = torch.autograd.grad(Block.apply(x, w, b).mul(gy).sum(), (x, w, b))
    for a, e in zip(got, ref):
        # sums of 300 terms of size 1, a chain of at most 64 + 8 roundings
        assert (a.double() - e).abs().max() <= 300 * 72 * E


REFUSALS = [
    ("2-d", lambda n, x, w: n.layer_norm(x[0])),
    ("CUDA", lambda n, x, w: n.layer_norm(x.cpu())),
    ("float32, float16", lambda n, x, w: n.layer_norm(x.double())),
    ("float32, float16", lambda n, x, w: n.layer_norm(x.int())),
    ("elements", lambda n, x, w: n.layer_norm(x, w[:-1])),
    ("elements", lambda n, x, w: n.layer_norm(x, w, w[None])),
    ("one type", lambda n, x, w: n.layer_norm(x, w, w.half())),
    ("must be on", lambda n, x, w: n.layer_norm(x, w.cpu())),
    ("eps", lambda n, x, w: n.layer_norm(x, w, eps=0.0)),
    ("eps", lambda n, x, w: n.layer_norm(x, w, eps=float("nan"))),
    ("eps", lambda n, x, w: n.layer_norm_grad(x, x, w, eps=float("inf"))),
    ("dtype", lambda n, x, w: n.layer_norm(x, w, dtype=torch.float64)),
    ("contiguous rows", lambda n, x, w: n.layer_norm(x.t())),
    ("contiguous rows", lambda n, x, w: n.layer_norm(x[:1].expand(4, -1))),
    ("shape", lambda n, x, w: n.layer_norm(x[:, :0])),
    ("shape", lambda n, x, w: n.layer_norm_grad(x[1:], x, w)),
    ("rate", lambda n, x, w: n.dropout(x, 1.01, 1)),
    ("rate", lambda n, x, w: n.dropout(x, float("nan"), 1)),
    ("residual", lambda n, x, w: n.dropout(x, 0.1, 1, residual=x[1:])),
    ("residual", lambda n, x, w: n.dropout(x, 0.1, 1, residual=x.half(), dtype=torch.float32)),
    ("seed", lambda n, x, w: n.dropout(x, 0.1, torch.zeros(2, dtype=torch.int64, device=x.device))),
    ("seed", lambda n, x, w: n.dropout(x, 0.1, torch.zeros(1, dtype=torch.int64))),
    ("seed", lambda n, x, w: n.dropout(x, 0.1, torch.zeros(1, dtype=torch.int32, device=x.device))),
]


@gpu
@pytest.mark.parametrize("i", range(len(REFUSALS)))
def test_refusals(i):
    what, call = REFUSALS[i]
    x, w = torch.zeros(4, 24, device="cuda"), torch.ones(24, device="cuda")
    with pytest.raises(ValueError, match=what):
        call(emb, x, w)


def test_the_c_calls_refuse_on_the_host():
    # each is rejected by the host's checks, before any CUDA call
    import ctypes
    bad = emb.EMB_ERR_INVALID_ARG
    n = ctypes.c_size_t()
    assert emb.lib.emb_layer_norm_grad_workspace(-1, 8, ctypes.byref(n)) == bad
    assert emb.lib.emb_layer_norm_grad_workspace(4, 0, ctypes.byref(n)) == bad
    assert emb.lib.emb_layer_norm_grad_workspace(4, 2 ** 24 + 1, ctypes.byref(n)) == bad
    assert emb.lib.emb_layer_norm_grad_workspace(4, 8, ctypes.byref(n)) == emb.EMB_OK and n.value >= 256
    at = 0x10000
    ok = [at, 0, 8, 4, 8, at, at, 0, 1e-5, at, 0, None]
    for i, v in ((0, None), (0, at + 2), (1, 3), (2, 7), (3, -1), (4, 0), (5, at + 1), (7, 5), (8, 0.0), (8, float("inf")), (9, None), (10, -1)):
        args = list(ok)
        args[i] = v
        assert emb.lib.emb_layer_norm(*args) == bad, (i, v)
    ok = [at, 0, 8, at, 0, 8, 4, 8, at, 0, 1e-5, at, at, at, at, 1 << 30, None]
    for i, v in ((0, None), (1, 3), (2, 7), (3, None), (6, -1), (10, 1e-30), (11, at + 2), (12, at + 1), (14, None), (14, at + 8), (15, 16)):
        args = list(ok)
        args[i] = v
        assert emb.lib.emb_layer_norm_grad(*args) == bad, (i, v)
    ok = [at, 0, 8, 4, 8, 0.1, 1, None, 0, None, 0, at, 0, None]
    for i, v in ((0, None), (1, 4), (2, 4), (3, -1), (3, 2 ** 62), (4, 0), (5, -0.1), (5, 1.5), (5, float("nan")), (7, at + 4), (9, at), (11, None), (12, 9)):
        args = list(ok)
        args[i] = v
        assert emb.lib.emb_dropout(*args) == bad, (i, v)
