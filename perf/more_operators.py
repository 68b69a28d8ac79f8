"""Cases for the operators around the experts of a recommender's dense side.

A block of the dense side is x + dropout(experts(layer_norm(x))) of the pooled
embeddings (a row is a sample, or one table's vector of a sample).  Three kinds of
case:

  norm     layer norm of rows and, in training, the gradients of the rows, the
           weight and the bias
  dropout  dropout by a counter-based generator, with or without the residual it
           is added to and, in training, the gradient
  layer    the whole expert layer of a few tokens: up, activation, down, weighted sum

`own` false: plain torch operations in 32 bits, rounded once at the end.
`own` true: this package's calls.
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# --------------------------------------------------------------------------- #
# cases
# --------------------------------------------------------------------------- #
def listed():
    return [
        # one request's pooled features of 26 tables of 128; latency
        dict(name="norm_request", op="norm", rows=1, width=3328, src="f32", dtype="bf16", param="f32", train=False),
        # a training batch of the 26 x 128 model, from the layer's fp32 output to bf16 rows and back
        dict(name="norm_train", op="norm", rows=16384, width=3328, src="f32", dtype="bf16", param="f32", train=True),
        # an odd batch of an odd width: rows that no vector fits
        dict(name="norm_odd", op="norm", rows=1777, width=1025, src="f16", dtype="f16", param="f32", train=True),
        # every table's vector normalised by itself: many short rows
        dict(name="norm_tables", op="norm", rows=425984, width=128, src="bf16", dtype="bf16", param="bf16", train=True),
        # an online update's few samples, added to their residual
        dict(name="dropout_small", op="dropout", rows=7, width=3328, src="bf16", dtype="bf16", rate=0.1, residual=True,
             train=False),
        # an odd number of elements, fp32 rows to fp16
        dict(name="dropout_odd", op="dropout", rows=4097, width=1025, src="f32", dtype="f16", rate=0.5, residual=False,
             train=True),
        # a training batch behind the experts: dropout, residual, and the gradient
        dict(name="dropout_train", op="dropout", rows=32768, width=2048, src="bf16", dtype="bf16", rate=0.1, residual=True,
             train=True),
        # one request's sample through 2 of 16 experts, from the embedding layer's fp32; latency
        dict(name="layer_request", op="layer", tokens=1, k=2, experts=16, width=3328, hidden=1024, out=1024, src="f32",
             dtype="bf16", act="relu", dropped=0.0),
        # a few samples, widths that fill no tile, assignments lost to the experts' capacity
        dict(name="layer_ragged", op="layer", tokens=7, k=3, experts=12, width=1032, hidden=776, out=520, src="f16",
             dtype="f16", act="gelu", dropped=0.3),
        # a serving batch of gated experts
        dict(name="layer_gated", op="layer", tokens=16, k=2, experts=32, width=2048, hidden=1408, out=2048, src="bf16",
             dtype="bf16", act="swiglu", dropped=0.0),
        # a serving batch over many experts: about 3 rows each, every expert's weights read
        dict(name="layer_serve", op="layer", tokens=48, k=4, experts=64, width=1024, hidden=2048, out=1024, src="f16",
             dtype="f16", act="silu", dropped=0.0),
        # more samples than experts: about 16 rows each
        dict(name="layer_crowd", op="layer", tokens=64, k=4, experts=16, width=3328, hidden=2048, out=1024, src="bf16",
             dtype="bf16", act="relu", dropped=0.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi, unit=1):
    """An odd multiple of `unit` (sizes that fill no tile), or, one time in three, a power of two."""
    if rng.random() < 1 / 3:
        return 2 ** rng.randint(math.ceil(math.log2(lo)), math.floor(math.log2(hi)))
    return unit * (2 * (_log_int(rng, lo, hi) // (2 * unit)) + 1)


def _draw_once(rng):
    op = rng.choice(["norm", "dropout", "layer"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "layer":
        experts = _log_int(rng, 2, 128)
        c = dict(op=op, tokens=_log_int(rng, 1, 64), k=min(experts, rng.choice([1, 2, 2, 3, 4, 6, 8])), experts=experts,
                 width=_size(rng, 64, 4096, 8), hidden=_size(rng, 64, 4096, 8), out=_size(rng, 64, 4096, 8),
                 src=rng.choice(["f32", dtype]), dtype=dtype, act=rng.choice(["relu", "silu", "gelu", "swiglu"]))
        c["dropped"] = rng.choice([0.0, 0.0, 0.3]) if c["tokens"] >= 4 else 0.0
        return c
    c = dict(op=op, rows=_size(rng, 1, 425984), width=_size(rng, 16, 16384, rng.choice([1, 8, 8])),
             src=rng.choice(["f32", dtype]), dtype=rng.choice([dtype, dtype, "f32"]), train=rng.random() < 0.6)
    if op == "norm":
        c["param"] = rng.choice(["f32", "f32", c["dtype"]])
    else:
        c["rate"], c["residual"] = rng.choice([0.1, 0.1, 0.25, 0.5]), rng.random() < 0.5
    return c


def draw(rng):
    most = {}
    for c in listed():
        w, m = work(c), most.setdefault(c["op"], {"bytes": 0.0, "flops": 0.0})
        for key in m:
            m[key] = max(m[key], w[key])
    while True:
        c = _draw_once(rng)
        w = work(c)
        if all(w[key] <= most[c["op"]][key] for key in w):
            # the largest weights a drawn case may hold: twice those of the listed cases
            if c["op"] != "layer" or c["experts"] * c["hidden"] * (_up(c) * c["width"] + c["out"]) <= 64 * 2048 * 4096:
                return c


def _up(case):
    """Rows of the first weight for each hidden unit: a gated activation has two."""
    return 2 if case["act"] == "swiglu" else 1


# --------------------------------------------------------------------------- #
# inputs
# --------------------------------------------------------------------------- #
def _normal(g, *shape, dtype, scale=1.0):
    x = torch.randn(*shape, generator=g, device="cuda")
    return x.mul_(scale).to(_DTYPES[dtype])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": case}
    if case["op"] == "layer":
        T, k, E, D, H, N = (case[n] for n in ("tokens", "k", "experts", "width", "hidden", "out"))
        # a router's choice: k distinct experts a token, some more liked than others
        scores = torch.randn(T, E, generator=g, device="cuda") + 0.4 * torch.randn(E, generator=g, device="cuda")
        top, ids = torch.topk(scores, k, dim=1)
        s["weights"] = torch.softmax(top, dim=1).float().contiguous()
        if case["dropped"] > 0:
            lost = torch.rand(T, k, generator=g, device="cuda") < case["dropped"]
            lost[0] = True      # a token without experts
            ids = torch.where(lost, torch.full_like(ids, -1), ids)
        s["ids"] = ids.to(torch.int32).contiguous()
        s["x"] = _normal(g, T, D, dtype=case["src"])
        s["up"] = _normal(g, E, _up(case) * H, D, dtype=case["dtype"], scale=1 / math.sqrt(D))
        s["down"] = _normal(g, E, N, H, dtype=case["dtype"], scale=1 / math.sqrt(H))
        return s
    R, D = case["rows"], case["width"]
    if case["op"] == "norm":
        # pooled embeddings: rows of different sizes, columns of different means
        size = torch.exp(0.5 * torch.randn(R, 1, generator=g, device="cuda"))
        x = torch.randn(R, D, generator=g, device="cuda") + 0.5 * torch.randn(D, generator=g, device="cuda")
        s["x"] = x.mul_(size).to(_DTYPES[case["src"]])
        s["weight"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(_DTYPES[case["param"]])
        s["bias"] = (0.2 * torch.randn(D, generator=g, device="cuda")).to(_DTYPES[case["param"]])
    else:
        s["x"] = _normal(g, R, D, dtype=case["src"])
        s["residual"] = _normal(g, R, D, dtype=case["dtype"]) if case["residual"] else None
        s["seed"] = torch.randint(0, 2 ** 62, (1,), generator=g, device="cuda")     # int64: a graph's replays may change it
        s["offset"] = int(seed) % 1000003                                           # the program's count of dropouts so far
    if case["train"]:
        s["grad_y"] = _normal(g, R, D, dtype=case["dtype"])
    return s


# --------------------------------------------------------------------------- #
# the plain forms
# --------------------------------------------------------------------------- #
_EPS = 1e-5
_M0, _M1, _W0, _W1 = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85   # Philox4x32 (Salmon et al., 2011)
_ROUNDS, _LOW = 7, 0xFFFFFFFF


def _plain_norm(s):
    case, x = s["case"], s["x"].float()
    xc = x - x.mean(1, keepdim=True)
    rstd = 1 / (xc.square().mean(1, keepdim=True) + _EPS).sqrt()
    h = xc * rstd
    w = s["weight"].float()
    out = {"y": (h * w + s["bias"].float()).to(_DTYPES[case["dtype"]])}
    if case["train"]:
        g = s["grad_y"].float()
        gw = g * w
        dx = rstd * (gw - gw.mean(1, keepdim=True) - h * (gw * h).mean(1, keepdim=True))
        out["grad_x"] = dx.to(s["x"].dtype)
        out["grad_weight"] = (g * h).sum(0, dtype=torch.float64).to(s["weight"].dtype)
        out["grad_bias"] = g.sum(0, dtype=torch.float64).to(s["weight"].dtype)
    return out


def _kept(s):
    """The mask [rows, width]: 16 bits for each element, eight elements to a counter."""
    n = s["x"].numel()
    threshold = round(s["case"]["rate"] * 65536)
    index = torch.arange((n + 7) // 8, device="cuda")
    k0, k1 = s["seed"] & _LOW, (s["seed"] >> 32) & _LOW
    c0, c1 = index & _LOW, index >> 32
    c2, c3 = (torch.full_like(index, v) for v in (s["offset"] & _LOW, s["offset"] >> 32))
    for _ in range(_ROUNDS):
        p0, p1 = c0 * _M0, c2 * _M1     # 64 bits, of which the sign is one
        c0, c1, c2, c3 = ((p1 >> 32) & _LOW) ^ c1 ^ k0, p1 & _LOW, ((p0 >> 32) & _LOW) ^ c3 ^ k1, p0 & _LOW
        k0, k1 = (k0 + _W0) & _LOW, (k1 + _W1) & _LOW
    words = torch.stack([c0, c1, c2, c3], 1)
    bits = torch.stack([words & 0xFFFF, words >> 16], 2).reshape(-1)[:n]
    return (bits >= threshold).reshape(s["x"].shape), 1 / (1 - threshold / 65536)


def _plain_dropout(s):
    case = s["case"]
    keep, scale = _kept(s)
    y = torch.where(keep, s["x"].float() * scale, 0.0)
    if case["residual"]:
        y = y + s["residual"].float()
    out = {"y": y.to(_DTYPES[case["dtype"]])}
    if case["train"]:
        out["grad_x"] = torch.where(keep, s["grad_y"].float() * scale, 0.0).to(s["x"].dtype)
    return out


def _activate(act, h):
    if act == "swiglu":
        gate, up = h.chunk(2, dim=2)
        return gate / (1 + torch.exp(-gate)) * up
    if act == "silu":
        return h / (1 + torch.exp(-h))
    if act == "gelu":
        return 0.5 * h * (1 + torch.erf(h * math.sqrt(0.5)))
    return torch.clamp(h, min=0)


def _plain_layer(s):
    case, ids = s["case"], s["ids"].long()
    T, k, E = case["tokens"], case["k"], case["experts"]
    x = s["x"].to(_DTYPES[case["dtype"]]).float()     # the products' type
    has = ids >= 0
    if T * k <= E:      # the chosen experts' weights, one after another
        at = ids.clamp(min=0).reshape(-1)
        rows = x.repeat_interleave(k, 0)[:, None, :]
        h = _activate(case["act"], rows @ s["up"][at].float().transpose(1, 2))
        y = (h @ s["down"][at].float().transpose(1, 2)).reshape(T, k, -1)
        out = (torch.where(has, s["weights"], 0.0)[:, :, None] * y * has[:, :, None]).sum(1)
    else:               # every token through every expert
        share = torch.zeros(T, E, device="cuda").scatter_add_(1, ids.clamp(min=0), torch.where(has, s["weights"], 0.0))
        h = _activate(case["act"], x[None] @ s["up"].float().transpose(1, 2))
        y = h @ s["down"].float().transpose(1, 2)
        out = (y * share.t()[:, :, None]).sum(0)
    return {"out": out.to(_DTYPES[case["dtype"]])}


# --------------------------------------------------------------------------- #
# one pass
# --------------------------------------------------------------------------- #
def _own(s):
    import dlrm_sparse_embedding_gb300 as emb
    case = s["case"]
    dt = _DTYPES[case["dtype"]]
    if case["op"] == "norm":
        out = {"y": emb.layer_norm(s["x"], s["weight"], s["bias"], eps=_EPS, dtype=dt)}
        if case["train"]:
            out["grad_x"], out["grad_weight"], out["grad_bias"] = emb.layer_norm_grad(s["grad_y"], s["x"], s["weight"], eps=_EPS)
        return out
    if case["op"] == "dropout":
        out = {"y": emb.dropout(s["x"], case["rate"], s["seed"], s["offset"], residual=s["residual"], dtype=dt)}
        if case["train"]:
            out["grad_x"] = emb.dropout_grad(s["grad_y"], case["rate"], s["seed"], s["offset"], dtype=s["x"].dtype)
        return out
    return {"out": emb.expert_layer(s["ids"], s["x"], s["up"], s["down"], s["weights"], activation=case["act"], dtype=dt)}


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "dropout": _plain_dropout, "layer": _plain_layer}[state["case"]["op"]](state)


# --------------------------------------------------------------------------- #
# what a pass cannot do without
# --------------------------------------------------------------------------- #
def work(case):
    b = _BYTES[case["dtype"]]
    sb = _BYTES[case["src"]]
    if case["op"] == "layer":
        T, k, E, D, H, N = (case[n] for n in ("tokens", "k", "experts", "width", "hidden", "out"))
        kept = T * k * (1 - case["dropped"])
        active = E * (1 - (1 - k / E * (1 - case["dropped"])) ** T)
        weights = _up(case) * D + N
        return {"bytes": b * active * H * weights + sb * T * D + b * T * N + 8.0 * T * k, "flops": 2.0 * kept * H * weights}
    n = float(case["rows"]) * case["width"]
    if case["op"] == "norm":
        pb = 2.0 * _BYTES[case["param"]] * case["width"]
        if case["train"]:       # the rows, the gradient; normalised rows, the rows' gradient, both parameters'
            return {"bytes": n * (2 * sb + 2 * b) + 2 * pb, "flops": 20.0 * n}
        return {"bytes": n * (sb + b) + pb, "flops": 8.0 * n}
    total = n * (sb + b + (b if case["residual"] else 0))
    if case["train"]:
        total += n * (sb + b)
    return {"bytes": total + 8.0, "flops": (4.0 if case["train"] else 2.0) * n}


# --------------------------------------------------------------------------- #
# the definitions in 64 bits
# --------------------------------------------------------------------------- #
def _exact_mask(n, rate, seed, offset):
    """One flat mask, by numpy's unsigned numbers."""
    u = np.uint64
    low, half = u(_LOW), u(32)
    ctr = np.arange((n + 7) // 8, dtype=np.uint64)
    a, b = ctr & low, ctr >> half
    c, d = np.full_like(ctr, offset & _LOW), np.full_like(ctr, offset >> 32)
    key = [seed & _LOW, (seed >> 32) & _LOW]
    for r in range(_ROUNDS):
        first, second = a * u(_M0), c * u(_M1)
        a = (second >> half) ^ b ^ u((key[0] + r * _W0) & _LOW)
        c = (first >> half) ^ d ^ u((key[1] + r * _W1) & _LOW)
        b, d = second & low, first & low
    bits = np.empty((ctr.size, 8), dtype=np.uint16)
    for i, word in enumerate((a, b, c, d)):
        bits[:, 2 * i] = word & u(0xFFFF)
        bits[:, 2 * i + 1] = word >> u(16)
    return bits.reshape(-1)[:n] >= round(rate * 65536)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        x, w, b = s["x"].double(), s["weight"].double(), s["bias"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        h = x.sub_(mean).mul_(torch.rsqrt(var + _EPS))
        out = {"y": torch.addcmul(b, h, w)}
        if case["train"]:
            g = s["grad_y"].double()
            out["grad_weight"], out["grad_bias"] = torch.einsum("rd,rd->d", g, h), torch.einsum("rd->d", g)
            n = case["width"]
            g.mul_(w)
            along = torch.einsum("rd,rd->r", g, h)[:, None] / n
            out["grad_x"] = (g - torch.einsum("rd->r", g)[:, None] / n - h * along) * torch.rsqrt(var + _EPS)
        return out
    if case["op"] == "dropout":
        mask = torch.from_numpy(_exact_mask(s["x"].numel(), case["rate"], int(s["seed"]), s["offset"])).cuda()
        mask = mask.reshape(s["x"].shape).double() / (1 - round(case["rate"] * 65536) / 65536)
        y = s["x"].double() * mask
        out = {"y": y + s["residual"].double() if case["residual"] else y}
        if case["train"]:
            out["grad_x"] = s["grad_y"].double() * mask
        return out
    x, ids, weights = s["x"].to(_DTYPES[case["dtype"]]).double(), s["ids"].tolist(), s["weights"].tolist()
    H = case["hidden"]
    out = torch.zeros(case["tokens"], case["out"], dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        chosen = [(t, w) for t in range(case["tokens"]) for i, w in zip(ids[t], weights[t]) if i == e]
        if not chosen:
            continue
        z = torch.mm(x[[t for t, _ in chosen]], s["up"][e].double().t())
        if case["act"] == "swiglu":
            z = z[:, :H] * torch.sigmoid(z[:, :H]) * z[:, H:]
        elif case["act"] == "silu":
            z = z * torch.sigmoid(z)
        elif case["act"] == "gelu":
            z = z * torch.special.ndtr(z)
        else:
            z = torch.where(z > 0, z, torch.zeros_like(z))
        y = torch.mm(z, s["down"][e].double().t())
        for i, (t, w) in enumerate(chosen):
            out[t] += w * y[i]
    return {"out": out}
