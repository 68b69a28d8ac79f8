"""Cases for the expert and update operators of the dense side of a recommender.

The pooled embeddings of a sample (its token here) go to the experts its router
chose, through the experts' products and back, weighted; the experts' weights
are stepped by an orthogonalised update.  Four kinds of case:

  dispatch   expert ids -> the plan (tokens sorted by expert), the tokens' rows
             in expert order and, in training, the gradient of the tokens
  combine    rows in expert order -> tokens, weighted, and in training the
             gradients of the rows and of the weights
  linear     each expert's product with its own weights over its own rows, and
             in training the gradients of the rows and of the weights
  orthogonal a batch of matrices orthogonalised by Newton-Schulz products

`own` false: plain torch operations in 32 bits, rounded once at the end.
`own` true: this package's calls.
"""
import math

import torch

own = False

_DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}
_A, _B, _C = 3.4445, -4.7750, 2.0315   # the quintic's coefficients
_EPS = 1e-7


# --------------------------------------------------------------------------- #
# cases
# --------------------------------------------------------------------------- #
def listed():
    return [
        # one request's sample: its 26 pooled features of 128 to 2 of 16 experts; latency
        dict(name="dispatch_request", op="dispatch", tokens=1, k=2, experts=16, width=3328, src="bf16",
             dtype="bf16", dropped=0.0, train=False),
        # a training batch of the 26 x 128 model, from the layer's fp32 output to bf16 rows and back
        dict(name="dispatch_train", op="dispatch", tokens=16384, k=2, experts=32, width=3328, src="f32",
             dtype="bf16", dropped=0.02, train=True),
        # a few samples, experts' outputs of an odd width, 4 experts each
        dict(name="combine_request", op="combine", tokens=3, k=4, experts=16, width=777, dtype="f16",
             dropped=0.0, train=False),
        # a training batch whose capacity drops assignments, forward and both gradients
        dict(name="combine_train", op="combine", tokens=32768, k=4, experts=64, width=2048, dtype="bf16",
             dropped=0.05, train=True),
        # one sample through 2 of 16 experts: a product of single rows, bound by the weights
        dict(name="linear_request", op="linear", tokens=1, k=2, experts=16, width=3328, out=1024, dtype="bf16",
             dropped=0.0, train=False),
        # a serving batch of a few samples: about 3 rows an expert, every expert's weights read
        dict(name="linear_serve", op="linear", tokens=48, k=4, experts=64, width=1024, out=2048, dtype="f16",
             dropped=0.0, train=False),
        # odd counts, widths that fill no tile, dropped assignments; forward and both gradients
        dict(name="linear_ragged", op="linear", tokens=1777, k=2, experts=12, width=1032, out=776, dtype="f16",
             dropped=0.3, train=True),
        # inference over a batch of the 26 x 128 model
        dict(name="linear_batch", op="linear", tokens=16384, k=2, experts=16, width=3328, out=1024, dtype="bf16",
             dropped=0.0, train=False),
        # a training batch: forward and both gradients, large enough to be bound by the tensor cores
        dict(name="linear_train", op="linear", tokens=32768, k=2, experts=32, width=1024, out=4096, dtype="bf16",
             dropped=0.02, train=True),
        # many small experts' updates at once
        dict(name="orthogonal_small", op="orthogonal", batch=32, rows=128, cols=256, dtype="bf16", steps=5,
             spectrum="flat"),
        # one tall matrix of odd sizes, fp32 momentum
        dict(name="orthogonal_odd", op="orthogonal", batch=1, rows=1777, cols=519, dtype="f32", steps=5,
             spectrum="decay"),
        # the 16 experts of linear_batch
        dict(name="orthogonal_experts", op="orthogonal", batch=16, rows=1024, cols=3328, dtype="bf16", steps=5,
             spectrum="decay"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi, unit=1):
    """An odd multiple of `unit` (sizes that fill no tile), or, one time in three, a power of two."""
    if rng.random() < 1 / 3:
        return 2 ** rng.randint(math.ceil(math.log2(lo)), math.floor(math.log2(hi)))
    return unit * (2 * (_log_int(rng, lo, hi) // (2 * unit)) + 1)


def _draw_once(rng):
    op = rng.choice(["dispatch", "combine", "linear", "orthogonal"])
    if op == "orthogonal":
        return dict(op=op, batch=_log_int(rng, 1, 32), rows=_size(rng, 24, 3327), cols=_size(rng, 24, 3327),
                    dtype=rng.choice(["bf16", "bf16", "f32", "f16"]), steps=rng.choice([5, 5, 3, 6]),
                    spectrum=rng.choice(["flat", "decay"]))
    experts, tokens = _log_int(rng, 2, 128), _size(rng, 1, 32767)
    c = dict(op=op, tokens=tokens, k=min(experts, rng.choice([1, 2, 2, 3, 4, 6, 8])), experts=experts,
             dtype=rng.choice(["bf16", "bf16", "f16"]), dropped=rng.choice([0.0, 0.02, 0.3]) if tokens >= 8 else 0.0,
             train=rng.random() < 0.6)
    if op == "linear":
        c["width"], c["out"] = _size(rng, 64, 4096, 8), _size(rng, 64, 4096, 8)
    else:
        c["width"] = _size(rng, 32, 3327, rng.choice([1, 8, 8]))
    if op == "dispatch":
        c["src"] = rng.choice(["f32", c["dtype"]])
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
            # the largest weight array a drawn case may hold: that of the listed cases
            if c["op"] != "linear" or c["experts"] * c["width"] * c["out"] <= 32 * 1024 * 4096:
                return c


# --------------------------------------------------------------------------- #
# inputs
# --------------------------------------------------------------------------- #
def _route(case, g):
    """A router's choice: k distinct experts a token, some experts more liked than others; `dropped` of the
    assignments lost to the experts' capacity (id -1), and then the whole first token."""
    T, k, E = case["tokens"], case["k"], case["experts"]
    liked = 0.4 * torch.randn(E, generator=g, device="cuda")
    scores = torch.randn(T, E, generator=g, device="cuda") + liked
    top, ids = torch.topk(scores, k, dim=1)
    weights = torch.softmax(top, dim=1)
    if case["dropped"] > 0:
        lost = torch.rand(T, k, generator=g, device="cuda") < case["dropped"]
        lost[0] = True
        ids = torch.where(lost, torch.full_like(ids, -1), ids)
    return ids.to(torch.int32), weights.float().contiguous()


def _plan(ids, E):
    """offsets[E + 1], src[T * k] and pos[T, k] of a stable sort by expert; assignments without one go last."""
    T, k = ids.shape
    flat = ids.reshape(-1).long()
    valid = (flat >= 0) & (flat < E)
    key = torch.where(valid, flat, torch.full_like(flat, E))
    order = torch.argsort(key, stable=True)
    offsets = torch.searchsorted(key[order], torch.arange(E + 1, device=ids.device))
    at = torch.empty_like(order)
    at[order] = torch.arange(T * k, device=ids.device)
    src = torch.where(torch.arange(T * k, device=ids.device) < offsets[E], order, torch.full_like(order, -1))
    pos = torch.where(valid, at, torch.full_like(at, -1)).reshape(T, k)
    return offsets.int(), src.int(), pos.int()


def _normal(g, *shape, dtype, scale=1.0):
    x = torch.randn(*shape, generator=g, device="cuda")
    return x.mul_(scale).to(_DTYPES[dtype])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": case}
    if case["op"] == "orthogonal":
        B, M, N = case["batch"], case["rows"], case["cols"]
        if case["spectrum"] == "flat":
            G = torch.randn(B, M, N, generator=g, device="cuda")
        else:   # a gradient's spectrum: summed outer products that fall off, over noise
            r = min(M, N, 64)
            fall = torch.arange(1, r + 1, device="cuda", dtype=torch.float32).pow(-0.75)
            G = torch.randn(B, M, r, generator=g, device="cuda") * fall @ torch.randn(B, r, N, generator=g, device="cuda")
            G += 0.3 * torch.randn(B, M, N, generator=g, device="cuda")
        s["update"] = (G * 1e-2).to(_DTYPES[case["dtype"]])
        return s
    T, k, E, D = case["tokens"], case["k"], case["experts"], case["width"]
    ids, weights = _route(case, g)
    if case["op"] == "dispatch":
        s["ids"] = ids
        s["x"] = _normal(g, T, D, dtype=case["src"])
        if case["train"]:
            s["grad_rows"] = _normal(g, T * k, D, dtype=case["dtype"])
        return s
    offsets, src, pos = _plan(ids, E)
    s.update(offsets=offsets, src=src, pos=pos)
    kept = int(offsets[E])
    if case["op"] == "combine":
        s["weights"] = weights
        s["rows"] = _normal(g, T * k, D, dtype=case["dtype"])
        if case["train"]:
            s["grad_out"] = _normal(g, T, D, dtype=case["dtype"])
        return s
    # linear: rows past the last group are zero, as a dispatch leaves them
    counts = (offsets[1:] - offsets[:-1]).cpu()
    s["capacity"] = max(1, int(counts.max()))
    s["active"] = torch.nonzero(counts).reshape(-1).cuda()
    s["rows"] = _normal(g, T * k, D, dtype=case["dtype"])
    s["rows"][kept:] = 0
    s["weight"] = _normal(g, E, case["out"], D, dtype=case["dtype"], scale=1 / math.sqrt(D))
    if case["train"]:
        s["grad_rows"] = _normal(g, T * k, case["out"], dtype=case["dtype"])
        s["grad_rows"][kept:] = 0
    return s


# --------------------------------------------------------------------------- #
# the plain forms
# --------------------------------------------------------------------------- #
def _plain_dispatch(s):
    case, ids, x = s["case"], s["ids"], s["x"]
    k, dt = case["k"], _DTYPES[case["dtype"]]
    offsets, src, pos = _plan(ids, case["experts"])
    at = src.long()
    rows = x[(at.clamp(min=0) // k)] * (at >= 0)[:, None]
    out = {"offsets": offsets, "src": src, "pos": pos, "rows": rows.to(dt)}
    if case["train"]:
        p = pos.long()
        g = s["grad_rows"][p.clamp(min=0)].float() * (p >= 0)[:, :, None]
        out["grad_x"] = g.sum(1).to(x.dtype)
    return out


def _plain_combine(s):
    case, p = s["case"], s["pos"].long()
    dt = _DTYPES[case["dtype"]]
    y = s["rows"][p.clamp(min=0)].float() * (p >= 0)[:, :, None]
    w = s["weights"] * (p >= 0)
    out = {"out": (y * w[:, :, None]).sum(1).to(dt)}
    if case["train"]:
        g = s["grad_out"].float()
        out["grad_weights"] = (y * g[:, None, :]).sum(2)
        at = s["src"].long().clamp(min=0)
        scale = (w.reshape(-1)[at] * (s["src"] >= 0))[:, None]
        out["grad_rows"] = (g[at // case["k"]] * scale).to(dt)
    return out


def _plain_linear(s):
    case, off = s["case"], s["offsets"].long()
    dt, active, cap = _DTYPES[case["dtype"]], s["active"], s["capacity"]
    P, E = case["tokens"] * case["k"], case["experts"]
    # the active experts' rows, padded to the largest group
    lane = torch.arange(cap, device="cuda")
    first, count = off[active], off[active + 1] - off[active]
    mask = lane[None, :] < count[:, None]
    idx = torch.where(mask, first[:, None] + lane[None, :], 0)
    x = s["rows"].float()[idx] * mask[:, :, None]
    w = s["weight"][active].float()
    # where each row's product stands in the padded array
    r = torch.arange(P, device="cuda")
    e = torch.searchsorted(off[1:], r, right=True).clamp(max=E - 1)
    slot = torch.zeros(E, dtype=torch.long, device="cuda")
    slot[active] = torch.arange(active.numel(), device="cuda")
    back = torch.where(r < off[E], slot[e] * cap + r - off[e], 0)
    kept = (r < off[E])[:, None]

    def unpad(y):
        return (y.reshape(-1, y.shape[2])[back] * kept).to(dt)

    if not active.numel():
        out = {"rows": torch.zeros(P, case["out"], dtype=dt, device="cuda")}
        if case["train"]:
            out["grad_in"], out["grad_weight"] = torch.zeros_like(s["rows"]), torch.zeros_like(s["weight"])
        return out
    out = {"rows": unpad(x @ w.transpose(1, 2))}
    if case["train"]:
        g = s["grad_rows"].float()[idx] * mask[:, :, None]
        out["grad_in"] = unpad(g @ w)
        grad_weight = torch.zeros(s["weight"].shape, device="cuda")
        grad_weight[active] = g.transpose(1, 2) @ x
        out["grad_weight"] = grad_weight.to(dt)
    return out


def _plain_orthogonal(s):
    case, X = s["case"], s["update"].float()
    tall = case["rows"] > case["cols"]
    if tall:
        X = X.transpose(1, 2)
    X = X / (X.square().sum((1, 2), keepdim=True).sqrt() + _EPS)
    for _ in range(case["steps"]):
        A = X @ X.transpose(1, 2)
        X = _A * X + (_B * A + _C * (A @ A)) @ X
    return (X.transpose(1, 2) if tall else X).to(torch.bfloat16).contiguous()


# --------------------------------------------------------------------------- #
# one pass
# --------------------------------------------------------------------------- #
def _own(s):
    import dlrm_sparse_embedding_gb300 as emb
    case = s["case"]
    if case["op"] == "orthogonal":
        return emb.orthogonalize(s["update"], steps=case["steps"], coefficients=(_A, _B, _C), eps=_EPS)
    dt = _DTYPES[case["dtype"]]
    if case["op"] == "dispatch":
        plan = emb.expert_sort(s["ids"], case["experts"])
        out = {"offsets": plan.offsets, "src": plan.src, "pos": plan.pos,
               "rows": emb.expert_dispatch(plan, s["x"], dtype=dt)}
        if case["train"]:
            out["grad_x"] = emb.expert_dispatch_grad(plan, s["grad_rows"], dtype=s["x"].dtype)
        return out
    plan = emb.ExpertPlan(s["offsets"], s["src"], s["pos"])
    if case["op"] == "combine":
        out = {"out": emb.expert_combine(plan, s["rows"], s["weights"])}
        if case["train"]:
            out["grad_rows"], out["grad_weights"] = emb.expert_combine_grad(plan, s["grad_out"], s["rows"], s["weights"])
        return out
    out = {"rows": emb.expert_linear(plan, s["rows"], s["weight"])}
    if case["train"]:
        out["grad_in"], out["grad_weight"] = emb.expert_linear_grad(plan, s["grad_rows"], s["rows"], s["weight"])
    return out


def run(state):
    if own:
        return _own(state)
    return {"dispatch": _plain_dispatch, "combine": _plain_combine, "linear": _plain_linear,
            "orthogonal": _plain_orthogonal}[state["case"]["op"]](state)


# --------------------------------------------------------------------------- #
# what a pass cannot do without
# --------------------------------------------------------------------------- #
def work(case):
    op = case["op"]
    if op == "orthogonal":
        m, n = sorted((case["rows"], case["cols"]))
        # a step: X X^T and A A are symmetric (half of 2 m m n and of 2 m m m), the last product is whole
        flops = case["batch"] * case["steps"] * (m * m * n + m * m * m + 2.0 * m * m * n)
        return {"bytes": case["batch"] * m * n * (_BYTES[case["dtype"]] + 2.0), "flops": flops}
    T, k, D, b = case["tokens"], case["k"], case["width"], _BYTES[case["dtype"]]
    P = T * k
    kept = P * (1 - case["dropped"])
    plan = 4.0 * (2 * P + case["experts"] + 1)
    if op == "dispatch":
        sb = _BYTES[case["src"]]
        n = 4.0 * P + plan + sb * T * D + b * P * D            # ids; plan; tokens; rows
        if case["train"]:
            n += b * kept * D + sb * T * D                     # rows' gradient; tokens' gradient
        return {"bytes": n, "flops": kept * D if case["train"] else 0.0}
    if op == "combine":
        n = 4.0 * P + 4.0 * P + b * kept * D + b * T * D       # pos, weights; rows; tokens
        flops = 2.0 * kept * D
        if case["train"]:
            n += b * T * D + b * P * D + 4.0 * P               # tokens' gradient; rows' and weights' gradients
            flops += 3.0 * kept * D
        return {"bytes": n, "flops": flops}
    E, N = case["experts"], case["out"]
    active = E * (1 - (1 - k / E) ** T) if k < E else E
    n = b * (kept * D + active * N * D + P * N) + 4.0 * (E + 1)
    flops = 2.0 * kept * D * N
    if case["train"]:
        n += b * (kept * N + P * D + E * N * D)
        flops *= 3
    return {"bytes": n, "flops": flops}


# --------------------------------------------------------------------------- #
# the definitions in 64 bits
# --------------------------------------------------------------------------- #
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "orthogonal":
        done = []
        for G in s["update"].double():
            X = G / (torch.linalg.norm(G) + _EPS)
            for _ in range(case["steps"]):
                if X.shape[0] <= X.shape[1]:
                    S = torch.mm(X, X.t())
                    X = torch.addmm(X, torch.addmm(S, S, S, beta=_B, alpha=_C), X, beta=_A)
                else:
                    S = torch.mm(X.t(), X)
                    X = torch.addmm(X, X, torch.addmm(S, S, S, beta=_B, alpha=_C), beta=_A)
            done.append(X)
        return torch.stack(done)
    T, k, E, D = case["tokens"], case["k"], case["experts"], case["width"]
    if case["op"] == "dispatch":
        ids = s["ids"].cpu().reshape(-1).tolist()
        groups = [[] for _ in range(E)]
        for a, e in enumerate(ids):
            if 0 <= e < E:
                groups[e].append(a)
        order = [a for grp in groups for a in grp]
        offsets, pos = [0], [-1] * len(ids)
        for grp in groups:
            offsets.append(offsets[-1] + len(grp))
        for p, a in enumerate(order):
            pos[a] = p
        i32 = dict(dtype=torch.int32, device="cuda")
        rows = torch.zeros(T * k, D, dtype=torch.float64, device="cuda")
        token = torch.tensor([a // k for a in order], dtype=torch.long, device="cuda")
        rows[:len(order)] = s["x"].double()[token]
        out = {"offsets": torch.tensor(offsets, **i32),
               "src": torch.tensor(order + [-1] * (len(ids) - len(order)), **i32),
               "pos": torch.tensor(pos, **i32).reshape(T, k), "rows": rows}
        if case["train"]:
            dx = torch.zeros(T, D, dtype=torch.float64, device="cuda")
            p = out["pos"].long()
            for j in range(k):
                has = torch.nonzero(p[:, j] >= 0).reshape(-1)
                dx[has] += s["grad_rows"][p[has, j]].double()
            out["grad_x"] = dx
        return out
    if case["op"] == "combine":
        p, w = s["pos"].long(), s["weights"].double()
        out = torch.zeros(T, D, dtype=torch.float64, device="cuda")
        dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
        drows = torch.zeros(T * k, D, dtype=torch.float64, device="cuda")
        for j in range(k):
            has = torch.nonzero(p[:, j] >= 0).reshape(-1)
            y = s["rows"][p[has, j]].double()
            out[has] += w[has, j, None] * y
            if case["train"]:
                gr = s["grad_out"][has].double()
                dw[has, j] = torch.einsum("td,td->t", gr, y)
                drows[p[has, j]] = w[has, j, None] * gr
        return {"out": out, "grad_rows": drows, "grad_weights": dw} if case["train"] else {"out": out}
    off = s["offsets"].tolist()
    f64 = dict(dtype=torch.float64, device="cuda")
    y = torch.zeros(T * k, case["out"], **f64)
    dx = torch.zeros(T * k, D, **f64) if case["train"] else None
    dW = torch.zeros(E, case["out"], D, **f64) if case["train"] else None
    for e in range(E):
        a, b = off[e], off[e + 1]
        if a < b:
            W, x = s["weight"][e].double(), s["rows"][a:b].double()
            y[a:b] = torch.mm(x, W.t())
            if case["train"]:
                g = s["grad_rows"][a:b].double()
                dx[a:b], dW[e] = torch.mm(g, W), torch.mm(g.t(), x)
    return {"rows": y, "grad_in": dx, "grad_weight": dW} if case["train"] else {"rows": y}
