"""Measured cases of the expert layer's forward operators and of the gradients that go with them.

Operators: `route` and `route_grad` (the router's decision from logits and its gradient),
`swiglu` and `linear` (the experts' variable-size products with bias, activation, residual and
scatter in the epilogue), `bias_grad` (the gradient of those products' bias) and `combine` (the
weighted sum of a token's expert outputs on top of the residual stream).

With `own` false, `run` computes an operator in plain torch operations in 32 bits (the router's
selection keys in 64); with `own` true it makes the library's calls.
"""
import math

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a single token of a decode step: what counts is the call's latency
        dict(name="route_one_token", op="route", T=1, E=128, k=8, dt="f32", score="softmax", bias=False,
             groups=1, keep_groups=1, renorm=True, scale=1.0, masked=False),
        # a training batch behind a router that is balanced by a bias on the selection, experts in
        # groups, some experts masked out for some tokens, an odd number of tokens
        dict(name="route_groups", op="route", T=16383, E=256, k=8, dt="bf16", score="sigmoid", bias=True,
             groups=8, keep_groups=4, renorm=True, scale=2.5, masked=True),
        # the router's gradient of a whole training batch (softmax over 128 experts, weights renormalised)
        dict(name="route_grad_train", op="route_grad", T=16384, E=128, k=8, dt="f32", score="softmax",
             renorm=True, scale=1.0),
        # the dense form of that gradient (weights not renormalised: every logit gets one), 16-bit logits
        dict(name="route_grad_dense", op="route_grad", T=8191, E=160, k=6, dt="bf16", score="softmax",
             renorm=False, scale=1.0),
        # the experts' first product in a decode step: a few rows per expert, the weights are what is read
        dict(name="swiglu_decode", op="swiglu", T=16, E=128, k=8, H=2048, I=768, dt="bf16", bias=False, pad=0),
        # the same product of the largest training layer (T = 16384, GLM-shaped)
        dict(name="swiglu_train", op="swiglu", T=16384, E=128, k=8, H=4096, I=1408, dt="bf16", bias=True, pad=0),
        # the experts' second product of a Qwen-shaped training layer, a ragged batch with padded tokens
        dict(name="linear_train", op="linear", T=8111, E=128, k=8, K=768, N=2048, dt="bf16", bias=True,
             residual=False, pad=97),
        # one expert that every token takes, its output added to the residual stream; 32-bit layer
        dict(name="linear_shared_f32", op="linear", T=1021, E=1, k=1, K=256, N=512, dt="f32", bias=True,
             residual=True, pad=0),
        # bias gradients of a training layer's experts
        dict(name="bias_grad_experts", op="bias_grad", T=8192, E=128, k=8, N=1536, dt="bf16", pad=0),
        # the same of one expert that takes every token: one long sum per column
        dict(name="bias_grad_shared", op="bias_grad", T=16381, E=1, k=1, N=4096, dt="bf16", pad=0),
        # a decode step's return to the residual stream
        dict(name="combine_decode", op="combine", T=13, E=128, k=8, H=2048, dt="bf16", residual=True, pad=0),
        # the same of the largest training layer, with empty slots
        dict(name="combine_train", op="combine", T=16384, E=128, k=8, H=4096, dt="bf16", residual=True, pad=501),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _experts(rng, most):
    return rng.choice([e for e in (1, 2, 5, 8, 16, 33, 60, 64, 96, 128, 160, 200, 256, 384, 512) if e <= most])


def draw(rng):
    op = rng.choice(["route", "route_grad", "swiglu", "linear", "bias_grad", "combine"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    if op in ("route", "route_grad"):
        T, E = _log(rng, 1, 32768), rng.choice([_experts(rng, 512), rng.randint(2, 300)])
        k = min(E, rng.choice([1, 2, 3, 4, 6, 8, 8, 10, 16]))
        c = dict(op=op, T=T, E=E, k=k, dt=dt, score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.6,
                 scale=rng.choice([1.0, 2.5, 16.0]))
        if op == "route":
            g = rng.choice([g for g in (1, 1, 2, 4, 8, 16) if E % g == 0])
            keep = rng.randint(-(-k * g // E), g)
            c.update(bias=rng.random() < 0.6, groups=g, keep_groups=keep, masked=rng.random() < 0.4)
        return c
    small = dt == "f32"
    unit = 4 if small else 8
    dim = lambda lo, hi: unit * _log(rng, lo // unit, hi // unit)  # noqa: E731
    T = _log(rng, 1, 1024 if small else 8192)
    E = _experts(rng, 16 if small else 128)
    k = min(E, rng.choice([1, 2, 4, 6, 8]))
    pad = rng.choice([0, 0, T // 9])
    c = dict(op=op, T=T, E=E, k=k, dt=dt, pad=pad)
    if op == "swiglu":
        c.update(H=dim(64, 512 if small else 4096), I=dim(32, 384 if small else 1408), bias=rng.random() < 0.5)
    elif op == "linear":
        c.update(K=dim(32, 384 if small else 1408), N=dim(64, 512 if small else 4096), bias=rng.random() < 0.5,
                 residual=rng.random() < 0.5)
    elif op == "bias_grad":
        c.update(N=dim(32, 4096))
    else:
        c.update(H=dim(32, 4096), residual=rng.random() < 0.7)
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _choose(g, T, E, k, pad):
    """Experts of each token (the more popular ones more often), the last `pad` tokens without any."""
    z = torch.randn((T, E), generator=g, device="cuda") + 0.4 * torch.randn((1, E), generator=g, device="cuda")
    idx = torch.topk(z, k, dim=1).indices.to(torch.int32)
    if pad:
        idx[T - pad:] = -1
    return idx.contiguous()


def _plan(idx, E):
    """The selection's perm and offsets for a forward pass that keeps every pair, and two host numbers."""
    flat = idx.reshape(-1).long()
    order = torch.argsort(torch.where(flat >= 0, flat, E), stable=True).to(torch.int32)
    counts = torch.bincount(flat[flat >= 0], minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=idx.device)
    offsets[1:] = torch.cumsum(counts, 0)
    return order.contiguous(), offsets, int(counts.sum()), max(1, int(counts.max()))


def prepare(case, seed):
    c, g = case, _generator(seed)
    dtype, op, T, E, k = DTYPE[c["dt"]], c["op"], c["T"], c["E"], c["k"]
    s = dict(case=c)
    f32, i32 = dict(dtype=torch.float32, device="cuda"), dict(dtype=torch.int32, device="cuda")
    if op == "route":
        z = _normal(g, (T, E), dtype, 1.3)
        if c["masked"]:  # experts that a token may not take; every 64th token may take none
            hide = torch.rand((T, E), generator=g, device="cuda") < 0.2
            hide |= (torch.arange(T, device="cuda") % 64 == 63)[:, None]
            z = z.masked_fill(hide, -math.inf)
        s.update(logits=z, bias=_normal(g, (E,), torch.float32, 0.05) if c["bias"] else None,
                 idx=torch.empty((T, k), **i32), w=torch.empty((T, k), **f32))
    elif op == "route_grad":
        s.update(logits=_normal(g, (T, E), dtype, 1.3), idx=_choose(g, T, E, k, T // 11),
                 dw=_normal(g, (T, k), torch.float32), dlogits=torch.empty((T, E), dtype=dtype, device="cuda"))
    elif op == "combine":
        s.update(y=_normal(g, (T * k, c["H"]), dtype), idx=_choose(g, T, E, k, c["pad"]),
                 w=torch.rand((T, k), generator=g, device="cuda"),
                 residual=_normal(g, (T, c["H"]), dtype) if c["residual"] else None,
                 Y=torch.empty((T, c["H"]), dtype=dtype, device="cuda"))
    else:
        idx = _choose(g, T, E, k, c["pad"])
        perm, offsets, M, most = _plan(idx, E)
        s.update(perm=perm, offsets=offsets, M=M, most=most)
        zeros = lambda n, d: torch.zeros((n, d), dtype=dtype, device="cuda")  # noqa: E731
        P = T * k
        if op == "swiglu":
            H, I = c["H"], c["I"]
            s.update(x=_normal(g, (T, H), dtype), W=_normal(g, (E, 2 * I, H), dtype, 0.02),
                     bias=_normal(g, (E, 2 * I), dtype, 0.1) if c["bias"] else None,
                     g=zeros(P, I), u=zeros(P, I), a=zeros(P, I), Ap=zeros(P, I))
        elif op == "linear":
            K, N = c["K"], c["N"]
            s.update(rows=_normal(g, (P, K), dtype), W=_normal(g, (E, N, K), dtype, 0.02),
                     bias=_normal(g, (E, N), dtype, 0.1) if c["bias"] else None,
                     residual=_normal(g, (P, N), dtype) if c["residual"] else None, out=zeros(P, N))
        else:
            s.update(rows=_normal(g, (P, c["N"]), dtype, 0.01), db=torch.empty((E, c["N"]), **f32))
    return s


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _run_own(s):
    from pruned_expert_backward_lrmoe_b200 import lrmoe as L
    c = s["case"]
    op = c["op"]
    if op in ("route", "route_grad"):
        how = dict(score_fn=L.LRMOE_SCORE_SOFTMAX if c["score"] == "softmax" else L.LRMOE_SCORE_SIGMOID,
                   renormalise=c["renorm"], scale=c["scale"])
    if op == "route":
        L.lrmoe_route(s["logits"], s["idx"], s["w"], bias=s["bias"], n_group=c["groups"],
                      topk_group=c["keep_groups"], **how)
        return {"idx": s["idx"], "w": s["w"]}
    if op == "route_grad":
        L.lrmoe_route_grad(s["logits"], s["idx"], s["dw"], s["dlogits"], **how)
        return {"dlogits": s["dlogits"]}
    if op == "swiglu":
        L.lrmoe_grouped_swiglu(s["x"], s["W"], s["offsets"], s["Ap"], perm=s["perm"], src_div=c["k"],
                               bias=s["bias"], g=s["g"], u=s["u"], a=s["a"])
        return {"Ap": s["Ap"], "g": s["g"], "u": s["u"], "a": s["a"]}
    if op == "linear":
        L.lrmoe_grouped_linear(s["rows"], s["W"], s["offsets"], s["out"], bias=s["bias"],
                               residual=s["residual"], perm=s["perm"])
        return {"out": s["out"]}
    if op == "bias_grad":
        L.lrmoe_grouped_bias_grad(s["rows"], s["offsets"], s["db"])
        return {"db": s["db"]}
    L.lrmoe_combine(s["y"], s["idx"], s["w"], c["E"], s["Y"], residual=s["residual"])
    return {"Y": s["Y"]}


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_scores(z, kind):
    """Scores of the experts a token may take (logit above -inf); 0 for the others."""
    open_ = z > -math.inf
    if kind == "sigmoid":
        return torch.where(open_, 1 / (1 + torch.exp(-z)), 0), open_
    top = z.amax(1, keepdim=True)
    e = torch.where(open_, torch.exp(z - torch.where(top > -math.inf, top, 0)), 0)
    return e / e.sum(1, keepdim=True).clamp_min(1e-300), open_


def _plain_route(s):
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    score, open_ = _plain_scores(s["logits"].double(), c["score"])  # 64 bits: neighbours in the order are near
    key = score if s["bias"] is None else score + s["bias"].double()
    may = open_
    if G > 1:
        inside = torch.where(open_, key, -math.inf).view(T, G, E // G)
        two = torch.sort(inside, dim=2, descending=True).values[:, :, :2]
        value = torch.where(two > -math.inf, two, 0).sum(2)
        value = torch.where(open_.view(T, G, E // G).any(2), value, -math.inf)
        best = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :c["keep_groups"]]
        kept = torch.zeros((T, G), dtype=torch.bool, device=key.device).scatter_(1, best, True)
        may = open_ & kept[:, :, None].expand(T, G, E // G).reshape(T, E)
    if s["bias"] is None:  # the score rises with the logit
        key = s["logits"].double()
    order = torch.sort(torch.where(may, key, -math.inf), dim=1, descending=True, stable=True).indices[:, :k]
    taken = may.gather(1, order)
    w = torch.where(taken, score.gather(1, order), 0)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    return {"idx": torch.where(taken, order, -1).to(torch.int32), "w": (w * c["scale"]).float()}


def _plain_route_grad(s):
    c = s["case"]
    z, idx = s["logits"].float(), s["idx"].long()
    score, _ = _plain_scores(z, c["score"])
    taken = idx >= 0
    at = idx.clamp_min(0)
    dw = torch.where(taken, s["dw"] * c["scale"], 0)
    if c["renorm"]:
        w = torch.where(taken, score.gather(1, at), 0)
        total = w.sum(1, keepdim=True).clamp_min(1e-30)
        dw = torch.where(taken, (dw - (dw * w).sum(1, keepdim=True) / total) / total, 0)
    ds = torch.zeros_like(z).scatter_add_(1, at, dw)
    if c["score"] == "sigmoid":
        dz = ds * score * (1 - score)
    else:
        dz = score * (ds - (ds * score).sum(1, keepdim=True))
    return {"dlogits": dz.to(s["logits"].dtype)}


def _places(s):
    """Expert and place inside it of every packed row."""
    rows = torch.arange(s["M"], device="cuda")
    e = torch.searchsorted(s["offsets"][1:].long(), rows, right=True)
    return e, rows - s["offsets"].long()[e]


def _plain_product(s, rows):
    """rows[r] . W[e(r)]^T + bias in 32 bits, over the experts' rows side by side."""
    e, j = _places(s)
    W = s["W"].float()
    side = torch.zeros((W.shape[0], s["most"], W.shape[2]), device="cuda")
    side[e, j] = rows.float()
    out = torch.bmm(side, W.transpose(1, 2))[e, j]
    return out if s["bias"] is None else out + s["bias"].float()[e]


def _plain_swiglu(s):
    c, M = s["case"], s["M"]
    at = s["perm"][:M].long()
    gu = _plain_product(s, s["x"][at // c["k"]])
    I = c["I"]
    g, u = gu[:, :I], gu[:, I:]
    a = (g / (1 + torch.exp(-g)) * u).to(s["x"].dtype)
    new = lambda: torch.zeros((c["T"] * c["k"], I), dtype=s["x"].dtype, device="cuda")  # noqa: E731
    Ap, G, U, A = new(), new(), new(), new()
    Ap[:M] = a
    G[at], U[at], A[at] = g.to(G.dtype), u.to(U.dtype), a
    return {"Ap": Ap, "g": G, "u": U, "a": A}


def _plain_linear(s):
    at = s["perm"][:s["M"]].long()
    y = _plain_product(s, s["rows"][:s["M"]])
    if s["residual"] is not None:
        y = y + s["residual"][at].float()
    out = torch.zeros((s["rows"].shape[0], y.shape[1]), dtype=s["rows"].dtype, device="cuda")
    out[at] = y.to(out.dtype)
    return {"out": out}


def _plain_bias_grad(s):
    e, j = _places(s)
    side = torch.zeros((s["case"]["E"], s["most"], s["rows"].shape[1]), device="cuda")
    side[e, j] = s["rows"][:s["M"]].float()
    return {"db": side.sum(1)}


def _plain_combine(s):
    c = s["case"]
    T, k = c["T"], c["k"]
    taken = (s["idx"] >= 0)[:, :, None]
    y = torch.where(taken, s["y"].view(T, k, c["H"]).float(), 0) * s["w"][:, :, None]
    out = y.sum(1)
    if s["residual"] is not None:
        out = out + s["residual"].float()
    return {"Y": out.to(s["y"].dtype)}


def run(state):
    if own:
        return _run_own(state)
    return {"route": _plain_route, "route_grad": _plain_route_grad, "swiglu": _plain_swiglu, "linear": _plain_linear,
            "bias_grad": _plain_bias_grad, "combine": _plain_combine}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# work
# ---------------------------------------------------------------------------
def work(case):
    c = case
    b, T, E, k, op = BYTES[c["dt"]], c["T"], c["E"], c["k"], c["op"]
    if op == "route":
        return {"bytes": T * E * b + (4 * E if c["bias"] else 0) + 8 * T * k, "flops": 4 * T * E}
    if op == "route_grad":
        return {"bytes": 2 * T * E * b + 8 * T * k, "flops": 6 * T * E}
    M = (T - c["pad"]) * k
    read = E * (1 - (1 - k / E) ** (T - c["pad"]))  # experts that any token takes
    if op == "swiglu":
        H, I = c["H"], c["I"]
        n = T * H + read * 2 * I * (H + (1 if c["bias"] else 0)) + 4 * M * I
        return {"bytes": n * b + 4 * M, "flops": 4 * M * H * I}
    if op == "linear":
        K, N = c["K"], c["N"]
        n = M * K + read * N * (K + (1 if c["bias"] else 0)) + M * N * (2 if c["residual"] else 1)
        return {"bytes": n * b + 4 * M, "flops": 2 * M * K * N}
    if op == "bias_grad":
        return {"bytes": M * c["N"] * b + 4 * E * c["N"], "flops": M * c["N"]}
    return {"bytes": (M + T * (2 if c["residual"] else 1)) * c["H"] * b + 8 * T * k, "flops": 2 * M * c["H"]}


# ---------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------
def _exact_route(c, s):
    """Each token for itself: scores, groups by their two best, then the best keys, ties to the lower number."""
    import numpy as np
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    z = s["logits"].double().cpu().numpy()
    b = np.zeros(E) if s["bias"] is None else s["bias"].double().cpu().numpy()
    shut = np.isneginf(z)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if c["score"] == "sigmoid":
            p = np.where(shut, 0.0, np.exp(-np.logaddexp(0.0, -z)))
        else:
            lse = np.logaddexp.reduce(z, axis=1, keepdims=True)
            p = np.where(shut, 0.0, np.exp(z - np.where(np.isneginf(lse), 0.0, lse)))
    order = p + b if s["bias"] is not None else z
    out = shut.copy()
    if G > 1:
        n = E // G
        inside = np.where(shut, -np.inf, p + b).reshape(T, G, n)
        first = inside.max(2)
        rest = inside.copy()
        np.put_along_axis(rest, inside.argmax(2)[:, :, None], -np.inf, 2)
        second = rest.max(2) if n > 1 else np.full_like(first, -np.inf)
        value = first + np.where(np.isneginf(second), 0.0, second)
        rank = np.argsort(np.argsort(-value, axis=1, kind="stable"), axis=1, kind="stable")
        out |= np.repeat(rank >= c["keep_groups"], n, axis=1)
    key = np.where(out, -np.inf, order)
    idx = np.argsort(-key, axis=1, kind="stable")[:, :k]
    shutout = np.take_along_axis(out, idx, 1)
    w = np.where(shutout, 0.0, np.take_along_axis(p, idx, 1))
    if c["renorm"]:
        total = w.sum(1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    return {"idx": np.where(shutout, -1, idx).astype(np.int32), "w": w * c["scale"]}


def _exact_route_grad(c, s):
    """Vector-Jacobian product of the weights, written out over the pairs of a token's slots."""
    z, idx, dw = s["logits"].double(), s["idx"].long(), s["dw"].double() * c["scale"]
    hot = torch.nn.functional.one_hot(idx.clamp_min(0), c["E"]).double() * (idx >= 0)[:, :, None]  # T k E
    p = torch.sigmoid(z) if c["score"] == "sigmoid" else torch.softmax(z, 1)
    slots = torch.einsum("tke,te->tk", hot, p)
    if c["score"] == "sigmoid":
        jac = hot * (p * (1 - p))[:, None, :]
    else:
        jac = slots[:, :, None] * (hot - p[:, None, :])  # d p_slot / d z
    if c["renorm"]:
        total = slots.sum(1, keepdim=True)
        total = torch.where(total > 0, total, 1.0)
        jac = jac / total[:, :, None] - (slots / total ** 2)[:, :, None] * jac.sum(1, keepdim=True)
    return {"dlogits": torch.einsum("tk,tke->te", dw, jac)}


def _exact_rows(s):
    off = s["offsets"].tolist()
    return [(e, off[e], off[e + 1]) for e in range(len(off) - 1) if off[e + 1] > off[e]]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    op = c["op"]
    if op == "route":
        return _exact_route(c, s)
    if op == "route_grad":
        return _exact_route_grad(c, s)
    wide = dict(dtype=torch.float64, device="cuda")
    if op == "swiglu":
        P, I = c["T"] * c["k"], c["I"]
        r = {n: torch.zeros((P, I), **wide) for n in ("Ap", "g", "u", "a")}
        for e, lo, hi in _exact_rows(s):
            at = s["perm"][lo:hi].long()
            gu = s["x"][torch.div(at, c["k"], rounding_mode="floor")].double() @ s["W"][e].double().t()
            if s["bias"] is not None:
                gu += s["bias"][e].double()
            r["g"][at], r["u"][at] = gu[:, :I], gu[:, I:]
            r["Ap"][lo:hi] = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
            r["a"][at] = r["Ap"][lo:hi]
        return r
    if op == "linear":
        out = torch.zeros((s["rows"].shape[0], c["N"]), **wide)
        for e, lo, hi in _exact_rows(s):
            y = s["rows"][lo:hi].double() @ s["W"][e].double().t()
            if s["bias"] is not None:
                y += s["bias"][e].double()
            at = s["perm"][lo:hi].long()
            out[at] = y if s["residual"] is None else y + s["residual"][at].double()
        return {"out": out}
    if op == "bias_grad":
        db = torch.zeros((c["E"], c["N"]), **wide)
        for e, lo, hi in _exact_rows(s):
            db[e] = s["rows"][lo:hi].double().sum(0)
        return {"db": db}
    w = torch.where(s["idx"] >= 0, s["w"].double(), 0.0)
    Y = torch.zeros((c["T"], c["H"]), **wide) if s["residual"] is None else s["residual"].double()
    for j in range(c["k"]):
        Y = Y + w[:, j:j + 1] * s["y"].view(c["T"], c["k"], c["H"])[:, j].double()
    return {"Y": Y}
