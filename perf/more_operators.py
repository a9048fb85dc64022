"""Measured cases of what closes a training step around the expert layer.

Operators: `balance` and `balance_grad` (per-expert counts, the balance loss and the z-loss of the
router, and their gradient on top of the routing weights'), `norm` (the norm of many gradient tensors
and the factor that clips it) and `adamw` (one AdamW step over many tensors, with states in 32 bits,
or in 8 bits with a scale to 256 values).

With `own` false, `run` computes an operator in plain torch operations in 32 bits (sums over all
gradients and the bias corrections in 64); with `own` true it makes the library's calls.
"""
import math
import random

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
BLOCK = 256      # values that share a scale of the 8-bit states
TOP = 448.0      # largest e4m3 value
HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8)
DECAY = 0.1


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a small layer's router on one short batch: what counts is the call's latency
        dict(name="balance_small", op="balance", T=257, E=16, k=2, dt="f32", score="softmax", B=1, pad=0, z=True),
        # the routing decision of the largest training layer, one loss over the whole batch, with z-loss
        dict(name="balance_train", op="balance", T=16384, E=128, k=8, dt="f32", score="softmax", B=1, pad=0, z=True),
        # sigmoid scores, a loss for each sequence of a ragged packed batch, padded tokens, 16-bit logits
        dict(name="balance_sequences", op="balance", T=65521, E=256, k=8, dt="bf16", score="sigmoid", B=29, pad=311, z=False),
        # the gradient of balance_train's losses on top of the routing weights' gradient
        dict(name="balance_grad_train", op="balance_grad", T=16384, E=128, k=8, dt="f32", score="softmax", B=1, pad=0, z=True,
             add=True),
        # the same for sequences, sigmoid scores, a number of experts that is no multiple of a vector
        dict(name="balance_grad_sequences", op="balance_grad", T=32749, E=250, k=6, dt="bf16", score="sigmoid", B=17, pad=97,
             z=False, add=False),
        # the norm of a router's and the biases' gradients (16-bit, ragged): a latency
        dict(name="norm_small", op="norm", set="ragged", count=5, most=70001, sizes=1, dt="f32", grad="bf16", clip=True),
        # the norm of all weight gradients of a Qwen-shaped layer (128 experts), with the clipping factor
        dict(name="norm_layer", op="norm", set="layer", E=128, H=2048, I=768, dt="f32", grad="f32", clip=True),
        # the step of a small 32-bit layer's tensors: a latency
        dict(name="adamw_small", op="adamw", set="layer", E=4, H=64, I=48, dt="f32", grad="f32", master=False, bits=32, clip=False),
        # a Qwen-shaped layer: 16-bit weights with 32-bit copies, 32-bit states, clipped gradients
        dict(name="adamw_layer", op="adamw", set="layer", E=128, H=2048, I=768, dt="bf16", grad="f32", master=True, bits=32,
             clip=True),
        # the same layer with 8-bit states and no copies: weights and states are rounded at random
        dict(name="adamw_layer_8bit", op="adamw", set="layer", E=128, H=2048, I=768, dt="bf16", grad="f32", master=False, bits=8,
             clip=True),
        # many tensors of odd sizes, 32 bits throughout
        dict(name="adamw_many", op="adamw", set="ragged", count=211, most=300007, sizes=2, dt="f32", grad="f32", master=False,
             bits=32, clip=False),
        # many tensors of odd sizes, 16-bit gradients, 8-bit states
        dict(name="adamw_many_8bit", op="adamw", set="ragged", count=67, most=2000003, sizes=3, dt="f32", grad="bf16",
             master=False, bits=8, clip=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["balance", "balance_grad", "norm", "adamw", "adamw"])
    if op in ("balance", "balance_grad"):
        T = _log(rng, 1, 65536)
        E = rng.choice([rng.choice([2, 4, 8, 16, 32, 60, 64, 96, 128, 160, 200, 256]), rng.randint(2, 256)])
        c = dict(op=op, T=T, E=E, k=min(E, rng.choice([1, 2, 3, 4, 6, 8, 8, 10])), dt=rng.choice(["bf16", "f32"]),
                 score=rng.choice(["softmax", "sigmoid"]), B=rng.choice([1, 1, _log(rng, 1, 200)]),
                 pad=rng.choice([0, 0, T // 13]), z=rng.random() < 0.5)
        if op == "balance_grad":
            c["add"] = rng.random() < 0.5
        return c
    c = dict(op=op)
    if rng.random() < 0.5:
        c.update(set="layer", E=_log(rng, 1, 64), H=8 * _log(rng, 4, 256), I=8 * _log(rng, 4, 96))
    else:
        c.update(set="ragged", count=_log(rng, 1, 300), most=_log(rng, 1, 500000), sizes=rng.randrange(1 << 20))
    if op == "norm":
        c.update(dt="f32", grad=rng.choice(["f32", "bf16"]), clip=rng.random() < 0.7)
        return c
    dt = rng.choice(["f32", "bf16"])
    c.update(dt=dt, grad=rng.choice(["f32", "bf16"]), master=dt == "bf16" and rng.random() < 0.5, bits=rng.choice([32, 8]),
             clip=rng.random() < 0.5)
    return c


def _sizes(c):
    """Numbers of values of the case's tensors."""
    if c["set"] == "layer":  # the experts' two weights and biases, and the router's weight
        E, H, I = c["E"], c["H"], c["I"]
        return [E * 2 * I * H, E * H * I, E * 2 * I, E * H, E * H]
    rng = random.Random(c["sizes"])
    return [_log(rng, 1, c["most"]) for _ in range(c["count"])]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _prepare_balance(c, g):
    T, E, k, B = c["T"], c["E"], c["k"], c["B"]
    z = torch.randn((T, E), generator=g, device="cuda") * 1.3 + 0.5 * torch.randn((1, E), generator=g, device="cuda")
    idx = torch.topk(z, k, dim=1).indices.to(torch.int32)
    if c["pad"]:
        idx[T - c["pad"]:] = -1
    idx[::97, k - 1] = -1  # a slot that found no expert here and there
    off = None
    if B > 1:  # ragged sequences that cover the batch, empty ones among them
        cut = torch.sort(torch.randint(0, T + 1, (B - 1,), generator=g, device="cuda")).values.to(torch.int32)
        off = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), T)]).contiguous()
    dtype = DTYPE[c["dt"]]
    z = z.to(dtype)
    s = dict(logits=z, idx=idx.contiguous(), off=off, coef=0.01, z_coef=0.001 if c["z"] else 0.0)
    counts, stats, _ = _plain_counts(c, s)
    i32, f32 = dict(dtype=torch.int32, device="cuda"), dict(dtype=torch.float32, device="cuda")
    if c["op"] == "balance":
        s.update(counts=torch.empty((B, E), **i32), stats=torch.empty((B + 1, 2), **i32), mean=torch.empty((B, E), **f32),
                 loss=torch.empty(2, **f32), work={})
    else:
        s.update(counts=counts, stats=stats, dloss=torch.rand(2, generator=g, device="cuda") + 0.5,
                 add=(torch.randn((T, E), generator=g, device="cuda") * 1e-6).to(dtype) if c["add"] else None,
                 dlogits=torch.empty((T, E), dtype=dtype, device="cuda"))
    return s


def _prepare_tensors(c, g):
    """All tensors of a kind lie one after the other in one buffer, each from a whole block on."""
    sizes = _sizes(c)
    blocks = [-(-n // BLOCK) for n in sizes]
    first = [0]
    for b in blocks:
        first.append(first[-1] + b)
    total = first[-1] * BLOCK
    per = torch.tensor(blocks, device="cuda")
    tensor_of = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), per)        # of each block
    place = (torch.arange(first[-1], device="cuda") - torch.tensor(first[:-1], device="cuda")[tensor_of]) * BLOCK
    left = torch.tensor(sizes, device="cuda")[tensor_of] - place                             # values from here to the end
    spare = None  # places behind a tensor's end hold zeros
    if any(n % BLOCK for n in sizes):
        ends = torch.nonzero(left < BLOCK).reshape(-1)
        inside = torch.arange(BLOCK, device="cuda")
        at = (ends * BLOCK)[:, None] + inside
        spare = at[inside >= left[ends][:, None]]

    def fill(scale, quiet=False):
        x = torch.randn(total, generator=g, device="cuda") * scale
        if quiet:  # experts that kept no row have no gradient
            x.view(-1, BLOCK)[torch.rand(total // BLOCK, generator=g, device="cuda") < 0.05] = 0
        if spare is not None:
            x[spare] = 0
        return x

    def views(flat):
        return [flat[a * BLOCK:a * BLOCK + n] for a, n in zip(first, sizes)]

    grad = fill(1e-3, quiet=True).to(DTYPE[c["grad"]])
    s = dict(sizes=sizes, views=views, grad=grad, tensor_of=tensor_of, place=place,
             max_norm=0.5 * 1e-3 * math.sqrt(sum(sizes)) if c["clip"] else math.inf)
    if c["op"] == "norm":
        s.update(out=torch.empty(2, device="cuda"), work={})
        return s
    p = fill(0.02)
    s.update(param=p.to(DTYPE[c["dt"]]), step=1000, seed=17, scale=torch.full((1,), 0.5, device="cuda") if c["clip"] else None)
    if c["master"]:
        s["master"] = p
    del p
    m, r = fill(3e-4), fill(1e-3).abs_()
    if c["bits"] == 32:
        s.update(m=m, v=r.square_(), m_scale=None, v_scale=None)
    else:
        for name, x in (("m", m), ("v", r)):
            x = x.view(-1, BLOCK)
            sc = x.abs().amax(1) / TOP
            s[name] = (x / sc.clamp_min(1e-30)[:, None]).to(torch.float8_e4m3fn).reshape(-1)
            s[name + "_scale"] = sc
    s["plan"] = {}
    return s


def prepare(case, seed):
    g = _generator(seed)
    s = _prepare_balance(case, g) if case["op"] in ("balance", "balance_grad") else _prepare_tensors(case, g)
    s["case"] = case
    return s


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _scale_views(s, name):
    """Each tensor's scales, side by side in one buffer."""
    n, out = 0, []
    for size in s["sizes"]:
        b = -(-size // BLOCK)
        out.append(s[name][n:n + b])
        n += b
    return out


def _plan(s, L):
    """The list of tensors, made once as a program that trains does."""
    if "list" not in s["plan"]:
        more = {}
        if s["case"]["bits"] == 8:
            more = dict(m_scale=_scale_views(s, "m_scale"), v_scale=_scale_views(s, "v_scale"))
        if s["case"]["master"]:
            more["master"] = s["views"](s["master"])
        s["plan"]["list"] = L.TensorList(s["views"](s["grad"]), params=s["views"](s["param"]), m=s["views"](s["m"]),
                                         v=s["views"](s["v"]), weight_decay=DECAY, **more)
    return s["plan"]["list"]


def _run_own(s):
    from pruned_expert_backward_lrmoe_b200 import lrmoe as L
    c, op = s["case"], s["case"]["op"]
    if op in ("balance", "balance_grad"):
        how = dict(seq_offsets=s["off"], coef=s["coef"], z_coef=s["z_coef"],
                   score_fn=L.LRMOE_SCORE_SOFTMAX if c["score"] == "softmax" else L.LRMOE_SCORE_SIGMOID)
    if op == "balance":
        if "ws" not in s["work"]:
            n = L.lrmoe_balance_workspace_bytes(c["T"], c["E"], c["B"])
            s["work"]["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        L.lrmoe_balance(s["logits"], s["idx"], s["counts"], s["stats"], s["mean"], s["loss"], s["work"]["ws"], **how)
        return {"counts": s["counts"], "stats": s["stats"], "mean": s["mean"], "loss": s["loss"]}
    if op == "balance_grad":
        L.lrmoe_balance_grad(s["logits"], s["idx"], s["counts"], s["stats"], s["dlogits"], dloss=s["dloss"], add=s["add"], **how)
        return {"dlogits": s["dlogits"]}
    if op == "norm":
        if "ws" not in s["work"]:
            s["work"]["list"] = L.TensorList(s["views"](s["grad"]))
            n = L.lrmoe_grad_norm_workspace_bytes(len(s["sizes"]))
            s["work"]["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        L.lrmoe_grad_norm(s["work"]["list"], s["out"], s["work"]["ws"], max_norm=s["max_norm"])
        return {"out": s["out"]}
    L.lrmoe_adamw(_plan(s, L), step=s["step"], grad_scale=s["scale"], seed=s["seed"], **HYPER)
    return _updated(s)


def _updated(s):
    return {k: s[k] for k in ("param", "master", "m", "v", "m_scale", "v_scale") if s.get(k) is not None}


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_counts(c, s):
    """counts [B][E], stats [B + 1][2] (tokens with a routed slot and pairs of each sequence; in the last row
    all such tokens and the sequences that have one), and each token's sequence (B: it does not count)."""
    T, E, k, B = c["T"], c["E"], c["k"], c["B"]
    idx = s["idx"].long()
    routed = (idx >= 0) & (idx < E)
    tokens = torch.arange(T, device="cuda")
    of = torch.zeros_like(tokens) if s["off"] is None else torch.searchsorted(s["off"][1:].long(), tokens, right=True)
    of = torch.where(routed.any(1), of, B)
    flat = torch.where(routed, of[:, None] * E + idx.clamp(0, E - 1), B * E)
    counts = torch.bincount(flat.reshape(-1), minlength=B * E + 1)[:B * E].view(B, E)
    n = torch.bincount(of, minlength=B + 1)[:B]
    stats = torch.stack([torch.cat([n, n.sum()[None]]), torch.cat([counts.sum(1), (n > 0).sum()[None]])], 1)
    return counts.to(torch.int32), stats.to(torch.int32), of


def _plain_scores(z, kind):
    """Each row's shares of the score, and the logarithm of the sum of its exponentials."""
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    lse = top + torch.log(total)
    if kind == "softmax":
        return e / total, lse
    s = 1 / (1 + torch.exp(-z))
    return s / s.sum(1, keepdim=True), lse


def _plain_balance(s):
    c = s["case"]
    B, E = c["B"], c["E"]
    counts, stats, of = _plain_counts(c, s)
    p, lse = _plain_scores(s["logits"].float(), c["score"])
    sums = torch.zeros((B + 1, E), device="cuda").index_add_(0, of, p)[:B]
    mean = sums / stats[:B, :1].clamp_min(1)
    load = E * counts.float() / stats[:B, 1:].clamp_min(1)
    loss = s["coef"] * (load * mean).sum() / stats[B, 1].clamp_min(1)
    zl = s["z_coef"] * torch.where(of < B, lse[:, 0].square(), 0).sum() / stats[B, 0].clamp_min(1)
    return {"counts": counts, "stats": stats, "mean": mean, "loss": torch.stack([loss, zl])}


def _plain_balance_grad(s):
    c = s["case"]
    B, E = c["B"], c["E"]
    _, _, of = _plain_counts(c, s)
    z = s["logits"].float()
    p, lse = _plain_scores(z, c["score"])
    n, pairs = s["stats"][:B, :1].clamp_min(1).float(), s["stats"][:B, 1:].clamp_min(1).float()
    D = E * s["counts"].float() / (pairs * n * s["stats"][B, 1].clamp_min(1)) * (s["coef"] * s["dloss"][0])
    D = torch.cat([D, D.new_zeros((1, E))])[of]
    dz = p * (D - (D * p).sum(1, keepdim=True))
    if c["score"] == "sigmoid":
        dz = dz / (1 + torch.exp(z))
    if s["z_coef"]:
        e = torch.exp(z - lse)
        dz = dz + torch.where((of < B)[:, None], 2 * s["z_coef"] * s["dloss"][1] / s["stats"][B, 0].clamp_min(1) * lse * e, 0)
    if s["add"] is not None:
        dz = dz + s["add"].float()
    return {"dlogits": dz.to(s["logits"].dtype)}


def _plain_norm(s):
    norm = torch.sqrt(s["grad"].float().square().sum(dtype=torch.float64))
    return {"out": torch.stack([norm, torch.where(norm > s["max_norm"], s["max_norm"] / norm, 1.0)]).float()}


MASK = 0xFFFFFFFF


def _mix(h):
    """32 bits, scrambled (in 64-bit integers)."""
    h = h ^ (h >> 16)
    h = h * 0x9E3779B1 & MASK
    h = h ^ (h >> 15)
    h = h * 0x6A09E667 & MASK
    return h ^ (h >> 16)


def _plain_words(s):
    """A random 32-bit word to each value, from the seed, the step, the tensor's number and the value's place."""
    key = _mix(_mix(_mix(s["seed"]) + s["step"] & MASK) + s["tensor_of"] & MASK)
    start = key + (s["place"] & MASK) + (s["place"] >> 32) * 0x632BE5AB
    return _mix((start[:, None] + torch.arange(BLOCK, device="cuda")) & MASK)


def _plain_round8(x, word16, floor):
    """x >= 0, at most 448, to one of its two e4m3 neighbours, the upper one in word16 + x's fraction > 1;
    with `floor` never to 0 unless x is."""
    low = torch.where(x < 2.0 ** -6, 2.0 ** -6, 0.0)  # there the values are 2^-9 apart
    bits = (x + low).view(torch.int32) + (word16 << 4).to(torch.int32)
    y = ((bits >> 20) << 20).view(torch.float32) - low
    if floor:
        y = torch.where(x > 0, y.clamp_min(2.0 ** -9), y)
    return y.clamp_max(TOP)


def _plain_pack8(x, word16, floor):
    scale = (x.abs().amax(1) / TOP)
    scale = torch.where(scale > 0, scale.clamp_min(2.0 ** -126), 0.0)
    inv = torch.where(scale > 0, 1 / scale, 0.0)[:, None]
    y = _plain_round8(x.abs() * inv, word16, floor)
    return torch.where(x < 0, -y, y).to(torch.float8_e4m3fn).reshape(-1), scale


def _plain_adamw(s):
    c, h = s["case"], HYPER
    eight = c["bits"] == 8
    g = s["grad"].float()
    if s["scale"] is not None:
        g = g * s["scale"]
    m, v = s["m"].float(), s["v"].float()
    if eight:
        m = (m.view(-1, BLOCK) * s["m_scale"][:, None]).view(-1)
        v = (v.view(-1, BLOCK) * s["v_scale"][:, None]).view(-1).square()
    m = h["beta1"] * m + (1 - h["beta1"]) * g
    v = h["beta2"] * v + (1 - h["beta2"]) * g * g
    del g
    c1, c2 = 1 - h["beta1"] ** s["step"], 1 - h["beta2"] ** s["step"]
    p = (s["master"] if c["master"] else s["param"]).float() * (1 - h["lr"] * DECAY)
    p = p - h["lr"] / c1 * m / (torch.sqrt(v) / math.sqrt(c2) + h["eps"])
    word = None
    if eight or (c["dt"] == "bf16" and not c["master"]):
        word = _plain_words(s)
    if c["master"]:
        s["master"].copy_(p)
    if c["dt"] == "bf16" and not c["master"]:
        low = ((word * 0x9E3779B1 & MASK) >> 16).to(torch.int32).view(-1)
        p = ((p.view(torch.int32) + low >> 16) << 16).view(torch.float32)
    s["param"].copy_(p)
    del p
    if not eight:
        s["m"].copy_(m)
        s["v"].copy_(v)
    else:
        for name, x, bits, floor in (("m", m, word & 0xFFFF, False), ("v", torch.sqrt(v), word >> 16, True)):
            q, sc = _plain_pack8(x.view(-1, BLOCK), bits, floor)
            s[name].copy_(q)
            s[name + "_scale"].copy_(sc)
    return _updated(s)


def run(state):
    if own:
        return _run_own(state)
    return {"balance": _plain_balance, "balance_grad": _plain_balance_grad, "norm": _plain_norm,
            "adamw": _plain_adamw}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# work
# ---------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] in ("balance", "balance_grad"):
        b, T, E, k, B = BYTES[c["dt"]], c["T"], c["E"], c["k"], c["B"]
        if c["op"] == "balance":
            return {"bytes": T * E * b + 4 * T * k + 8 * B * E, "flops": 6 * T * E}
        return {"bytes": T * E * b * (3 if c["add"] else 2) + 4 * T * k + 4 * B * E, "flops": 10 * T * E}
    n = sum(_sizes(c))
    if c["op"] == "norm":
        return {"bytes": n * BYTES[c["grad"]], "flops": 2 * n}
    kept = 4 if c["master"] or c["dt"] == "f32" else 2               # the value that the step starts from
    state = 8 if c["bits"] == 32 else 2 + 8 / BLOCK
    return {"bytes": n * (BYTES[c["grad"]] + 2 * kept + (2 if c["master"] else 0) + 2 * state), "flops": 14 * n}


# ---------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------
def _exact_routed(c, s):
    """Sequence and expert of every routed pair, and the sequence of every token that counts (else -1)."""
    idx = s["idx"].long()
    lengths = torch.tensor([c["T"]], device="cuda") if s["off"] is None else (s["off"][1:] - s["off"][:-1]).long()
    of = torch.repeat_interleave(torch.arange(c["B"], device="cuda"), lengths)
    token, slot = torch.nonzero(idx >= 0, as_tuple=True)
    counted = torch.full_like(of, -1)
    counted[token] = of[token]
    return of[token], idx[token, slot], counted


def _exact_balance(c, s):
    B, E = c["B"], c["E"]
    seq, expert, of = _exact_routed(c, s)
    counts = torch.zeros((B, E), dtype=torch.float64, device="cuda")
    counts.index_put_((seq, expert), torch.ones_like(seq, dtype=torch.float64), accumulate=True)
    z = s["logits"].double()
    p = torch.softmax(z, 1) if c["score"] == "softmax" else torch.nn.functional.normalize(torch.sigmoid(z), p=1, dim=1)
    member = torch.nn.functional.one_hot(of + 1, B + 1)[:, 1:].double()
    n = member.sum(0)
    mean = member.t() @ p / n.clamp_min(1)[:, None]
    share = counts / counts.sum(1, keepdim=True).clamp_min(1)
    live = (n > 0).sum().clamp_min(1)
    loss = s["coef"] * E * (share * mean).sum(1).sum() / live
    zl = s["z_coef"] * torch.logsumexp(z, 1)[of >= 0].square().mean().nan_to_num(0.0)
    stats = torch.zeros((B + 1, 2), dtype=torch.int32, device="cuda")
    stats[:B, 0], stats[:B, 1] = n.int(), counts.sum(1).int()
    stats[B, 0], stats[B, 1] = (of >= 0).sum(), (n > 0).sum()
    return {"counts": counts.int(), "stats": stats, "mean": mean, "loss": torch.stack([loss, zl])}


def _exact_balance_grad(c, s):
    """By automatic differentiation of the loss in 64 bits."""
    B, E = c["B"], c["E"]
    seq, expert, of = _exact_routed(c, s)
    z = s["logits"].double().requires_grad_(True)
    p = torch.softmax(z, 1) if c["score"] == "softmax" else torch.nn.functional.normalize(torch.sigmoid(z), p=1, dim=1)
    counts = torch.bincount(seq * E + expert, minlength=B * E).view(B, E).double()
    weight = counts / counts.sum(1, keepdim=True).clamp_min(1) * E
    inside = of >= 0
    n = torch.bincount(of[inside], minlength=B).double()
    weight = weight / n.clamp_min(1)[:, None] / (n > 0).sum().clamp_min(1)
    total = s["dloss"][0].double() * s["coef"] * (weight[of.clamp_min(0)] * p)[inside].sum()
    if s["z_coef"]:
        total = total + s["dloss"][1].double() * s["z_coef"] * torch.logsumexp(z, 1)[inside].square().sum() / inside.sum().clamp_min(1)
    dz, = torch.autograd.grad(total, z)
    return {"dlogits": dz if s["add"] is None else dz + s["add"].double()}


def _wrap(h, mul):
    """The product's low 32 bits, in 32-bit integers."""
    return h * (mul - (1 << 32) if mul >= 1 << 31 else mul)


def _down(h, n):
    """Logical shift of 32-bit integers."""
    return (h >> n) & ((1 << (32 - n)) - 1)


def _exact_mix(h):
    h = _wrap(h ^ _down(h, 16), 0x9E3779B1)
    h = _wrap(h ^ _down(h, 15), 0x6A09E667)
    return h ^ _down(h, 16)


def _i32(n):
    n %= 1 << 32
    return torch.tensor([n - (1 << 32) if n >= 1 << 31 else n], dtype=torch.int32, device="cuda")


def _exact_words(s):
    """Tensor by tensor; the places are below 2^32 here."""
    out = []
    step = _exact_mix(_exact_mix(_i32(s["seed"])) + _i32(s["step"]))
    for i, n in enumerate(s["sizes"]):
        key = _exact_mix(step + _i32(i))
        whole = -(-n // BLOCK) * BLOCK
        out.append(_exact_mix(torch.arange(whole, dtype=torch.int32, device="cuda") + key))
    return torch.cat(out)


def _exact_codes(x, chance, never_zero):
    """Values x / scale, scale = the block's largest / 448, each taken down to a multiple of its step after a
    random part of a step (`chance` 16 bits) is added."""
    x = x.view(-1, BLOCK)
    scale = x.abs().amax(1, keepdim=True) / TOP
    y = torch.where(scale > 0, x.abs() / torch.where(scale > 0, scale, 1.0), 0.0)
    step = torch.exp2(torch.floor(torch.log2(y.clamp_min(2.0 ** -6))) - 3)
    q = torch.floor(y / step + chance.view(-1, BLOCK).double() / 65536) * step
    if never_zero:
        q = torch.where((y > 0) & (q == 0), 2.0 ** -9, q)
    return (q.clamp_max(TOP) * torch.sign(x)).view(-1), scale.view(-1)


def _exact_adamw(c, s):
    h, t = HYPER, s["step"]
    g = s["grad"].double() * (0.5 if c["clip"] else 1.0)
    m, v = s["m"].double(), s["v"].double()
    if c["bits"] == 8:
        m = m * s["m_scale"].double().repeat_interleave(BLOCK)
        v = (v * s["v_scale"].double().repeat_interleave(BLOCK)).square_()
    m.lerp_(g, 1 - h["beta1"])
    v.lerp_(g.square_(), 1 - h["beta2"])
    del g
    p = (s["master"] if c["master"] else s["param"]).double()
    p.mul_(1 - h["lr"] * DECAY)
    root = torch.sqrt(v / (1 - h["beta2"] ** t)).add_(h["eps"])
    p.addcdiv_(m, root, value=-h["lr"] / (1 - h["beta1"] ** t))
    del root
    r = {"param": p}
    if c["master"]:
        r["master"] = p
    if c["bits"] == 32:
        r.update(m=m, v=v)
        return r
    word = _exact_words(s)
    r["m"], r["m_scale"] = _exact_codes(m, word & 0xFFFF, False)
    del m
    r["v"], r["v_scale"] = _exact_codes(v.sqrt_(), _down(word, 16), True)
    return r


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "balance":
        return _exact_balance(case, s)
    if case["op"] == "balance_grad":
        return _exact_balance_grad(case, s)
    if case["op"] == "norm":
        norm = math.sqrt(sum(float(t.double().square().sum()) for t in s["views"](s["grad"])))
        factor = min(1.0, s["max_norm"] / norm) if norm > 0 else 1.0
        return {"out": torch.tensor([norm, factor], dtype=torch.float64)}
    return _exact_adamw(case, s)
