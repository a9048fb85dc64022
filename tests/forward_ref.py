"""Plain 64-bit forms of the layer's forward operators and of their gradients (numpy), for tests.

They restate the definitions in include/lrmoe.h one token or one expert at a time and share no
code with the library.  tests/test_forward_cpu.py pins them to worked examples, brute force and
finite differences.
"""
from __future__ import annotations

import numpy as np

BAD_EXPERT, NONFINITE, BAD_INDEX = 1, 4, 16
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}  # half a step of the type, relative to the value


def scores(z, kind: str):
    """Scores of one token's logits (float64; entries that are not finite: 0)."""
    ok = np.isfinite(z)
    s = np.zeros_like(z)
    if not ok.any():
        return s
    if kind == "sigmoid":
        s[ok] = np.exp(-np.logaddexp(0.0, -z[ok]))
    else:
        e = np.exp(z[ok] - z[ok].max())
        s[ok] = e / e.sum()
    return s


def route(z, k, bias=None, kind="softmax", n_group=1, topk_group=1, renorm=True, scale=1.0):
    """(idx [T][k], w [T][k] float64, status) of logits z [T][E]."""
    z = np.asarray(z, np.float64)
    T, E = z.shape
    n = E // n_group
    idx = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    status = 0
    b = np.zeros(E) if bias is None else np.asarray(bias, np.float64)
    if np.isnan(z).any() or np.isposinf(z).any() or np.isnan(b).any() or np.isposinf(b).any():
        status |= NONFINITE
    for t in range(T):
        s = scores(z[t], kind)
        open_ = np.isfinite(z[t]) & np.isfinite(b)
        key = {e: float(s[e] + b[e]) for e in range(E) if open_[e]}
        values = []
        for g in range(n_group):
            best = sorted((key[e] for e in range(g * n, (g + 1) * n) if e in key), reverse=True)[:2]
            if best:
                values.append((-sum(best), g))
        kept = {g for _, g in sorted(values)[:topk_group]}
        order = {e: (z[t, e] if bias is None else c) for e, c in key.items() if e // n in kept}
        chosen = sorted(order, key=lambda e: (-order[e], e))[:k]
        idx[t, :len(chosen)] = chosen
        ws = s[chosen]
        if renorm and len(chosen):
            # relative to the largest: exact where all scores are tiny
            log = z[t, chosen] if kind == "softmax" else -np.logaddexp(0.0, -z[t, chosen])
            ws = np.exp(log - log.max())
            ws = ws / ws.sum()
        w[t, :len(chosen)] = scale * ws
    return idx, w, status


def weights(z, idx, kind, renorm, scale):
    """Weights of given slots as a function of the logits (for differences); z [T][E] finite."""
    T, k = idx.shape
    w = np.zeros((T, k))
    for t in range(T):
        s = scores(z[t], kind)
        on = idx[t] >= 0
        ws = s[idx[t][on]]
        w[t, on] = scale * (ws / ws.sum() if renorm and on.any() else ws)
    return w


def route_grad(z, idx, dw, kind="softmax", renorm=True, scale=1.0):
    """dz [T][E] float64 and the status word."""
    z, dw = np.asarray(z, np.float64), np.asarray(dw, np.float64).reshape(idx.shape)
    T, E = z.shape
    dz = np.zeros((T, E))
    status = 0
    for t in range(T):
        s = scores(z[t], kind)
        if kind == "softmax" and not renorm and (np.isnan(z[t]).any() or np.isposinf(z[t]).any()):
            status |= NONFINITE
        slots = []
        for j in range(idx.shape[1]):
            e = idx[t, j]
            if e >= E:
                status |= BAD_EXPERT
            elif e >= 0 and not np.isfinite(z[t, e]):
                if not np.isneginf(z[t, e]):
                    status |= NONFINITE
            elif e >= 0:
                slots.append((e, scale * dw[t, j]))
        D = np.zeros(E)
        if renorm and slots:
            total = sum(s[e] for e, _ in slots)
            mean = sum(d * s[e] for e, d in slots) / total
            slots = [(e, (d - mean) / total) for e, d in slots]
        for e, d in slots:
            D[e] += d
        dz[t] = s * (1 - s) * D if kind == "sigmoid" else s * (D - (D * s).sum())
    return dz, status


def product(rows, W, offsets, bias=None):
    """(rows[r] . W[e]^T + bias[e], sum_k |rows W| + |bias|) for packed rows; NaN elsewhere."""
    rows, W = np.asarray(rows, np.float64), np.asarray(W, np.float64)
    out = np.full((rows.shape[0], W.shape[1]), np.nan)
    mag = np.zeros_like(out)
    for e in range(W.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        out[lo:hi] = rows[lo:hi] @ W[e].T
        mag[lo:hi] = np.abs(rows[lo:hi]) @ np.abs(W[e]).T
        if bias is not None:
            out[lo:hi] += np.asarray(bias, np.float64)[e]
            mag[lo:hi] += np.abs(np.asarray(bias, np.float64)[e])
    return out, mag


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g))


def combine(y, idx, w, E, residual=None):
    """(Y [T][H], sum of magnitudes) of y [T*k][H]."""
    T, k = idx.shape
    H = y.shape[-1]
    out = np.zeros((T, H)) if residual is None else np.asarray(residual, np.float64).copy()
    mag = np.abs(out)
    for t in range(T):
        for j in range(k):
            if 0 <= idx[t, j] < E:
                v = float(w[t, j]) * np.asarray(y[t * k + j], np.float64)
                out[t] += v
                mag[t] += np.abs(v)
    return out, mag


def bias_grad(rows, offsets, E):
    rows = np.asarray(rows, np.float64)
    db = np.zeros((E, rows.shape[1]))
    mag = np.zeros_like(db)
    for e in range(E):
        db[e] = rows[offsets[e]:offsets[e + 1]].sum(0)
        mag[e] = np.abs(rows[offsets[e]:offsets[e + 1]]).sum(0)
    return db, mag


def plan_of(idx, E):
    """perm [T*k], offsets [E+1] of a selection that keeps every pair."""
    flat = idx.reshape(-1)
    order = np.argsort(np.where((flat >= 0) & (flat < E), flat, E), kind="stable").astype(np.int32)
    counts = np.bincount(flat[(flat >= 0) & (flat < E)], minlength=E)
    return order, np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
