"""Plain 64-bit forms of the router's losses, the gradient norm and the AdamW step (numpy), for tests.

They restate the definitions in include/lrmoe.h one token or one tensor at a time and share no code
with the library.  tests/test_step_cpu.py pins them to worked examples and finite differences.
"""
from __future__ import annotations

import numpy as np

from tests.forward_ref import BAD_EXPERT, NONFINITE

BLOCK = 256


# ---------------------------------------------------------------------------
# balance
# ---------------------------------------------------------------------------
def shares(z, kind):
    """(p, 1 - sigmoid or None, softmax, lse) of one token's logits; entries that are not finite: 0."""
    ok = np.isfinite(z)
    p, soft = np.zeros_like(z), np.zeros_like(z)
    if not ok.any():
        return p, p, soft, 0.0
    top = z[ok].max()
    soft[ok] = np.exp(z[ok] - top)
    lse = top + np.log(soft.sum())
    soft /= soft.sum()
    if kind == "softmax":
        return soft, np.ones_like(z), soft, lse
    log_s = -np.logaddexp(0.0, -z[ok])
    p[ok] = np.exp(log_s - log_s.max())
    p /= p.sum()
    rest = np.zeros_like(z)
    rest[ok] = np.exp(-np.logaddexp(0.0, z[ok]))
    return p, rest, soft, lse


def balance(z, idx, off=None, kind="softmax", coef=1.0, z_coef=0.0):
    """dict of counts, stats, mean, loss, status, and (n tokens' shares) for logits z [T][E]."""
    z = np.asarray(z, np.float64)
    T, E = z.shape
    off = [0, T] if off is None else [int(o) for o in off]
    B = len(off) - 1
    counts, stats = np.zeros((B, E), np.int64), np.zeros((B + 1, 2), np.int64)
    mean, zz, status, per = np.zeros((B, E)), 0.0, 0, np.zeros(B)
    if (idx >= E).any():
        status |= BAD_EXPERT
    if off[-1] > off[0] and not (z[off[0]:off[-1]] < np.inf).all():
        status |= NONFINITE
    for b in range(B):
        for t in range(off[b], off[b + 1]):
            named = [e for e in idx[t] if 0 <= e < E]
            if not named:
                continue
            for e in named:
                counts[b, e] += 1
            p, _, _, lse = shares(z[t], kind)
            mean[b] += p
            zz += lse * lse
            stats[b, 0] += 1
        stats[b, 1] = counts[b].sum()
        if stats[b, 0]:
            mean[b] /= stats[b, 0]
            per[b] = E * (counts[b] * mean[b]).sum() / stats[b, 1]
    stats[B] = stats[:B, 0].sum(), (stats[:B, 0] > 0).sum()
    loss = np.array([coef * per.sum() / stats[B, 1] if stats[B, 1] else 0.0,
                     z_coef * zz / stats[B, 0] if stats[B, 0] else 0.0])
    return dict(counts=counts, stats=stats, mean=mean, loss=loss, status=status)


def balance_grad(z, idx, off=None, kind="softmax", coef=1.0, z_coef=0.0, dloss=(1.0, 1.0), add=None):
    """(dz [T][E], magnitude [T][E]: the sizes of the terms of each element)."""
    z = np.asarray(z, np.float64)
    T, E = z.shape
    r = balance(z, idx, off, kind, coef, z_coef)
    off = [0, T] if off is None else [int(o) for o in off]
    dz = np.zeros_like(z) if add is None else np.array(add, np.float64)
    mag = np.abs(dz)
    N, live = r["stats"][-1]
    for b in range(len(off) - 1):
        n, m = r["stats"][b]
        for t in range(off[b], off[b + 1]):
            if not any(0 <= e < E for e in idx[t]):
                continue
            p, rest, soft, lse = shares(z[t], kind)
            D = dloss[0] * coef * E * r["counts"][b] / (m * n * live)
            dot = (D * p).sum()
            zt = 2 * dloss[1] * z_coef * lse / N
            dz[t] += p * rest * (D - dot) + zt * soft
            mag[t] += p * rest * (abs(D) + abs(dot)) + abs(zt) * soft
    return dz, mag


# ---------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------
def mix(h):
    h = np.asarray(h, np.uint64) & 0xFFFFFFFF
    h ^= h >> np.uint64(16)
    h = h * np.uint64(0x9E3779B1) & np.uint64(0xFFFFFFFF)
    h ^= h >> np.uint64(15)
    h = h * np.uint64(0x6A09E667) & np.uint64(0xFFFFFFFF)
    return h ^ (h >> np.uint64(16))


def words(seed, step, i, n, first=0):
    """The random words of values first .. first + n of tensor i."""
    key = mix(mix(mix(seed) + np.uint64(step)) + np.uint64(i))
    e = np.arange(first, first + n, dtype=np.uint64)
    return mix(key + (e & np.uint64(0xFFFFFFFF)) + (e >> np.uint64(32)) * np.uint64(0x632BE5AB))


def adamw(p, g, m, v, lr, step, beta1=0.9, beta2=0.999, eps=1e-8, decay=0.0, scale=1.0):
    """(p, m, v, size of the step's terms in p) after a step."""
    p, g, m, v = (np.asarray(x, np.float64) for x in (p, g, m, v))
    g = scale * g
    m1 = beta1 * m + (1 - beta1) * g
    v1 = beta2 * v + (1 - beta2) * g * g
    den = np.sqrt(v1 / (1 - beta2 ** step)) + eps
    rate = lr / (1 - beta1 ** step)
    size = rate * (np.abs(beta1 * m) + np.abs((1 - beta1) * g)) / den
    return p - lr * decay * p - rate * m1 / den, m1, v1, size


def blocks(x):
    """x as rows of 256, the last filled with zeros."""
    n = -(-x.size // BLOCK) * BLOCK
    return np.concatenate([x, np.zeros(n - x.size)]).reshape(-1, BLOCK)


def scales(x):
    top = np.abs(blocks(x)).max(1)
    return np.where(top > 0, np.maximum(top / 448, 2.0 ** -126), 0.0)


def spread(s, n):
    """One scale for each of n values."""
    return np.repeat(s, BLOCK)[:n]


def e4m3_step(x):
    """Spacing of the e4m3 values around |x| <= 448."""
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6))) - 3)


def codes(x, s, bits16, never_zero):
    """(values of the codes, distance of the decision from its border in steps) of x / s."""
    y = np.abs(x) / np.where(s > 0, s, 1.0)
    q = e4m3_step(y)
    at = y / q + bits16 / 65536.0
    c = np.minimum(np.floor(at) * q, 448.0)
    if never_zero:
        c = np.where((y > 0) & (c == 0), 2.0 ** -9, c)
    return c * np.sign(x), np.abs(at - np.round(at))


def bf16_random(x, bits16):
    """(x rounded to bf16 by 16 random bits, distance of the decision from its border in steps)."""
    x = np.asarray(x, np.float64)
    q = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -126))) - 7)
    at = np.abs(x) / q + bits16 / 65536.0
    return np.floor(at) * q * np.sign(x), np.abs(at - np.round(at))
