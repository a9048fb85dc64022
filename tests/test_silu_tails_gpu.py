"""The activation of lrmoe_grouped_swiglu on its own: gates from 0 to +-180, ups from 1e-20 to 3e38, infinities
and NaN.  Every row of x is (1, 0, ..., 0), so g and u are entries of the weights and exact; what is
left is silu(g) * u and one rounding.

Tolerances.  silu(g) u = (g h r) u h with h = exp(-|g| / 2) and r = 1 / (1 + h^2) for g < 0.  bf16: h is the square
of a power of two that is good to 2 ulp (2^-23 relative) and whose argument, 0.36 |g|, is off by 2^-23 relative (its
constant and its product); h comes in twice, so 8 + 1.0 |g| ulp; two squarings, the reciprocal, the sum and four
products add at most 6: 14 + |g|.  fp32: the exponential is good to 2 ulp, twice, and five operations to half
an ulp: 8 ulp.  Past |g| = 174 h is a subnormal number, off by 2^-149 twice.  The result is rounded once,
to half a step of its type, or half of its smallest number.
"""
import numpy as np
import pytest
import torch

from pruned_expert_backward_lrmoe_b200 import lrmoe as L
from tests import forward_ref as R

pytestmark = pytest.mark.gpu

TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
LEAST = {"bf16": 2.0 ** -133, "f32": 2.0 ** -149}
GATES = [0.0, 1e-30, 1e-3, 0.5, 1.0, 2.0, 5.0, 10.0, 20.0, 40.0, 64.0, 80.0, 86.0, 87.0, 87.5, 88.0, 88.5, 89.0, 90.0, 92.0,
         95.0, 100.0, 104.0, 110.0, 120.0, 140.0, 160.0, 170.0, 174.0, 176.0, 180.0]
UPS = [1.0, -3.0, 1e3, -1e10, 1e30, 3e38, 1e-20]


def run(gates, ups, dt, rows, gather, bias=False):
    """a of `rows` equal rows, as [rows][I], and the gates and ups as the type holds them."""
    n = len(gates)
    W = torch.zeros(1, 2 * n, 8, dtype=torch.float64)
    W[0, :n, 0], W[0, n:, 0] = torch.tensor(gates), torch.tensor(ups)
    b = None
    if bias:  # the same values by the bias
        b, W = W[:, :, 0].to(TYPE[dt]).cuda(), torch.zeros_like(W)
    W = W.to(TYPE[dt]).cuda()
    x = torch.zeros(rows, 8, dtype=TYPE[dt], device="cuda")
    x[:, 0] = 1
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    perm = torch.arange(rows, dtype=torch.int32, device="cuda") if gather else None
    Ap = torch.full((rows, n), 7.0, dtype=TYPE[dt], device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.lrmoe_grouped_swiglu(x, W, off, Ap, perm=perm, bias=b, status=st)
    assert int(st.item()) == 0
    held = (W[0, :, 0] if b is None else b[0]).double().cpu().numpy()
    return Ap.double().cpu().numpy(), held[:n], held[n:]


# rows: a one-SM tile, and tiles on SM pairs
@pytest.mark.parametrize("rows,gather,bias", [(1, False, False), (300, False, True), (1, True, True), (300, True, False)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_activation_over_the_range_of_the_gate(dt, rows, gather, bias):
    pairs = [(s * g, u) for g in GATES for s in (1, -1) for u in UPS]
    pairs += [(1.0, 1.0)] * (-len(pairs) % 8)
    a, g, u = run([p[0] for p in pairs], [p[1] for p in pairs], dt, rows, gather, bias)
    with np.errstate(over="ignore", under="ignore"):
        ref = R.silu(g) * u
        # silu itself in 64 bits; the product with u past the type's range is infinite in both
        inf = np.abs(ref) > 3.39e38
        h = np.exp(-np.abs(g) / 2)
        ulps = 14 + np.abs(g) if dt == "bf16" else np.full_like(g, 8.0)
        rel = ulps * 2.0 ** -23 + 2 * 2.0 ** -149 / h * (np.abs(g) > 174) + R.HALF[dt]
        tol = rel * np.abs(ref) + LEAST[dt] / 2 + 2.0 ** -149
    for row in a:
        bad = ~inf & ~(np.abs(row - ref) <= tol)
        assert not bad.any(), [(g[i], u[i], row[i], ref[i]) for i in np.flatnonzero(bad)[:6]]
        assert np.isinf(row[inf]).all() and (np.sign(row[inf]) == np.sign(ref[inf])).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_activation_of_infinities_and_nan(dt):
    """As the formula g / (1 + exp(-g)) * u gives them.  (g and u are formed in a product with zeros, in which
    an infinite weight alone would become NaN, so they come by the bias.)"""
    inf, nan = float("inf"), float("nan")
    a, _, _ = run([inf, inf, -inf, nan, 1.0, 1.0, -90.0, 0.0], [2.0, -2.0, 2.0, 1.0, nan, -inf, inf, inf], dt, 1, False, True)
    assert a[0, 0] == inf and a[0, 1] == -inf and a[0, 5] == -inf and a[0, 6] == -inf
    assert np.isnan(a[0, [2, 3, 4, 7]]).all()
