"""The weighted return to the token layout and the bias gradient against the 64-bit forms.

Tolerances (u = 2^-24): a combine is at most k fused multiply-adds and one addition, so its error is
below (k + 2) u times the sum of magnitudes, plus half a step of the output's type; a bias
gradient over m rows is at most m additions: (m + 2) u times the sum of magnitudes.
"""
import numpy as np
import pytest
import torch

from pruned_expert_backward_lrmoe_b200 import lrmoe as L
from tests import forward_ref as R

pytestmark = pytest.mark.gpu

TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24


def normal(shape, dt, seed, scale=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(TYPE[dt])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("residual", ["none", "given", "in place"])
@pytest.mark.parametrize("T,k,H", [(1, 1, 8), (1, 8, 2048), (13, 8, 1032), (300, 2, 64), (17, 32, 264), (5, 9, 4104),
                                   (65, 6, 248)])
def test_combine(T, k, H, residual, dt):
    E = 40
    rng = np.random.default_rng(T + k)
    idx = rng.integers(0, E, (T, k)).astype(np.int32)
    idx[rng.random((T, k)) < 0.2] = -1
    if T > 3:
        idx[1] = -1                           # nothing routed
        idx[2, 0] = E                         # no such expert
    w = rng.standard_normal((T, k)).astype(np.float32)
    y = normal((T * k, H), dt, 1)
    y[torch.from_numpy((idx < 0).reshape(-1))] = float("nan")   # rows of empty slots are not read
    res = None if residual == "none" else normal((T, H), dt, 2)
    ref, mag = R.combine(y.double().numpy(), idx, w, E, None if res is None else res.double().numpy())
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    Y = torch.full((T, H), float("nan"), dtype=TYPE[dt], device="cuda")
    r = None
    if residual == "given":
        r = res.cuda()
    elif residual == "in place":
        Y.copy_(res)
        r = Y
    L.lrmoe_combine(y.cuda(), torch.from_numpy(idx).cuda(), torch.from_numpy(w).cuda(), E, Y, residual=r, status=st)
    got = Y.double().cpu().numpy()
    assert (np.abs(got - ref) <= (k + 2) * U * mag + R.HALF[dt] * np.abs(ref)).all()
    assert int(st.item()) == (R.BAD_EXPERT if T > 3 else 0)
    if residual == "none" and T > 3:
        assert (got[1] == 0).all()


def test_combine_offsets_past_32_bits():
    """y has more than 2^31 elements: the last tokens read the right rows."""
    T, k, H = 131073, 8, 2056
    y = torch.zeros(T * k, H, dtype=torch.bfloat16, device="cuda")
    idx = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    w = torch.ones(T, k, device="cuda")
    y[-8:] = torch.arange(1, 9, device="cuda")[:, None].to(torch.bfloat16)
    Y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    L.lrmoe_combine(y, idx, w, 4, Y)
    assert bool((Y[-1] == 36).all()) and not bool(Y[:-1].any())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("N", [8, 64, 136, 1032])
@pytest.mark.parametrize("sizes,first", [([1], 0), ([0, 5, 0, 33, 1, 300], 0), ([31, 32, 64, 7], 3), ([2500], 0),
                                         ([0, 0], 0)])
def test_bias_grad(sizes, first, N, accumulate, dt):
    E, M = len(sizes), first + sum(sizes)
    rows = normal((M + 9, N), dt, M + N)
    rows[:first] = float("nan")               # rows of no expert are not read
    rows[M:] = float("nan")
    off = np.concatenate([[first], first + np.cumsum(sizes)]).astype(np.int32)
    ref, mag = R.bias_grad(rows.double().numpy(), off, E)
    db = torch.full((E, N), 3.0 if accumulate else float("nan"), device="cuda")
    if accumulate:
        ref, mag = ref + 3.0, mag + 3.0
    L.lrmoe_grouped_bias_grad(rows.cuda(), torch.from_numpy(off).cuda(), db, accumulate=accumulate)
    got = db.double().cpu().numpy()
    m = np.array(sizes)[:, None]
    assert (np.abs(got - ref) <= (m + 2) * U * mag).all()
    again = torch.full((E, N), 3.0 if accumulate else float("nan"), device="cuda")
    L.lrmoe_grouped_bias_grad(rows.cuda(), torch.from_numpy(off).cuda(), again, accumulate=accumulate)
    assert torch.equal(db, again)
