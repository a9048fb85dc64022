"""Bias gradients of experts of very unequal size against 64 bits."""
import numpy as np
import pytest
import torch

from pruned_expert_backward_lrmoe_b200 import lrmoe as L

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E,N,hot", [(128, 1536, 40000), (160, 520, 9000)])
def test_bias_grad_of_one_long_expert_among_many(E, N, hot, dt):
    """One expert holds nearly all rows.  A thread adds every 32nd of a run of them, then 2 + 8 + 8 partial sums
    meet: below m / 32 + 24 additions, each off by 2^-24 of the sum of magnitudes at most."""
    rng = np.random.default_rng(E)
    sizes = rng.integers(0, 40, E)
    sizes[E // 3] = hot
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    M = int(off[-1])
    g = torch.Generator("cuda").manual_seed(N)
    rows = (torch.randn(M + 3, N, generator=g, device="cuda") + 0.5).to(dt)
    rows[M:] = float("nan")
    db = torch.full((E, N), float("nan"), device="cuda")
    L.lrmoe_grouped_bias_grad(rows, torch.from_numpy(off).cuda(), db)
    got = db.double()
    for e in range(E):
        r = rows[off[e]:off[e + 1]].double()
        m = int(sizes[e])
        assert bool(((got[e] - r.sum(0)).abs() <= (m / 32 + 24) * 2.0 ** -24 * r.abs().sum(0)).all()), e
