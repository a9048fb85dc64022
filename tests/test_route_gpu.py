"""Routing and its gradient on the GPU against the 64-bit forms: every width of the kernel, odd
expert counts, both scores and types, groups, near and exact ties, masked experts and rows,
NaN and infinities, one token to many.

Tolerances (u = 2^-24, D the largest |z - z_max| of a token, or |z| for sigmoid).  A score takes one
exponential (its argument is off by at most D u, the exponential by 2 ulp = 4 u), a sum of at
most 37 steps (32 per lane, 5 across), a division and two multiplications: its relative error is below
(2 D + 56) u.  A gradient is a product of such factors and a sum of at most 32 slots: below
(4 D + 150) u times the largest |scale dw| (every factor is at most 2 in magnitude: dw - mean), plus
half a step of its type.
"""
import numpy as np
import pytest
import torch

from pruned_expert_backward_lrmoe_b200 import lrmoe as L
from tests import forward_ref as R

pytestmark = pytest.mark.gpu

FN = {"softmax": L.LRMOE_SCORE_SOFTMAX, "sigmoid": L.LRMOE_SCORE_SIGMOID}
TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24


def spread(z, kind):
    """A bound of D; a score more than 110 below its reference is under 2e-48 and falls to atol."""
    z = np.where(np.isfinite(z), z, 0.0)
    return min(110.0, np.abs(z).max() * (2 if kind == "softmax" else 1))


def run(z, k, bias=None, kind="softmax", **how):
    T, E = z.shape
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.lrmoe_route(z, idx, w, bias=bias, score_fn=FN[kind], status=st, **how)
    return idx.cpu().numpy(), w.cpu().numpy(), int(st.item())


def check(z, k, bias=None, kind="softmax", n_group=1, topk_group=1, renorm=True, scale=1.0):
    """z: a CPU tensor of the logits' type."""
    b = None if bias is None else bias.numpy()
    zz = z.double().numpy()
    ri, rw, rs = R.route(zz, k, b, kind, n_group, topk_group, renorm, scale)
    gi, gw, gs = run(z.cuda(), k, None if bias is None else bias.cuda(), kind, n_group=n_group,
                     topk_group=topk_group, renormalise=renorm, scale=scale)
    np.testing.assert_array_equal(gi, ri)
    assert gs == rs
    tol = (2 * spread(zz, kind) + 56) * U
    np.testing.assert_allclose(gw, rw, rtol=tol, atol=1e-37)
    assert (gw[ri < 0] == 0).all()


def logits(T, E, dt, seed, sigma=1.3):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * sigma).to(TYPE[dt])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kind,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("T,E,k", [(1, 128, 8), (1, 1, 1), (5, 2, 2), (33, 31, 3), (7, 32, 32), (130, 33, 1),
                                   (64, 60, 4), (257, 128, 8), (19, 129, 8), (40, 256, 10), (9, 300, 31),
                                   (6, 512, 16), (11, 513, 8), (5, 1000, 32), (3, 1024, 8)])
def test_route(T, E, k, kind, renorm, dt):
    check(logits(T, E, dt, T + E + k), k, kind=kind, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,G,keep,biased", [
    (300, 256, 8, 8, 4, True), (300, 256, 8, 8, 4, False), (100, 128, 8, 1, 1, True), (65, 60, 6, 4, 2, True),
    (65, 160, 6, 32, 7, True), (33, 96, 4, 3, 1, False), (50, 16, 4, 16, 5, True), (50, 16, 3, 16, 3, False),
    (17, 1024, 32, 8, 2, True), (17, 480, 32, 5, 5, True), (64, 8, 2, 2, 1, True), (64, 72, 31, 8, 4, True)])
def test_route_bias_and_groups(T, E, k, G, keep, biased, kind, dt):
    bias = torch.randn(E, generator=torch.Generator().manual_seed(E)) * 0.05 if biased else None
    check(logits(T, E, dt, T + E + k), k, bias, kind, G, keep, True, 1.0)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("G", [1, 4])
def test_route_ties_and_near_ties(kind, biased, G):
    """Logits of a few values (exact ties everywhere), and fp32 neighbours whose scores round to the
    same fp32 value although they differ."""
    g = torch.Generator().manual_seed(3)
    T, E, k = 256, 64, 8
    z = torch.randint(-2, 3, (T, E), generator=g).float() * 0.5
    near = torch.full((T, E), 3.0)
    near += torch.randint(0, 40, (T, E), generator=g) * 2.0 ** -22       # a few ulps of 3.0
    z = torch.cat([z, near, torch.zeros(4, E)])
    bias = None
    if biased:  # zeros (ties stay exact), equal and nearly equal values
        bias = torch.zeros(E)
        bias[1::4] = 0.25
        bias[2::4] = 0.25 * (1 + 2.0 ** -23)
    check(z, k, bias, kind, G, max(1, G // 2), True, 1.0)


def test_route_large_bias_hides_the_scores_from_fp32():
    """With biases of 2^14 a score is below a few fp32 steps of the key."""
    g = torch.Generator().manual_seed(4)
    z, bias = torch.randn(128, 48, generator=g), torch.full((48,), 16384.0)
    check(z, 6, bias, "sigmoid", 1, 1, True, 1.0)
    check(z, 6, bias, "softmax", 4, 2, False, 1.0)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_route_a_coarse_key_below_a_fine_pair(kind):
    """Two experts of small scores, 8e-9 apart and told apart by fp32, above one of a large score and a
    negative bias whose key is within 6e-8 of theirs: only 64 bits say whether it is first."""
    T, E = 500, 6
    z = torch.full((T, E), -20.0, dtype=torch.float64)
    z[:, 0] = 0.0
    z[:, 1] = -7.0
    z[:, 4] = 4e-3
    s = torch.from_numpy(R.scores(z[0].numpy(), kind))
    z[:, 3] = -7.0 - 8e-9 / float(s[1])                                  # ds = s dz
    z[:, 4] += torch.linspace(-1, 1, T, dtype=torch.float64) * 6e-8 * 4  # ds = dz / 4
    for step in range(12):  # across the grid of the large score's fp32 values
        fine = 1e-4 + step * 1e-8
        bias = torch.tensor([-9.0, fine, 0.0, fine, 0.0, 0.0])
        bias[4] = float(s[1]) + 1e-4 - float(s[4])
        check(z.float(), 1, bias, kind)
        check(z.float(), 2, bias, kind)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_route_group_of_large_keys_of_both_signs(kind):
    """A group's value 1000 + s - 999.5 + s' is of the order of 1, its keys round by 3e-5."""
    T, E = 2000, 8
    g = torch.Generator().manual_seed(8)
    z = torch.zeros(T, E, dtype=torch.float64)
    z[:, 2:4] = z[:, 6:] = -float("inf")
    z[:, 0] = 0.01 * torch.randn(T, generator=g)
    bias = torch.tensor([1000.0, -999.5, 0.0, 0.0, 0.25, 0.25, 0.0, 0.0])
    # the two groups' values differ by some 1e-5: all scores but expert 0's and 4's are the same
    z[:, 4] = z[:, 0] + 8e-5 * torch.randn(T, generator=g, dtype=torch.float64)
    check(z.float(), 1, bias, kind, 2, 1)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("equal", [2, 3, 12])
@pytest.mark.parametrize("E", [40, 300])
def test_route_near_tie_behind_equal_experts(E, equal, kind):
    """Equal experts around the last slot, and after them one whose logit is an ulp larger but whose
    fp32 score is the same."""
    z = torch.full((4, E), -1.0)
    z += torch.linspace(0, 0.5, E)
    z[:, 5] = 4.0
    z[:, 6:6 + equal] = 3.0
    z[:, 6 + equal] = 3.0 + 2.0 ** -22
    bias = torch.zeros(E)
    for k in (1, 2, 3):
        check(z, k, bias, kind)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("G", [1, 4])
def test_route_masks(kind, dt, G):
    """-inf (some, all but a few, all), the lowest finite number, NaN and +inf, in logits and bias."""
    T, E, k = 40, 32, 6
    z = logits(T, E, dt, 5)
    hide = torch.rand(T, E, generator=torch.Generator().manual_seed(6)) < 0.5
    z = z.masked_fill(hide, float("-inf"))
    z[3] = float("-inf")
    z[4] = float("-inf")
    z[4, 17] = 1.0
    z[5, :] = torch.finfo(TYPE[dt]).min
    z[6, 1:] = torch.finfo(TYPE[dt]).min
    z[6, 0] = 0.5
    check(z, k, kind=kind, n_group=G, topk_group=max(1, G // 2), renorm=True)
    bias = torch.zeros(E)
    bias[2], bias[9] = float("-inf"), 0.3
    check(z, k, bias, kind, G, max(1, G // 2), True)
    z[7, 3], z[8, 4], z[9, :] = float("nan"), float("inf"), float("nan")
    check(z, k, kind=kind, n_group=G, topk_group=max(1, G // 2), renorm=False)
    bias[3], bias[4] = float("nan"), float("inf")
    check(z, k, bias, kind, G, max(1, G // 2), True)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_route_far_scores_do_not_vanish(kind):
    """All chosen scores below the smallest fp32 number: renormalised weights stay exact."""
    z = torch.linspace(-200, -190, 24).repeat(3, 1)
    if kind == "softmax":
        z[:, 0] = 20.0                       # takes the whole softmax; then hidden by the bias
    bias = torch.zeros(24)
    bias[0] = float("-inf")
    check(z, 4, bias if kind == "softmax" else None, kind, 1, 1, True)


def test_route_many_tokens_and_repeat():
    z = logits(40000, 128, "bf16", 9)
    check(z[:4000], 8, kind="softmax")
    a, b = run(z.cuda(), 8), run(z.cuda(), 8)
    assert (a[0] == b[0]).all() and (a[1].view(np.uint32) == b[1].view(np.uint32)).all()
    want = torch.sort(z.float(), dim=1, descending=True, stable=True).indices[:, :8]
    np.testing.assert_array_equal(a[0], want.numpy())


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,G,keep", [(256, 8, 8, 4), (128, 8, 1, 1), (160, 6, 8, 3), (32, 31, 1, 1), (512, 10, 1, 1),
                                        (40, 32, 1, 1)])
def test_route_selects_by_64_bits_among_many_tokens(E, k, G, keep, kind):
    """20000 tokens of each scale of logits and biases: some come as near as fp32 cannot tell."""
    g = torch.Generator("cuda").manual_seed(E + k)
    for sigma in (0.01, 1.0, 6.0):
        for size in (None, 0.0, 0.02, 1.0, 1e4):
            z = torch.randn(20000, E, generator=g, device="cuda") * sigma
            bias = None if size is None else torch.randn(E, generator=g, device="cuda") * size
            d = z.double()
            key = 1 / (1 + torch.exp(-d)) if kind == "sigmoid" else torch.softmax(d, 1)
            key = key + (0 if bias is None else bias.double())
            value = key.view(-1, G, E // G).topk(min(2, E // G), 2).values.sum(2)
            kept = torch.zeros_like(value, dtype=torch.bool)
            kept.scatter_(1, value.sort(dim=1, descending=True, stable=True).indices[:, :keep], True)
            order = (d if bias is None else key).masked_fill(~kept.repeat_interleave(E // G, 1), -float("inf"))
            want = order.sort(dim=1, descending=True, stable=True).indices[:, :k].int().cpu().numpy()
            got, _, st = run(z, k, bias, kind, n_group=G, topk_group=keep)
            np.testing.assert_array_equal(got, want)
            assert st == 0


def test_route_offsets_past_32_bits():
    """More than 2^31 logits: the last tokens read and write the right rows."""
    T, E, k = 4194310, 513, 2
    z = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    z[-4:, 500], z[-4:, 7] = 9.0, 8.0
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    L.lrmoe_route(z, idx, w, renormalise=False, score_fn=L.LRMOE_SCORE_SIGMOID)
    assert idx[-4:].tolist() == [[500, 7]] * 4 and idx[-5].tolist() == [0, 1]
    assert bool((idx[:-4] == torch.tensor([0, 1], device="cuda")).all())
    dw = torch.zeros(T, k, device="cuda")
    dw[-1] = 1.0
    dz = torch.full_like(z, float("nan"))
    for renorm, fn in ((False, L.LRMOE_SCORE_SIGMOID), (False, L.LRMOE_SCORE_SOFTMAX)):
        L.lrmoe_route_grad(z, idx, dw, dz, renormalise=renorm, score_fn=fn)
        assert not bool(dz[:-1].any()) and bool(dz[-1, 500] != 0) and not bool(dz.isnan().any())


# ---------------------------------------------------------------------------
# gradient
# ---------------------------------------------------------------------------
def check_grad(z, idx, dw, kind, renorm, scale, skip=None):
    dt = "bf16" if z.dtype == torch.bfloat16 else "f32"
    zz = z.double().numpy()
    ref, rs = R.route_grad(zz, idx, dw.numpy(), kind, renorm, scale)
    out = torch.full(z.shape, float("nan"), dtype=z.dtype, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.lrmoe_route_grad(z.cuda(), torch.from_numpy(idx).cuda(), dw.cuda(), out, score_fn=FN[kind],
                       renormalise=renorm, scale=scale, status=st)
    got = out.double().cpu().numpy()
    big = np.nan_to_num(dw.numpy(), nan=0.0)
    tol = (4 * spread(zz, kind) + 150) * U * scale * np.abs(big).max()
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= tol + R.HALF[dt] * np.abs(ref)).all(), np.abs(got - ref).max()
    assert int(st.item()) == rs


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 128, 8), (37, 31, 3), (64, 128, 8), (21, 160, 6), (9, 257, 10),
                                   (5, 1024, 32), (33, 60, 1), (8, 33, 31)])
def test_route_grad(T, E, k, kind, renorm, dt):
    z = logits(T, E, dt, T * E)
    rng = np.random.default_rng(T + k)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    dw = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32))
    if T > 4:
        idx[1, 0] = -1
        dw[1, 0] = float("nan")              # an empty slot's dw is not read
        idx[2] = -1
        idx[3, k - 1] = E + 5                # no such expert
        idx[4, :] = idx[4, 0]                # one expert in every slot
    check_grad(z, idx, dw, kind, renorm, 2.5)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_grad_masked_logits(kind, renorm):
    z = logits(12, 40, "f32", 1)
    rng = np.random.default_rng(2)
    idx = np.stack([rng.permutation(40)[:4] for _ in range(12)]).astype(np.int32)
    dw = torch.from_numpy(rng.standard_normal((12, 4)).astype(np.float32))
    z[0, :] = float("-inf")
    z[1, idx[1, 0]] = float("-inf")
    z[2, idx[2, 1]] = float("nan")
    z[3, idx[3, 2]] = float("inf")
    check_grad(z, idx, dw, kind, renorm, 1.0)


def test_route_grad_takes_the_flat_dw_of_router_grad_and_torch_agrees():
    """The dw of lrmoe_router_grad is flat; autograd of the plain formula gives the same gradient."""
    z = logits(50, 64, "f32", 8).requires_grad_()
    idx, w, _ = run(z.detach().cuda(), 6)
    dw = torch.randn(50 * 6, generator=torch.Generator().manual_seed(1))
    s = torch.softmax(z.double(), 1).gather(1, torch.from_numpy(idx).long())
    ((s / s.sum(1, keepdim=True)) * dw.view(50, 6)).sum().backward()
    out = torch.empty(50, 64, device="cuda")
    L.lrmoe_route_grad(z.detach().cuda(), torch.from_numpy(idx).cuda(), dw.cuda(), out)
    tol = (4 * spread(z.detach().numpy(), "softmax") + 150) * U * dw.abs().max().item()
    assert (out.cpu() - z.grad).abs().max().item() <= tol


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_route_grad_of_one_renormalised_slot_is_zero(kind, dt):
    """Its weight is the constant scale, whatever the logits."""
    z = logits(257, 60, dt, 9).cuda()
    idx = torch.randint(0, 60, (257, 1), device="cuda", dtype=torch.int32)
    dz = torch.full_like(z, float("nan"))
    L.lrmoe_route_grad(z, idx, torch.randn(257, 1, device="cuda"), dz, score_fn=FN[kind], renormalise=True, scale=2.5)
    assert (dz == 0).all()
