"""The router's losses, counts and their gradient against the 64-bit forms.

Tolerances (u = 2^-24): an exponential of d = z - max is within (4 |d| + 4) u of itself (the difference, its
product with log2 e and that constant are rounded, ex2.approx is good to 2^-22), a sum of it and at most
1024 others adds 37 additions, the quotient 4 more: a share is within K = 8 d + 100 of itself, twice that
where sigmoids and 1 - sigmoid are multiplied.  Sums over tokens: a run's tokens go to 8 warps and those to
at most 592 runs, each a chain of additions: depth = run + 8 + 592 / 4 + 64 (16 warps and 296 runs take fewer).  lse is within (K + 4 |zmax|) u.
"""
import numpy as np
import pytest
import torch

from pruned_expert_backward_lrmoe_b200 import lrmoe as L
from tests import forward_ref as R
from tests import step_ref as S

pytestmark = pytest.mark.gpu

TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
FN = {"softmax": L.LRMOE_SCORE_SOFTMAX, "sigmoid": L.LRMOE_SCORE_SIGMOID}
U = 2.0 ** -24
TINY = 2.0 ** -120  # what ex2 flushes


class Case:
    def __init__(self, T, E, k, dt, off=None, seed=0, scale=1.3, masks=True):
        rng = np.random.default_rng(seed + T + E)
        self.T, self.E, self.k, self.dt = T, E, k, dt
        z = torch.from_numpy(rng.standard_normal((T, E)) * scale).to(TYPE[dt])
        idx = rng.integers(0, E, (T, k)).astype(np.int32)
        if masks and T > 8:
            idx[rng.random((T, k)) < 0.1] = -1
            idx[T - T // 8:] = -1                   # padded tokens
            z[T - 1] = float("nan")                 # whose logits may be anything that is flagged
            z[rng.random((T, E)) < 0.1] = -float("inf")
            z[3] = -float("inf")                    # nothing left, and still routed
            idx[3, 0] = 0
            z[4] = torch.finfo(TYPE[dt]).min        # not masked, but the lowest number
        self.z, self.idx = z.cuda(), torch.from_numpy(idx).cuda()
        self.zd, self.idxn = z.double().numpy(), idx
        self.off = off
        self.offt = None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
        self.B = 1 if off is None else len(off) - 1
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def outputs(self, fill=77):
        i = dict(dtype=torch.int32, device="cuda")
        return dict(counts=torch.full((self.B, self.E), fill, **i), stats=torch.full((self.B + 1, 2), fill, **i),
                    mean_score=torch.full((self.B, self.E), float(fill), device="cuda"),
                    loss=torch.full((2,), float(fill), device="cuda"),
                    workspace=torch.full((L.lrmoe_balance_workspace_bytes(self.T, self.E, self.B),), 0xEE, dtype=torch.uint8,
                                         device="cuda"))

    def forward(self, out, kind="softmax", coef=1.0, z_coef=0.0, **kw):
        L.lrmoe_balance(self.z, self.idx, seq_offsets=self.offt, score_fn=FN[kind], coef=coef, z_coef=z_coef,
                        status=self.status, **out, **kw)
        return out

    def share_error(self):
        z = np.where(np.isfinite(self.zd), self.zd, 0)
        z = np.where(np.abs(z) > 1e30, 0, z)
        d = z.max(initial=0) - z.min(initial=0)
        return (2 * (8 * d + 100)) * U, d

    def check_forward(self, out, kind, coef, z_coef):
        ref = S.balance(self.zd, self.idxn, self.off, kind, coef, z_coef)
        assert out["counts"].cpu().numpy().tolist() == ref["counts"].tolist()
        assert out["stats"].cpu().numpy().tolist() == ref["stats"].tolist()
        e, d = self.share_error()
        depth = max(64, -(-self.T // 592)) + 8 + 148 + 64 + self.B
        e += depth * U
        mean = out["mean_score"].double().cpu().numpy()
        assert (np.abs(mean - ref["mean"]) <= e * ref["mean"] + TINY).all()
        loss = out["loss"].double().cpu().numpy()
        assert abs(loss[0] - ref["loss"][0]) <= 2 * e * abs(ref["loss"][0])
        fine = self.zd[(self.idxn >= 0).any(1)]
        top = np.abs(np.where(np.isfinite(fine), fine, 0)).max(initial=0)
        # of lse, then of its square
        le = e + (4 * top + 4 * d) * U
        if ref["loss"][1] > torch.finfo(torch.float32).max:
            # a row of the lowest logits: lse^2 is 1e76, the nearest fp32 to its share of the mean is infinite
            assert loss[1] == np.inf
        elif z_coef:
            assert abs(loss[1] - ref["loss"][1]) <= z_coef * (2 * le * np.sqrt(ref["loss"][1] / z_coef) + le * le) \
                + depth * U * ref["loss"][1]
        else:
            assert loss[1] == 0
        return ref

    def grad(self, out, kind="softmax", coef=1.0, z_coef=0.0, dloss=None, add=None, dz=None):
        dz = torch.full((self.T, self.E), 77.0, dtype=TYPE[self.dt], device="cuda") if dz is None else dz
        L.lrmoe_balance_grad(self.z, self.idx, out["counts"], out["stats"], dz, seq_offsets=self.offt,
                             score_fn=FN[kind], coef=coef, z_coef=z_coef, dloss=dloss, add=add, status=self.status)
        return dz

    def check_grad(self, dz, kind, coef, z_coef, dloss=(1.0, 1.0), add=None):
        a = None if add is None else add.double().cpu().numpy()
        ref, mag = S.balance_grad(self.zd, self.idxn, self.off, kind, coef, z_coef, dloss, a)
        e, d = self.share_error()
        top = np.abs(np.where(np.isfinite(self.zd), self.zd, 0))
        top = np.where(top > 1e30, 0, top).max(initial=0)
        tol = 3 * (e + 8 * top * U) * mag + R.HALF[self.dt] * np.abs(ref) + TINY
        got = dz.double().cpu().numpy()
        assert (np.abs(got - ref) <= tol).all(), np.abs(got - ref).max()


SIZES = [(1, 1, 1), (1, 16, 2), (7, 8, 2), (257, 16, 2), (100, 33, 4), (513, 60, 6), (300, 64, 8), (130, 100, 3), (1000, 128, 8),
         (77, 250, 6), (64, 256, 32), (90, 300, 7), (33, 512, 9), (41, 1000, 5), (20, 1024, 8), (5000, 8, 1)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_balance_and_its_gradient(T, E, k, kind, dt):
    c = Case(T, E, k, dt)
    out = c.forward(c.outputs(), kind, 0.7, 0.3)
    ref = c.check_forward(out, kind, 0.7, 0.3)
    flagged = int(c.status.item())
    assert flagged == ref["status"] == (R.NONFINITE if T > 8 else 0)
    c.check_grad(c.grad(out, kind, 0.7, 0.3), kind, 0.7, 0.3)
    up = torch.tensor([1.5, -0.25], device="cuda")
    add = (torch.randn(T, E, device="cuda") * 1e-3).to(TYPE[dt])
    dz = c.grad(out, kind, 0.7, 0.3, up, add)
    c.check_grad(dz, kind, 0.7, 0.3, (1.5, -0.25), add)
    same = add.clone()
    c.grad(out, kind, 0.7, 0.3, up, same, same)               # in place
    assert torch.equal(same, dz)
    # tokens that do not count get what was there, or zeros
    none = torch.from_numpy(~((c.idxn >= 0).any(1))).cuda()
    assert torch.equal(dz[none], add[none]) and not c.grad(out, kind, 0.7, 0.0)[none].any()
    again = c.forward(c.outputs(5), kind, 0.7, 0.3)
    assert all(torch.equal(out[n], again[n]) for n in ("counts", "stats", "mean_score", "loss"))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_z_loss(T, E, k, kind, dt):
    """Without masked or lowest logits, whose squares would outweigh all others."""
    c = Case(T, E, k, dt, seed=8, scale=3.0, masks=False)
    out = c.forward(c.outputs(), kind, 0.5, 0.2)
    c.check_forward(out, kind, 0.5, 0.2)
    assert np.isfinite(out["loss"].cpu().numpy()).all() and int(c.status.item()) == 0
    c.check_grad(c.grad(out, kind, 0.5, 0.2), kind, 0.5, 0.2)


OFFSETS = {"covering": lambda T: [0, 1, T // 3, T // 3, T - 2, T], "inside": lambda T: [5, 6, 6, T // 2, T - 9],
           "empty": lambda T: [3, 3, 3], "one": lambda T: [2, T - 1], "all at the end": lambda T: [T, T],
           "each token": lambda T: list(range(T + 1))}


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("which", list(OFFSETS))
@pytest.mark.parametrize("T,E,k", [(200, 16, 2), (2001, 128, 4), (333, 70, 3)])
def test_sequences(T, E, k, which, kind, dt):
    c = Case(T, E, k, dt, off=OFFSETS[which](T), seed=3)
    lo, hi = c.off[0], c.off[-1]
    out = c.forward(c.outputs(), kind, 2.0, 0.1)
    ref = c.check_forward(out, kind, 2.0, 0.1)
    dz = c.grad(out, kind, 2.0, 0.1)
    c.check_grad(dz, kind, 2.0, 0.1)
    assert int(c.status.item()) == ref["status"]           # what lies behind the sequences is not read
    assert not dz[:lo].any() and not dz[hi:].any()


@pytest.mark.parametrize("T,E,k", [(1024, 16, 2), (1025, 16, 2), (256, 128, 8), (257, 128, 8), (128, 256, 4), (129, 256, 4),
                                   (70, 600, 3), (18944, 32, 2), (18945, 128, 2)])
def test_one_sequence_given_by_its_bounds(T, E, k):
    """The same tokens as one sequence without and with bounds: a single launch or two, runs added by one block or more."""
    c = Case(T, E, k, "f32", seed=6, masks=False)
    a = c.forward(c.outputs(), "softmax", 1.5, 0.2)
    c.check_forward(a, "softmax", 1.5, 0.2)
    c.offt = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    b = c.forward(c.outputs(), "softmax", 1.5, 0.2)
    c.check_forward(b, "softmax", 1.5, 0.2)
    assert torch.equal(a["counts"], b["counts"]) and torch.equal(a["stats"], b["stats"])
    for n in ("mean_score", "loss"):  # at most the order of the runs' sums differs
        assert ((a[n] - b[n]).abs() <= 300 * U * a[n].abs()).all()


@pytest.mark.parametrize("kind,dt", [("softmax", "f32"), ("sigmoid", "bf16")])
def test_long_runs(kind, dt):
    """Runs and warps with more tokens than they look at at a time, cut by sequences."""
    T = 200001
    c = Case(T, 8, 2, dt, off=[3, 70000, 70001, 130001, T - 5], seed=9, masks=False)
    c.idxn[::7] = -1
    c.idx.copy_(torch.from_numpy(c.idxn))
    out = c.forward(c.outputs(), kind, 1.0, 0.5)
    c.check_forward(out, kind, 1.0, 0.5)
    c.check_grad(c.grad(out, kind, 1.0, 0.5), kind, 1.0, 0.5)


def test_many_short_sequences():
    """More sequences than a block sums at a time, some of them empty."""
    rng = np.random.default_rng(5)
    T = 3000
    off = np.sort(np.concatenate([[0, T], rng.integers(0, T + 1, 1500)])).tolist()
    c = Case(T, 24, 2, "f32", off=off)
    out = c.forward(c.outputs(), "softmax", 1.0, 0.5)
    c.check_forward(out, "softmax", 1.0, 0.5)
    c.check_grad(c.grad(out, "softmax", 1.0, 0.5), "softmax", 1.0, 0.5)


def test_bad_ids_and_bad_offsets_are_flagged():
    c = Case(50, 16, 2, "f32", masks=False)
    c.idxn[7] = [16, 3]
    c.idxn[8] = [99, 2 ** 31 - 1]
    c.idx.copy_(torch.from_numpy(c.idxn))
    out = c.forward(c.outputs(), "softmax", 1.0, 0.5)
    c.check_forward(out, "softmax", 1.0, 0.5)
    assert int(c.status.item()) == R.BAD_EXPERT
    c.check_grad(c.grad(out, "softmax", 1.0, 0.5), "softmax", 1.0, 0.5)
    for off in ([0, 30, 20], [-5, 10, 50], [0, 10, 51], [60, 70, 80]):
        d = Case(50, 16, 2, "f32", off=off, masks=False)
        d.grad(d.forward(d.outputs()))
        assert int(d.status.item()) == R.BAD_INDEX, off


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("shift", [-300.0, -90.0, 90.0, 300.0, 1e4])
def test_logits_far_from_zero(kind, shift):
    """Sigmoids that vanish or saturate together keep their proportions."""
    c = Case(60, 40, 4, "f32", masks=False)
    c.z += shift
    c.zd = c.z.double().cpu().numpy()
    out = c.forward(c.outputs(), kind, 1.0, 1e-4)
    c.check_forward(out, kind, 1.0, 1e-4)
    c.check_grad(c.grad(out, kind, 1.0, 1e-4), kind, 1.0, 1e-4)
    assert int(c.status.item()) == 0


def test_a_share_of_one():
    """A single expert left to each token: its share is 1 and nothing moves it."""
    c = Case(40, 12, 1, "f32", masks=False)
    c.z.fill_(-float("inf"))
    c.z.scatter_(1, c.idx.long(), 2.0)
    c.zd = c.z.double().cpu().numpy()
    out = c.forward(c.outputs(), "softmax", 1.0, 0.0)
    c.check_forward(out, "softmax", 1.0, 0.0)
    assert not c.grad(out, "softmax", 1.0, 0.0).any()


def test_offsets_past_32_bits():
    """Logits of more than 2^31 elements: the last tokens are read and written in their places."""
    T, E, k = (1 << 23) + 40, 256, 1
    z = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    z[T - 3:, 7] = 3.0
    idx = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    idx[T - 3:] = 7
    idx[0] = 1
    c = Case(1, E, k, "bf16", masks=False)
    c.T, c.z, c.idx = T, z, idx
    out = c.forward(c.outputs(), "softmax", 1.0, 1.0)
    e3 = np.exp(3.0)
    p = e3 / (e3 + 255)
    assert out["stats"].tolist() == [[4, 4], [4, 1]]
    assert out["counts"][0, 7].item() == 3 and out["counts"][0, 1].item() == 1
    np.testing.assert_allclose(out["mean_score"][0, 7].item(), (3 * p + 1 / 256) / 4, rtol=2e-5)
    np.testing.assert_allclose(out["loss"][1].item(), (3 * np.log(e3 + 255) ** 2 + np.log(256.0) ** 2) / 4, rtol=2e-5)
    dz = torch.full((T, E), 7.0, dtype=torch.bfloat16, device="cuda")
    c.grad(out, "softmax", 1.0, 0.0, dz=dz)
    D = 256 * np.array([3.0, 1.0]) / 16
    dot = p * D[0] + D[1] / (e3 + 255)
    np.testing.assert_allclose(dz[T - 3:, 7].float().cpu().numpy(), p * (D[0] - dot), rtol=2 ** -8 + 1e-4)
    assert not dz[1:T - 3].any()
