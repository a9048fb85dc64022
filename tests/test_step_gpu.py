"""A whole training step of a layer as it is used: forward, the router's losses, backward, their gradient on top of
the router's, the norm over all gradients and the AdamW step; captured, replayed on several streams, between guard
pages."""
import numpy as np
import pytest
import torch

from pruned_expert_backward_lrmoe_b200 import lrmoe as L
from tests import step_ref as S
from tests.test_canary_gpu import Guard
from tests.test_forward_gpu import Layer, TOL
from tests.test_forward_graphs_gpu import differences, poison

pytestmark = pytest.mark.gpu

COEF, ZCOEF = 0.02, 0.001


class Trainer:
    """A layer with a router weight, its losses and its optimiser."""

    def __init__(self, T, E, k, H, I, dt, bits=32, master=False, seed=0, new=None):
        self.la = la = Layer(T, E, k, H, I, dt, seed=seed, new=new)
        new = new or (lambda shape, dtype: torch.empty(shape, dtype=dtype, device="cuda"))
        i32, f32 = torch.int32, torch.float32
        self.bal = dict(counts=new((1, E), i32), stats=new((2, 2), i32), mean_score=new((1, E), f32), loss=new((2,), f32),
                        workspace=new((L.lrmoe_balance_workspace_bytes(T, E, 1),), torch.uint8))
        self.params = [la.W_gu, la.W_down, la.b_gu, la.b_down]
        self.grads = [la.out["dW_gu"], la.out["dW_down"], la.db_gu, la.db_down]
        self.states = L.alloc_adamw(self.params, bits, master)
        self.list = L.TensorList(self.grads, self.params, weight_decay=[0.1, 0.1, 0.0, 0.0], **self.states)
        self.norm = new((2,), f32)
        self.nws = new((L.lrmoe_grad_norm_workspace_bytes(4),), torch.uint8)
        self.t = torch.ones(1, dtype=i32, device="cuda")
        self.lr = torch.full((1,), 1e-2, device="cuda")

    def step(self, max_norm=1.0):
        la, st = self.la, self.la.out["status"]
        la.forward()
        L.lrmoe_balance(la.logits, la.idx, coef=COEF, z_coef=ZCOEF, status=st, **self.bal)
        la.backward()
        L.lrmoe_balance_grad(la.logits, la.idx, self.bal["counts"], self.bal["stats"], la.dz, coef=COEF, z_coef=ZCOEF,
                             add=la.dz, status=st)
        L.lrmoe_grad_norm(self.list, self.norm, self.nws, max_norm=max_norm, status=st)
        L.lrmoe_adamw(self.list, lr=self.lr, step=self.t, grad_scale=self.norm[1:], seed=7, status=st)

    def results(self):
        return [self.la.Y, self.la.out["dX"], self.la.dz, self.norm] + [self.bal[n] for n in ("counts", "stats", "mean_score", "loss")]

    def kept(self):
        return self.params + [t for ts in self.states.values() for t in ts]


def copy_all(to, source):
    for a, b in zip(to, source):
        a.view(torch.uint8).copy_(b.view(torch.uint8)) if a.element_size() == 1 else a.copy_(b)


def clones(ts):
    return [t.view(torch.uint8).clone().view(t.dtype) if t.element_size() == 1 else t.clone() for t in ts]


@pytest.mark.parametrize("dt,bits,master,T,E,k,H,I", [("f32", 32, False, 130, 8, 2, 64, 36), ("bf16", 32, True, 517, 5, 3, 264, 136),
                                                      ("bf16", 8, False, 301, 8, 2, 136, 264), ("bf16", 8, True, 67, 33, 4, 104, 40)])
def test_training_step(dt, bits, master, T, E, k, H, I):
    tr = Trainer(T, E, k, H, I, dt, bits, master)
    la = tr.la
    la.out["status"].zero_()
    ref = None
    p0 = [p.double() for p in (tr.states["master"] if master else tr.params)]
    la.forward()
    ref = la.reference()
    tr.step(max_norm=0.5)
    assert int(la.out["status"].item()) == 0
    # the losses and their gradient on top of the router's, by autograd in 64 bits
    z = torch.where(torch.isfinite(la.logits), la.logits, 0).double().requires_grad_()
    on = (la.idx >= 0).any(1)
    p = torch.softmax(z, 1)
    c = torch.bincount(la.idx[la.idx >= 0].long(), minlength=E).double()
    balance = COEF * E * (c / c.sum() * p[on].mean(0)).sum()
    zl = ZCOEF * torch.logsumexp(z, 1)[on].square().mean()
    got = tr.bal["loss"].double()
    assert abs(got[0] - balance) <= 1e-5 * balance and abs(got[1] - zl) <= 1e-5 * zl
    assert tr.bal["counts"][0].long().tolist() == c.long().tolist()
    (balance + zl).backward()
    want = ref["dz"] + z.grad
    assert (la.dz.double() - want).norm() <= 4 * TOL[dt] * want.norm()
    # the norm and the step, from the gradients that were computed
    norm = torch.sqrt(sum(g.double().square().sum() for g in tr.grads))
    factor = min(1.0, 0.5 / norm.item())
    assert abs(tr.norm[0].item() - norm.item()) <= 2e-6 * norm.item() and abs(tr.norm[1].item() - factor) <= 2e-6
    now = tr.states["master"] if master else tr.params
    for a, b, g, wd in zip(p0, now, tr.grads, (0.1, 0.1, 0.0, 0.0)):
        x, _, _, size = S.adamw(a.cpu().numpy(), g.double().cpu().numpy(), 0, 0, 1e-2, 1, 0.9, 0.999, 1e-8, wd, factor)
        tol = 20 * 2.0 ** -24 * (np.abs(x) + size) + (0 if b.dtype == torch.float32 else 2.0 ** -7) * np.abs(x)
        # where the scaled gradient is next to eps the quotient's error is that of its square's place in 32 bits
        tol += 1e-2 * (np.abs(factor * g.double().cpu().numpy()) < 1e-18)
        assert (np.abs(b.double().cpu().numpy() - x) <= tol).all()


@pytest.mark.parametrize("bits,master", [(32, True), (8, False)])
def test_captured_steps_on_streams_at_once(bits, master):
    """Two captured steps replayed on two streams beside an eager one on a third, from changing states and with the step's
    number and rate changing on the device: each replay writes what an eager step does.  (The backward's grouped products
    keep state between launches, so they stay outside.)"""
    trs = [Trainer(301, 8, 2, 136, 264, "bf16", bits, master, seed=s) for s in (1, 2, 3)]

    def part(tr):
        la, st = tr.la, tr.la.out["status"]
        L.lrmoe_balance(la.logits, la.idx, coef=COEF, z_coef=ZCOEF, status=st, **tr.bal)
        L.lrmoe_balance_grad(la.logits, la.idx, tr.bal["counts"], tr.bal["stats"], la.dz, coef=COEF, z_coef=ZCOEF, status=st)
        L.lrmoe_grad_norm(tr.list, tr.norm, tr.nws, max_norm=0.5, status=st)
        L.lrmoe_adamw(tr.list, lr=tr.lr, step=tr.t, grad_scale=tr.norm[1:], seed=7, status=st)

    results = lambda tr: [tr.la.dz, tr.norm] + [tr.bal[n] for n in ("counts", "stats", "mean_score", "loss")]  # noqa: E731
    starts, wants = [], []
    for tr in trs:
        tr.la.out["status"].zero_()
        tr.step()
        starts.append(clones(tr.kept()))
        wants.append([])
        for r in (0, 1):
            copy_all(tr.kept(), starts[-1])
            tr.t.fill_(2 + r)
            tr.lr.fill_(0.01 * (1 + r))
            poison(results(tr))
            part(tr)
            wants[-1].append(clones(results(tr) + tr.kept()))
        assert any(not torch.equal(a, b) for a, b in zip(*[[t for t in w if t.element_size() > 1] for w in wants[-1]]))
    graphs = []
    for tr in trs[:2]:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            part(tr)
        graphs.append(gr)
    streams = [torch.cuda.Stream() for _ in trs]
    wrong = [torch.zeros((), dtype=torch.int64, device="cuda") for _ in trs]
    torch.cuda.synchronize()
    for r in range(20):
        for i, (tr, st) in enumerate(zip(trs, streams)):
            with torch.cuda.stream(st):
                copy_all(tr.kept(), starts[i])
                tr.t.fill_(2 + (r & 1))
                tr.lr.fill_(0.01 * (1 + (r & 1)))
                poison(results(tr))
                graphs[i].replay() if i < 2 else part(tr)
                wrong[i] += differences(results(tr) + tr.kept(), wants[i][r & 1])
    torch.cuda.synchronize()
    assert [int(w.item()) for w in wrong] == [0, 0, 0]
    assert all(int(tr.la.out["status"].item()) == 0 for tr in trs)


def test_guard_pages_of_a_step():
    G = Guard()
    tr = Trainer(97, 6, 2, 72, 40, "bf16", 8, False, new=G.empty)
    tr.la.out["status"].zero_()
    tr.step()
    assert int(tr.la.out["status"].item()) == 0
    G.check()


def test_a_step_skipped_for_its_norm():
    """An infinity in one gradient: the factor is 0 and weights and states stay."""
    tr = Trainer(67, 8, 2, 64, 128, "bf16", 8, False)
    tr.la.out["status"].zero_()
    tr.step()
    before = clones(tr.kept())
    tr.la.db_gu[0, 0] = float("inf")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.lrmoe_grad_norm(tr.list, tr.norm, tr.nws, max_norm=1.0, status=st)
    L.lrmoe_adamw(tr.list, lr=tr.lr, step=2, grad_scale=tr.norm[1:], status=st)
    assert int(st.item()) == L.ST_NONFINITE and int(differences(tr.kept(), before).item()) == 0


def test_another_device_than_the_current_one_is_refused():
    if torch.cuda.device_count() < 2:
        with pytest.raises(ValueError, match="CUDA"):
            L.lrmoe_grad_norm(L.TensorList([torch.zeros(4)]), torch.zeros(2), torch.zeros(1 << 20, dtype=torch.uint8))
        return
    t = [torch.zeros(8, device="cuda:1") for _ in range(4)]
    with pytest.raises(ValueError, match="cuda:1"):
        L.lrmoe_adamw(L.TensorList([t[0]], [t[1]], [t[2]], [t[3]]), lr=0.1, step=1)
