"""The layer's forward and backward as they are used together: routing, the experts' products, the
combine, the pruned backward over every pair, the bias and router gradients, against autograd of
the same formulas in 64 bits; in a captured graph, on another stream, between guard pages, and
with the checked-index build.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from pruned_expert_backward_lrmoe_b200 import lrmoe as L
from tests.test_canary_gpu import Guard

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
# As the backward's parity tests: the Frobenius error of a tensor against 64 bits, 1e-5 for 32-bit
# storage and 2e-2 for 16-bit storage (a dozen roundings of at most 2^-8 each).  The logits'
# gradient is a difference of routing-weight gradients, which are several times larger: 4 times.
TOL = {"bf16": 2e-2, "f32": 1e-5}


class Layer:
    """Inputs and buffers of one layer."""

    def __init__(self, T, E, k, H, I, dt, seed=0, new=None):
        self.T, self.E, self.k, self.H, self.I, self.dt = T, E, k, H, I, dt
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s, scale=1.0: (torch.randn(*s, generator=g, device="cuda") * scale)  # noqa: E731
        st = TYPE[dt]
        new = new or (lambda shape, dtype: torch.empty(shape, dtype=dtype, device="cuda"))
        P = T * k
        self.P = P
        put = lambda t: new(t.shape, t.dtype).copy_(t)  # noqa: E731
        self.logits = put(rand(T, E))
        self.logits[T - 2:] = float("-inf")                 # padded tokens
        self.x, self.dY, self.res = (put(rand(T, H).to(st)) for _ in range(3))
        self.W_gu = put(rand(E, 2 * I, H, scale=H ** -0.5).to(st))
        self.W_down = put(rand(E, H, I, scale=I ** -0.5).to(st))
        self.b_gu, self.b_down = put(rand(E, 2 * I, scale=0.1).to(st)), put(rand(E, H, scale=0.1).to(st))
        i32, f32 = torch.int32, torch.float32
        self.idx, self.w = new((T, k), i32), new((T, k), f32)
        self.quota, self.counts = new((E,), i32), new((E,), i32)
        self.out = {n: new(t.shape, t.dtype) for n, t in L.alloc_buffers(T, k, E, H, I, st).items()}
        self.g, self.u, self.a, self.Ap = (new((P, I), st) for _ in range(4))
        self.y, self.Y = new((P, H), st), new((T, H), st)
        self.db_gu, self.db_down = new((E, 2 * I), f32), new((E, H), f32)
        self.dw, self.dz = new((P,), f32), new((T, E), f32)
        for t in (self.g, self.u, self.a, self.y):          # pairs of padded tokens stay as they are
            t.zero_()

    def forward(self, **kw):
        o = self.out
        st = o["status"]
        L.lrmoe_route(self.logits, self.idx, self.w, status=st, **kw)
        L.lrmoe_quota_controller(self.idx, self.E, 0, -1, self.quota, self.counts, st)
        L.lrmoe_select_quota(self.idx, self.w, self.quota, o["counts"], o["kept"], o["offsets"], o["perm"],
                             o["pos"], o["workspace"], st)
        L.lrmoe_grouped_swiglu(self.x, self.W_gu, o["offsets"], self.Ap, perm=o["perm"], src_div=self.k,
                               bias=self.b_gu, g=self.g, u=self.u, a=self.a, status=st)
        L.lrmoe_grouped_linear(self.Ap, self.W_down, o["offsets"], self.y, bias=self.b_down, perm=o["perm"],
                               status=st)
        L.lrmoe_combine(self.y, self.idx, self.w, self.E, self.Y, residual=self.res, status=st)

    def backward(self):
        o = self.out
        inp = dict(topk_idx=self.idx, topk_w=self.w, quota=self.quota, x=self.x, dY=self.dY, g=self.g, u=self.u,
                   a=self.a, W_gu=self.W_gu, W_down=self.W_down)
        L.lrmoe_pruned_backward(inp, o)
        L.lrmoe_grouped_bias_grad(o["dGUp"], o["offsets"], self.db_gu, status=o["status"])
        L.lrmoe_grouped_bias_grad(o["DYp"], o["offsets"], self.db_down, status=o["status"])
        L.lrmoe_router_grad(self.idx, self.dY, self.y, self.E, self.dw, status=o["status"])
        L.lrmoe_route_grad(self.logits, self.idx, self.dw, self.dz, status=o["status"])

    def results(self):
        r = dict(Y=self.Y, dX=self.out["dX"], dW_gu=self.out["dW_gu"], dW_down=self.out["dW_down"],
                 db_gu=self.db_gu, db_down=self.db_down, dz=self.dz, idx=self.idx, w=self.w)
        return {n: t.clone() for n, t in r.items()}

    def reference(self):
        """The same by autograd in 64 bits, for the experts in idx."""
        d = lambda t: t.double().detach().requires_grad_()  # noqa: E731
        z = torch.where(torch.isfinite(self.logits), self.logits, 0).double().requires_grad_()
        x, Wg, Wd, bg, bd = d(self.x), d(self.W_gu), d(self.W_down), d(self.b_gu), d(self.b_down)
        idx = self.idx.long()
        on = idx >= 0
        s = torch.softmax(z, 1).gather(1, idx.clamp_min(0))
        w = torch.where(on, s / s.sum(1, keepdim=True), 0.0)
        Y = self.res.double()
        for e in range(self.E):
            t, j = torch.nonzero(idx == e, as_tuple=True)
            gu = x[t] @ Wg[e].T + bg[e]
            a = torch.nn.functional.silu(gu[:, :self.I]) * gu[:, self.I:]
            Y = Y.index_add(0, t, w[t, j][:, None] * (a @ Wd[e].T + bd[e]))
        Y.backward(self.dY.double())
        return dict(Y=Y.detach(), dX=x.grad, dW_gu=Wg.grad, dW_down=Wd.grad, db_gu=bg.grad, db_down=bd.grad,
                    dz=z.grad, w=w.detach())


SIZES = [("f32", 67, 8, 2, 64, 128), ("bf16", 67, 8, 2, 64, 128), ("bf16", 517, 5, 3, 264, 136),
         ("bf16", 3, 40, 8, 2056, 264), ("f32", 130, 33, 4, 100, 36), ("bf16", 1500, 6, 2, 2048, 392)]


@pytest.mark.parametrize("dt,T,E,k,H,I", SIZES)
def test_forward_and_backward_of_a_layer(dt, T, E, k, H, I):
    layer = Layer(T, E, k, H, I, dt)
    layer.out["status"].zero_()
    layer.forward()
    layer.backward()
    assert int(layer.out["status"].item()) == 0
    got, ref = layer.results(), layer.reference()
    assert (layer.idx[T - 2:] == -1).all() and (layer.idx[:T - 2] >= 0).all()
    assert torch.equal(got["Y"][T - 2:], layer.res[T - 2:])
    for n, r in ref.items():
        err = (got[n].double() - r).norm().item() / r.norm().item()
        assert err <= TOL[dt] * (4 if n == "dz" else 1), (n, err)


def test_shared_expert_on_top_of_the_routed_ones():
    """A dense expert (E = 1, identity offsets) whose linear product adds to the combined output in
    place, and its gradients by the grouped calls."""
    T, H, I = 259, 136, 264
    layer = Layer(T, 8, 2, H, I, "bf16")
    layer.out["status"].zero_()
    layer.forward()
    g = torch.Generator(device="cuda").manual_seed(9)
    Wg = (torch.randn(1, 2 * I, H, generator=g, device="cuda") * H ** -0.5).bfloat16()
    Wd = (torch.randn(1, H, I, generator=g, device="cuda") * I ** -0.5).bfloat16()
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    before = layer.Y.double()
    A = torch.empty(T, I, dtype=torch.bfloat16, device="cuda")
    L.lrmoe_grouped_swiglu(layer.x, Wg, off, A)
    L.lrmoe_grouped_linear(A, Wd, off, layer.Y, residual=layer.Y)
    gu = layer.x.double() @ Wg[0].double().T
    want = before + (torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]) @ Wd[0].double().T
    assert ((layer.Y.double() - want).norm() / want.norm()).item() < TOL["bf16"]


def test_one_graph_of_forward_and_backward():
    """Captured once, replayed on new inputs: the eager bits."""
    la = Layer(301, 8, 2, 136, 264, "bf16")
    la.out["status"].zero_()
    la.forward()
    la.backward()
    want = la.results()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        la.forward()
        la.backward()
    gr.replay()
    torch.cuda.synchronize()
    for n, t in la.results().items():
        assert torch.equal(t, want[n]), n
    la.x.copy_(torch.randn_like(la.x, dtype=torch.float32))
    la.logits[:-2].copy_(torch.randn_like(la.logits[:-2]))
    gr.replay()
    torch.cuda.synchronize()
    got = la.results()
    la.forward()
    la.backward()
    torch.cuda.synchronize()
    for n, t in la.results().items():
        assert torch.equal(t, got[n]), n


def test_graphs_on_streams_at_once():
    """The forward operators and their gradients share no state: two graphs replayed on two streams at
    once, beside eager calls on a third, give the eager bits."""
    def step(la):
        la.forward()
        L.lrmoe_grouped_bias_grad(la.a, la.out["offsets"], db[la])
        L.lrmoe_route_grad(la.logits, la.idx, la.dw, la.dz)

    layers = [Layer(301, 8, 2, 136, 264, "bf16", seed=s) for s in (1, 2, 3)]
    db = {la: torch.empty(8, 264, device="cuda") for la in layers}
    outputs = lambda la: [t.clone() for t in (la.Y, la.y, la.g, la.Ap, la.idx, la.w, la.dz, db[la])]  # noqa: E731
    want = []
    for la in layers:
        la.out["status"].zero_()
        la.dw.normal_()
        la.Ap.zero_()
        step(la)
        want.append(outputs(la))
    graphs = []
    for la in layers[:2]:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step(la)
        graphs.append(gr)
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(100):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        with torch.cuda.stream(streams[2]):
            step(layers[2])
    torch.cuda.synchronize()
    for la, w in zip(layers, want):
        for t, v in zip(outputs(la), w):
            assert torch.equal(t, v)


def test_explicit_stream_argument():
    la = Layer(64, 8, 2, 64, 128, "bf16")
    la.out["status"].zero_()
    la.forward()
    torch.cuda.synchronize()
    want, s = la.results(), torch.cuda.Stream()
    la.Y.zero_()
    torch.cuda.synchronize()
    L.lrmoe_combine(la.y, la.idx, la.w, 8, la.Y, residual=la.res, stream=s)
    s.synchronize()
    assert torch.equal(la.Y, want["Y"])


@pytest.mark.parametrize("dt,T,E,k,H,I", SIZES + [("bf16", 17, 1, 1, 64, 64), ("f32", 5, 3, 3, 8, 4)])
def test_guard_pages(dt, T, E, k, H, I):
    """Every buffer of the chain sits between sentinel pages that stay unchanged."""
    G = Guard()
    la = Layer(max(T, 3), E, k, H, I, dt, new=G.empty)
    keep = {n: getattr(la, n).clone() for n in ("logits", "x", "dY", "res", "W_gu", "W_down", "b_gu", "b_down")}
    la.out["status"].zero_()
    for score in (L.LRMOE_SCORE_SIGMOID, L.LRMOE_SCORE_SOFTMAX):
        la.forward(score_fn=score)
        la.backward()
    for renorm in (True, False):
        L.lrmoe_route_grad(la.logits, la.idx, la.dw, la.dz, renormalise=renorm)
    G.check()
    for n, t in keep.items():
        assert torch.equal(getattr(la, n), t), n


def test_checked_build():
    """The chain on the checked-index library gives status 0, and offsets that fall or end past the
    rows set LRMOE_ST_BAD_INDEX and write nothing (the grouped products) or count as empty experts
    (the bias gradient)."""
    env = dict(os.environ, LRMOE_CHECKED="1", PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "forward_checked_child.py")], env=env,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "ok" in r.stdout
