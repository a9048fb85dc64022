"""The gradient norm and the AdamW step over many tensors against the 64-bit forms.

Tolerances (u = 2^-24).  m: two products, a sum and the factor 1 - beta1 rounded to 32 bits, of the scaled
gradient (one more): 5 u of the two terms' sizes; v alike with the square: 7 u of itself.  The step: rate
and 1 / sqrt(1 - beta2^t) are rounded (2 u), the root of v is within 3.5 u + 2 u (sqrt.approx is good to
2^-23), its product and sum with eps 2 u, the quotient 2 u + 1: 15 u of the step's terms, and the sums
3 u of weight and step.  Codes: x = value / scale is within 8 u more of itself, at most 16 steps of a code, so the
choice between two neighbours is that of 64 bits where it lies further than 16 * 32 u = 3.1e-5 from its border.
"""
import math

import numpy as np
import pytest
import torch

from pruned_expert_backward_lrmoe_b200 import lrmoe as L
from tests import forward_ref as R
from tests import step_ref as S
from tests.test_canary_gpu import Guard

pytestmark = pytest.mark.gpu

TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24
NEAR = 1e-4


class Tensors:
    """Tensors of the given shapes with states that a few steps could have left."""

    def __init__(self, shapes, dt="f32", grad="f32", bits=32, master=False, seed=0, decay=0.1, fresh=False, new=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda s, scale: torch.randn(s, generator=g, device="cuda") * scale  # noqa: E731
        new = new or (lambda shape, dtype: torch.empty(shape, dtype=dtype, device="cuda"))
        put = lambda t: new(t.shape, t.dtype).copy_(t)  # noqa: E731
        self.dt, self.bits, self.master, self.shapes = dt, bits, master, shapes
        self.decay = [decay * (i % 3) for i in range(len(shapes))]
        full = [rand(s, 0.05) for s in shapes]
        self.state = {"params": [put(p.to(TYPE[dt])) for p in full]}
        if master:
            self.state["master"] = [put(p) for p in full]
        self.grads = [put(rand(s, 1e-3).to(TYPE[grad])) for s in shapes]
        m = [rand(s, 0.0 if fresh else 3e-4) for s in shapes]
        r = [rand(s, 0.0 if fresh else 1e-3).abs() for s in shapes]
        if bits == 32:
            self.state.update(m=[put(x) for x in m], v=[put(x * x) for x in r])
        else:
            for name, xs in (("m", m), ("v", r)):
                self.state[name], self.state[name + "_scale"] = [], []
                for x in xs:
                    sc = torch.from_numpy(S.scales(x.double().cpu().numpy().reshape(-1))).float().cuda()
                    q = x.reshape(-1) / sc.repeat_interleave(256)[:x.numel()].clamp_min(1e-30)
                    q = q.to(torch.float8_e4m3fn).view(torch.uint8).reshape(x.shape)
                    self.state[name].append(new(q.shape, torch.uint8).copy_(q).view(torch.float8_e4m3fn))
                    self.state[name + "_scale"].append(put(sc))
        self.list = L.TensorList(self.grads, weight_decay=self.decay, **self.state)

    def host(self):
        """Everything as it is, in 64 bits, one dict a tensor."""
        out = []
        for i, g in enumerate(self.grads):
            d = {n: ts[i].double().cpu().numpy().reshape(-1) for n, ts in self.state.items()}
            d["grad"] = g.double().cpu().numpy().reshape(-1)
            out.append(d)
        return out

    def check(self, before, lr, step, beta1, beta2, eps, scale, seed):
        after = self.host()
        for i, (a, b) in enumerate(zip(before, after)):
            n = a["grad"].size
            if n == 0:
                continue
            m0, v0 = a["m"], a["v"]
            if self.bits == 8:
                m0 = m0 * S.spread(a["m_scale"], n)
                v0 = (v0 * S.spread(a["v_scale"], n)) ** 2
            p0 = a["master"] if self.master else a["params"]
            p, m, v, size = S.adamw(p0, a["grad"], m0, v0, lr, step, beta1, beta2, eps, self.decay[i], scale)
            tol = 3 * U * (np.abs(p0) + size) + 15 * U * size
            w = S.words(seed, step, i, n)
            if self.master:
                assert (np.abs(b["master"] - p) <= tol).all(), i
                assert (b["params"] == torch.from_numpy(b["master"]).float().bfloat16().double().numpy()).all(), i
            elif self.dt == "f32":
                assert (np.abs(b["params"] - p) <= tol).all(), i
            else:
                want, edge = S.bf16_random(p, (w * np.uint64(0x9E3779B1) & np.uint64(0xFFFFFFFF)) >> np.uint64(16))
                # p is at most 256 steps of a bf16; its error there
                sure = edge > 256 * tol / np.maximum(np.abs(p), 1e-30) + 2.0 ** -15
                assert (b["params"][sure] == want[sure]).all(), i
                assert (np.abs(b["params"] - p) <= 2 * 2.0 ** -7 * np.abs(p) + tol).all(), i
            sm = 5 * U * (np.abs(beta1 * m0) + np.abs((1 - beta1) * scale * a["grad"])) + 2.0 ** -140
            if self.bits == 32:
                assert (np.abs(b["m"] - m) <= sm).all(), i
                assert (np.abs(b["v"] - v) <= 7 * U * v + 2.0 ** -140).all(), i
                continue
            for name, x, bits, keep in (("m", m, w & np.uint64(0xFFFF), False), ("v", np.sqrt(v), w >> np.uint64(16), True)):
                s = S.scales(x)
                assert (np.abs(b[name + "_scale"] - s) <= 16 * U * s).all(), (i, name)
                want, edge = S.codes(x, S.spread(s, n), bits.astype(np.float64), keep)
                # m's error is relative to its terms, which may be larger than itself
                y = np.abs(x) / np.maximum(S.spread(s, n), 1e-300)
                loose = (sm / np.maximum(S.spread(s, n), 1e-300) + 32 * U * y) / S.e4m3_step(y)
                sure = edge > loose + NEAR
                assert (b[name][sure] == want[sure]).all(), (i, name)
                assert (np.abs(b[name] - want) <= S.e4m3_step(np.maximum(y, np.abs(want)))).all(), (i, name)
                assert sure.mean() > 0.99 or n < 5000, (i, name)
                if keep:
                    assert (b[name][x > 0] > 0).all(), i


SHAPES = [(1,), (3,), (4,), (255,), (256,), (257,), (2047,), (2048,), (2049,), (0,), (7, 33), (4, 96, 64), (5, 1000), (300001,)]
HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-8)
KINDS = [("f32", "f32", False), ("f32", "bf16", False), ("bf16", "f32", True), ("bf16", "bf16", True), ("bf16", "f32", False),
         ("bf16", "bf16", False)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dt,grad,master", KINDS)
def test_step(dt, grad, master, bits):
    t = Tensors(SHAPES, dt, grad, bits, master)
    scale = torch.tensor([0.25], device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for step, seed, sc in ((1, 0, None), (2, 12345, scale), (1000, 2 ** 32 - 1, scale)):
        before = t.host()
        L.lrmoe_adamw(t.list, step=step, seed=seed, grad_scale=sc, status=st, **HYPER)
        t.check(before, step=step, seed=seed, scale=1.0 if sc is None else 0.25, **HYPER)
    assert int(st.item()) == 0


@pytest.mark.parametrize("bits", [32, 8])
def test_first_step_from_nothing(bits):
    """Without history the step is lr sign(g), whatever the gradient's size."""
    shapes = [(1000,), (3, 5)]
    t = Tensors(shapes, bits=bits, fresh=True, decay=0.0)
    st = L.alloc_adamw(t.state["params"], bits)
    for n in st:
        for x, y in zip(st[n], t.state[n]):
            assert x.shape == y.shape and x.dtype == y.dtype and (x.float() == y.float()).all()
    before = t.host()
    L.lrmoe_adamw(t.list, step=1, **HYPER)
    t.check(before, step=1, seed=0, scale=1.0, **HYPER)
    for a, b in zip(before, t.host()):
        moved = a["params"] - b["params"]
        # eps 1e-8 beside gradients of 1e-3 and more than 1e-6: within 1e-2
        big = np.abs(a["grad"]) > 1e-6
        assert (np.abs(moved - HYPER["lr"] * np.sign(a["grad"]))[big] <= 1.1e-2 * HYPER["lr"]).all()


@pytest.mark.parametrize("count", [1, 24, 25, 112, 113, 448, 449, 1000])
@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors(count, bits):
    """More tensors than fit a launch; each of its own size, empty ones among them."""
    rng = np.random.default_rng(count)
    t = Tensors([(int(n),) for n in rng.integers(0, 700, count)], bits=bits)
    if not any(g.numel() for g in t.grads):
        return
    before = t.host()
    L.lrmoe_adamw(t.list, step=3, seed=9, **HYPER)
    t.check(before, step=3, seed=9, scale=1.0, **HYPER)
    out, ws = torch.zeros(2, device="cuda"), torch.empty(L.lrmoe_grad_norm_workspace_bytes(count), dtype=torch.uint8, device="cuda")
    L.lrmoe_grad_norm(t.list, out, ws)
    want = math.sqrt(sum((a["grad"] ** 2).sum() for a in before))
    assert abs(out[0].item() - want) <= 20 * U * want and out[1].item() == 1.0


def test_step_and_rate_on_the_device():
    a, b = Tensors(SHAPES, bits=8, seed=4), Tensors(SHAPES, bits=8, seed=4)
    step, lr = torch.tensor([7], dtype=torch.int32, device="cuda"), torch.tensor([1e-2], device="cuda")
    L.lrmoe_adamw(a.list, lr=1e-2, step=7, seed=3)
    L.lrmoe_adamw(b.list, lr=lr, step=step, seed=3)
    for n in a.state:
        for x, y in zip(a.state[n], b.state[n]):
            # the two corrections may be rounded from 64-bit numbers that differ in their last bits
            x, y = x.double(), y.double()
            assert ((x - y).abs() <= 4 * U * x.abs() + (S.e4m3_step(0.0) if n in "mv" else 0)).all(), n
    step.fill_(0)                                            # counts as 1
    c, d = Tensors(SHAPES, seed=4), Tensors(SHAPES, seed=4)
    L.lrmoe_adamw(c.list, lr=1e-2, step=1)
    L.lrmoe_adamw(d.list, lr=lr, step=step)
    for x, y in zip(c.state["params"], d.state["params"]):
        assert ((x - y).abs() <= 4 * U * x.abs() + 1e-2 * 4 * U).all()


@pytest.mark.parametrize("n", [5000, 200])
def test_products_and_sums_of_the_states_are_rounded_one_by_one(n):
    """Bit for bit what elementary operations give: whether a value next to a border of its 8-bit code falls on one side
    or the other hangs on the last bit."""
    t = Tensors([(n,)], seed=12)
    g, m, v = t.grads[0] * 0.5, t.state["m"][0].clone(), t.state["v"][0].clone()
    b1, b2, a1, a2 = (torch.tensor(x, device="cuda") for x in (0.9, 0.95, 1 - 0.9, 1 - 0.95))
    L.lrmoe_adamw(t.list, lr=1e-3, step=10, beta1=0.9, beta2=0.95, grad_scale=torch.tensor([0.5], device="cuda"))
    x, y = b1 * m, a1 * g
    m1 = x + y
    x, y = b2 * v, a2 * g * g
    v1 = x + y
    assert torch.equal(t.state["m"][0], m1) and torch.equal(t.state["v"][0], v1)
    # and from 8-bit states the scales, which show the largest of each block
    e = Tensors([(n,)], bits=8, seed=12)
    spread = lambda s: s.repeat_interleave(256)[:n]  # noqa: E731
    m0 = e.state["m"][0].float() * spread(e.state["m_scale"][0])
    v0 = (e.state["v"][0].float() * spread(e.state["v_scale"][0])).square()
    L.lrmoe_adamw(e.list, lr=1e-3, step=10, beta1=0.9, beta2=0.95, grad_scale=torch.tensor([0.5], device="cuda"))
    x, y = b1 * m0, a1 * (e.grads[0] * 0.5)
    top = torch.nn.functional.pad((x + y).abs(), (0, -n % 256)).view(-1, 256).amax(1)
    assert torch.equal(e.state["m_scale"][0], top * (1 / torch.tensor(448.0, device="cuda")))


@pytest.mark.parametrize("beta1,beta2", [(0.0, 0.0), (0.9, 0.0), (0.0, 0.999), (0.9999, 0.99999)])
def test_betas(beta1, beta2):
    t = Tensors([(3000,), (17,)])
    before = t.host()
    how = dict(lr=1e-3, beta1=beta1, beta2=beta2, eps=1e-6)
    L.lrmoe_adamw(t.list, step=5, **how)
    t.check(before, step=5, seed=0, scale=1.0, **how)


@pytest.mark.parametrize("dt,grad,master", KINDS)
@pytest.mark.parametrize("bits", [32, 8])
def test_gradients_that_are_not_finite_leave_their_elements(bits, dt, grad, master):
    t = Tensors([(700,), (40,)], dt, grad, bits, master, decay=0.0)
    bad = [3, 255, 256, 699]
    for i, x in zip(bad, (float("nan"), float("inf"), -float("inf"), 1e30)):  # the last one's square overflows
        t.grads[0][i] = x
    before = t.host()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.lrmoe_adamw(t.list, step=2, status=st, **HYPER)
    after = t.host()
    assert int(st.item()) == R.NONFINITE
    for n in ("params",) + (("master",) if master else ()) + (("m", "v") if bits == 32 else ()):
        assert (after[0][n][bad] == before[0][n][bad]).all(), n
    assert all(np.isfinite(x).all() for d in after for n, x in d.items() if n != "grad")
    if bits == 8:  # held again with the block's new scale
        for n in ("m", "v"):
            old, new = (d[0][n][bad] * S.spread(d[0][n + "_scale"], 700)[bad] for d in (before, after))
            step = S.e4m3_step(np.abs(after[0][n][bad])) * S.spread(after[0][n + "_scale"], 700)[bad]
            assert (np.abs(new - old) <= 1.01 * step).all()
    good = np.ones(700, bool)
    good[bad] = False
    assert (after[0]["params"][good] != before[0]["params"][good]).mean() > (0.9 if dt == "f32" else 0.05)


def test_scale_of_zero_skips_the_step():
    t = Tensors(SHAPES, "bf16", bits=8)
    before = t.host()
    L.lrmoe_adamw(t.list, step=2, grad_scale=torch.zeros(1, device="cuda"), **HYPER)
    for a, b in zip(before, t.host()):
        assert all((a[n] == b[n]).all() for n in a)


def test_random_rounding_is_right_on_average():
    """One value in every element of a block but the largest: the mean of its codes is the value."""
    n = 256 * 4096
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.full((n,), 0.3717, device="cuda")
    g[::256] = 1.0
    p.fill_(1.0)
    st = L.alloc_adamw([p], 8)
    t = L.TensorList([g], [p], **st)
    L.lrmoe_adamw(t, lr=1e-3 * 0.7, step=1, beta1=0.9, beta2=0.9, seed=11)
    inner = torch.ones(n, dtype=torch.bool, device="cuda")
    inner[::256] = False
    for name, want in (("m", 0.3717), ("v", 0.3717)):
        x = st[name][0].double()[inner]          # the codes; the block's largest value is 448
        q = float(S.e4m3_step(want * 448))
        assert set((x / q).unique().tolist()) <= {math.floor(want * 448 / q), math.ceil(want * 448 / q)}
        # a choice between neighbours has a standard deviation of half a step at most
        assert abs(x.mean().item() - want * 448) < 5 * 0.5 * q / math.sqrt(n)
    x = p.double()  # 1 - 7e-4, between 1 - 2^-8 and 1
    assert set(x.unique().tolist()) <= {1.0, 1 - 2.0 ** -8}
    assert abs(x.mean().item() - (1 - 7e-4)) < 5 * 0.5 * 2.0 ** -8 / math.sqrt(n) + 1e-6


def test_root_is_that_of_cuda():
    """The root behind the 8-bit states against torch's square root: a block of one value shows it as its scale.  It
    is right to the last bit but where the root lies next to the middle of two numbers: less than one in 10^5."""
    n = 1 << 18
    g = torch.zeros(n, 256, device="cuda")
    e = torch.empty(n, device="cuda").uniform_(-55, 40, generator=torch.Generator(device="cuda").manual_seed(2))
    g[:, 5] = torch.exp2(e)
    p = torch.zeros_like(g)
    st = L.alloc_adamw([p], 8)
    L.lrmoe_adamw(L.TensorList([g], [p], **st), lr=1e-3, step=1, beta1=0.9, beta2=0.9)
    a2 = torch.tensor(1 - 0.9, device="cuda")
    want = torch.sqrt(a2 * g[:, 5] * g[:, 5]) * (1 / torch.tensor(448.0))
    got = st["v_scale"][0]
    off = got != want
    assert off.sum().item() <= n * 1e-5
    assert ((got - want).abs() <= 2 * U * want).all()


def test_rounding_depends_on_seed_and_step_alone():
    def after(seed, step, seed_of_data=0):
        t = Tensors([(5000,)], "bf16", bits=8, seed=seed_of_data)
        L.lrmoe_adamw(t.list, step=step, seed=seed, **HYPER)
        return [x.view(torch.uint8 if x.element_size() == 1 else torch.int16) for x in (t.state["m"][0], t.state["params"][0])]

    a, b, c = after(1, 5), after(1, 5), after(2, 5)
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and not any(torch.equal(x, y) for x, y in zip(a, c))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dt,grad,master", KINDS)
def test_nothing_outside_the_tensors_is_written(dt, grad, master, bits):
    G = Guard()
    t = Tensors([(1,), (5,), (255,), (2050,), (9999,)], dt, grad, bits, master, new=G.empty)
    before = t.host()
    L.lrmoe_adamw(t.list, step=4, **HYPER)
    t.check(before, step=4, seed=0, scale=1.0, **HYPER)
    out = G.empty((2,), torch.float32)
    ws = G.empty((L.lrmoe_grad_norm_workspace_bytes(5),), torch.uint8)
    L.lrmoe_grad_norm(t.list, out, ws)
    G.check()


@pytest.mark.parametrize("at", [2 ** 31 + 12345, 2 ** 32 + 300])
def test_offsets_past_32_bits(at):
    """The last values of a tensor with more than 2^31 and 2^32 values take their step, with their random words."""
    n = at + 77
    kw = dict(device="cuda")
    p, g = torch.zeros(n, dtype=torch.bfloat16, **kw), torch.zeros(n, dtype=torch.bfloat16, **kw)
    st = L.alloc_adamw([p], 8)
    t = L.TensorList([g], [p], **st)
    tail = torch.linspace(-1, 1, 77).bfloat16()
    g[at:], p[at:] = tail.cuda(), 1.0
    L.lrmoe_adamw(t, lr=1e-3, step=1, beta1=0.9, beta2=0.9, seed=5)
    x, _, _, _ = S.adamw(np.ones(77), tail.double().numpy(), 0, 0, 1e-3, 1, 0.9, 0.9)
    w = S.words(5, 1, 0, 77, at)
    want, edge = S.bf16_random(x, (w * np.uint64(0x9E3779B1) & np.uint64(0xFFFFFFFF)) >> np.uint64(16))
    sure = edge > 1e-3
    assert sure.sum() > 60
    assert (p[at:].double().cpu().numpy()[sure] == want[sure]).all()
    assert not p[:2048].any() and not st["m"][0][:at // 256 * 256].view(torch.uint8).any()
    out, ws = torch.zeros(2, **kw), torch.empty(L.lrmoe_grad_norm_workspace_bytes(1), dtype=torch.uint8, **kw)
    L.lrmoe_grad_norm(t, out, ws, max_norm=1.0)
    norm = tail.double().norm().item()
    assert abs(out[0].item() - norm) <= 1e-6 * norm and abs(out[1].item() - 1 / norm) <= 1e-6


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------
def norm_of(tensors, max_norm=math.inf):
    out = torch.full((2,), 77.0, device="cuda")
    ws = torch.full((L.lrmoe_grad_norm_workspace_bytes(len(tensors)),), 0xEE, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.lrmoe_grad_norm(L.TensorList(tensors), out, ws, max_norm=max_norm, status=st)
    return out[0].item(), out[1].item(), int(st.item())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shapes", [[(1,)], [(0,)], [(0,), (0, 4)], [(5,), (0,), (2049,)], SHAPES, [(1000, 3001)],
                                    [(32 * 2048,)], [(32 * 2048 + 1,)], [(7,)] * 32, [(7,)] * 33, [(4 * 2048,)], [(4 * 2048 + 1,)]])
def test_norm(shapes, dt):
    g = torch.Generator(device="cuda").manual_seed(1)
    ts = [torch.randn(s, generator=g, device="cuda").to(TYPE[dt]) for s in shapes]
    want = math.sqrt(sum(t.double().square().sum().item() for t in ts))
    # 16 squares and sums in 32 bits, halved by the root, and one rounding
    for most in (math.inf, want * 2 + 1, want / 3 if want else 1.0):
        norm, factor, st = norm_of(ts, most)
        assert st == 0 and abs(norm - want) <= 20 * U * want
        assert abs(factor - (min(1.0, most / want) if want else 1.0)) <= 20 * U


@pytest.mark.parametrize("scale", [1e-44, 1e-30, 1e-22, 1e18, 1e25, 2e37, 3e37])
def test_norm_of_values_whose_squares_leave_32_bits(scale):
    x = torch.tensor([3.0, 0.0, -4.0, 12.0], device="cuda") * scale
    want = x.double().norm().item()
    norm, factor, st = norm_of([x, x.new_zeros(5000)], want / 2)
    if not math.isfinite(want):  # 12 * 3e37 is more than 32 bits hold: the gradient itself is infinite
        assert (norm, factor, st) == (math.inf, 0.0, R.NONFINITE)
        return
    # max_norm itself is a 32-bit number: 1e-44 / 2 is a few of its smallest steps, so not half of the norm
    half = float(np.float32(want / 2)) / want
    assert st == 0 and abs(norm - want) <= 4 * U * want + 2.0 ** -150 and abs(factor - half) <= 4 * U


def test_norm_that_is_not_finite():
    for x in (float("nan"), float("inf")):
        t = torch.ones(3000, device="cuda")
        t[2777] = x
        norm, factor, st = norm_of([t], 1.0)
        assert not math.isfinite(norm) and factor == 0.0 and st == R.NONFINITE
