"""Captured forward operators, with every output filled with a wrong value before each replay and
compared after each: a replay that skips a tile, a row or a whole call cannot pass on what an
earlier call left behind, nor a wrong round on a later right one."""
import pytest
import torch

from pruned_expert_backward_lrmoe_b200 import lrmoe as L
from tests.test_forward_gpu import Layer

pytestmark = pytest.mark.gpu

ROUNDS = 60


def poison(tensors):
    for t in tensors:
        t.fill_(77)


def differences(tensors, want):
    """Number of bytes that differ, on the device."""
    return sum((t.reshape(-1).view(torch.uint8) != v.reshape(-1).view(torch.uint8)).sum() for t, v in zip(tensors, want))


# experts of a few rows (one-SM tiles), and of several tiles each (both launches of a product)
@pytest.mark.parametrize("T,E,k", [(301, 8, 2), (1500, 3, 2)])
def test_graphs_on_streams_at_once_write_every_output_in_every_round(T, E, k):
    """Two graphs replayed on two streams at once, beside eager calls on a third, on inputs that change."""
    I, H = 264, 136
    layers = [Layer(T, E, k, H, I, "bf16", seed=s) for s in (1, 2, 3)]
    db = [torch.empty(E, I, device="cuda") for _ in layers]

    def outputs(i):
        la = layers[i]
        return [la.Y, la.y, la.g, la.u, la.a, la.Ap, la.idx, la.w, la.dz, db[i]]

    def step(i):
        la = layers[i]
        la.forward()
        L.lrmoe_grouped_bias_grad(la.Ap, la.out["offsets"], db[i])
        L.lrmoe_route_grad(la.logits, la.idx, la.dw, la.dz)

    sets, want = [], []
    for i, la in enumerate(layers):
        la.out["status"].zero_()
        la.dw.normal_()
        other = Layer(T, E, k, H, I, "bf16", seed=10 + i)
        sets.append([(la.x.clone(), la.logits.clone()), (other.x, other.logits)])
        want.append([])
        for x, z in sets[i]:
            la.x.copy_(x)
            la.logits.copy_(z)
            poison(outputs(i))
            step(i)
            want[i].append([t.clone() for t in outputs(i)])
    assert all(not torch.equal(w[0][0], w[1][0]) for w in want)
    graphs = []
    for i in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step(i)
        graphs.append(gr)
    wrong = [torch.zeros((), dtype=torch.int64, device="cuda") for _ in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for r in range(ROUNDS):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                layers[i].x.copy_(sets[i][r & 1][0])
                layers[i].logits.copy_(sets[i][r & 1][1])
                poison(outputs(i))
                graphs[i].replay() if i < 2 else step(i)
                wrong[i] += differences(outputs(i), want[i][r & 1])
    torch.cuda.synchronize()
    assert [int(w.item()) for w in wrong] == [0, 0, 0]
    assert all(int(la.out["status"].item()) == 0 for la in layers)


def test_a_graph_of_forward_and_backward_writes_every_result():
    la = Layer(301, 8, 2, 136, 264, "bf16")
    la.out["status"].zero_()
    results = lambda: [la.Y, la.out["dX"], la.out["dW_gu"], la.out["dW_down"], la.db_gu, la.db_down, la.dz,  # noqa: E731
                       la.idx, la.w, la.dw]
    la.forward()
    la.backward()
    want = [t.clone() for t in results()]
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        la.forward()
        la.backward()
    for _ in range(3):
        poison(results() + [la.Ap])
        gr.replay()
        assert int(differences(results(), want).item()) == 0
    assert int(la.out["status"].item()) == 0
