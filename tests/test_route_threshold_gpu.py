"""Routing of tokens of which more keys reach the threshold of the first selection than a warp has lanes,
against 64 bits: they go on to the selection by rounds, and the near ones to the order in fp64, which
uses the same words of shared memory."""
import pytest
import torch

from pruned_expert_backward_lrmoe_b200 import lrmoe as L

pytestmark = pytest.mark.gpu

FN = {"softmax": L.LRMOE_SCORE_SOFTMAX, "sigmoid": L.LRMOE_SCORE_SIGMOID}


# Lanes hold ceil(E / 32) experts rounded up to a power of two: with k = 16 and these E hardly more
# lanes than slots hold any, and most tokens have more keys above the threshold than fit the lanes.
# The equal and nearly equal logits then send many of them on to the order in fp64.
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,G,keep", [(130, 16, 1, 1), (160, 16, 1, 1), (300, 16, 1, 1), (72, 16, 1, 1),
                                        (160, 16, 8, 4), (32, 32, 1, 1), (48, 32, 1, 1), (64, 31, 1, 1)])
@pytest.mark.parametrize("size", [None, 0.0, 0.02, 1e4])
def test_route_of_many_keys_at_the_threshold(E, k, G, keep, kind, size):
    g = torch.Generator("cuda").manual_seed(E + k)
    T = 20000
    z = torch.randn(T, E, generator=g, device="cuda")
    near = 3.0 + torch.randint(0, 40, (T // 2, E), generator=g, device="cuda") * 2.0 ** -22
    z[::2] = torch.where(torch.rand(T // 2, E, generator=g, device="cuda") < 0.3, near, z[::2])
    bias = None if size is None else torch.randn(E, generator=g, device="cuda") * size
    d = z.double()
    s = 1 / (1 + torch.exp(-d)) if kind == "sigmoid" else torch.softmax(d, 1)
    key = s + (0 if bias is None else bias.double())
    value = key.view(T, G, E // G).topk(min(2, E // G), 2).values.sum(2)
    kept = torch.zeros_like(value, dtype=torch.bool)
    kept.scatter_(1, value.sort(dim=1, descending=True, stable=True).indices[:, :keep], True)
    order = (d if bias is None else key).masked_fill(~kept.repeat_interleave(E // G, 1), -float("inf"))
    want = order.sort(dim=1, descending=True, stable=True).indices[:, :k]
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.lrmoe_route(z, idx, w, bias=bias, score_fn=FN[kind], n_group=G, topk_group=keep, status=st)
    assert torch.equal(idx.long(), want) and int(st.item()) == 0
    ref = s.gather(1, want)
    ref = ref / ref.sum(1, keepdim=True)
    # |z| and |z - z_max| / 2 stay below 6: the routing tests' (2 D + 56) u with D = 12
    assert bool(((w - ref).abs() <= 80 * 2.0 ** -24 * ref).all())
