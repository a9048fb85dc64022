"""The operators that close a training step without a GPU: the 64-bit forms that the GPU tests compare with
are pinned to worked examples and differences, and the entry points refuse what they cannot do."""
import ctypes

import numpy as np
import pytest
import torch

from pruned_expert_backward_lrmoe_b200 import build as B
from pruned_expert_backward_lrmoe_b200 import lrmoe as L
from tests import step_ref as S

NULL, FAKE = ctypes.c_void_p(0), ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10004)
UNEVEN = ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


# ---------------------------------------------------------------------------
# the 64-bit forms
# ---------------------------------------------------------------------------
def test_balance_worked_example():
    z = np.log(np.array([[3.0, 1.0], [1.0, 1.0], [1.0, 3.0], [1.0, 1.0]]))
    idx = np.array([[0, -1], [0, 1], [1, 0], [-1, -1]], np.int32)
    r = S.balance(z, idx, coef=2.0, z_coef=1.0)
    assert r["counts"].tolist() == [[3, 2]] and r["stats"].tolist() == [[3, 5], [3, 1]]
    np.testing.assert_allclose(r["mean"], [[0.5, 0.5]])
    # E sum c P / m = 2 (3/2 + 2/2) / 5 = 1; z: (log^2 4 + log^2 2 + log^2 4) / 3 = 3 log^2 2
    np.testing.assert_allclose(r["loss"], [2.0, 3 * np.log(2) ** 2])
    # two sequences and an empty one: each counts alone; the padded token is in none
    r = S.balance(z, idx, [0, 1, 1, 3])
    assert r["counts"].tolist() == [[1, 0], [0, 0], [2, 2]] and r["stats"].tolist() == [[1, 1], [0, 0], [2, 4], [3, 2]]
    np.testing.assert_allclose(r["mean"], [[0.75, 0.25], [0, 0], [0.375, 0.625]])
    np.testing.assert_allclose(r["loss"], [(1.5 + 1.0) / 2, 0])


def test_balance_of_even_routing_is_coef():
    rng = np.random.default_rng(0)
    T, E = 24, 6
    idx = np.arange(T * 2).reshape(T, 2) % E
    r = S.balance(rng.standard_normal((T, E)), idx, coef=0.5)
    np.testing.assert_allclose(r["loss"][0], 0.5)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("off", [None, [0, 3, 3, 8], [1, 4, 7]])
def test_balance_grad_is_the_difference_of_the_losses(kind, off):
    rng = np.random.default_rng(1)
    T, E, k, h = 9, 5, 3, 1e-6
    z = rng.standard_normal((T, E))
    z[2, 1] = -np.inf
    z[5] = -np.inf
    idx = rng.integers(-1, E, (T, k)).astype(np.int32)
    idx[4] = -1
    how = dict(off=off, kind=kind, coef=0.7, z_coef=0.3)
    up = np.array([1.5, -0.5])
    got, _ = S.balance_grad(z, idx, dloss=up, **how)
    for t in range(T):
        for e in range(E):
            if not np.isfinite(z[t, e]):
                assert got[t, e] == 0
                continue
            a, b = z.copy(), z.copy()
            a[t, e] += h
            b[t, e] -= h
            d = (S.balance(a, idx, **how)["loss"] - S.balance(b, idx, **how)["loss"]) @ up / (2 * h)
            assert abs(d - got[t, e]) < 1e-8, (t, e)


def test_adamw_is_torch_s():
    g = torch.Generator().manual_seed(3)
    p = torch.randn(50, generator=g, dtype=torch.float64).requires_grad_()
    opt = torch.optim.AdamW([p], lr=0.01, betas=(0.8, 0.97), eps=1e-6, weight_decay=0.2)
    q, m, v = p.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for t in range(1, 5):
        p.grad = torch.randn(50, generator=g, dtype=torch.float64)
        q, m, v, _ = S.adamw(q, p.grad.numpy(), m, v, 0.01, t, 0.8, 0.97, 1e-6, 0.2)
        opt.step()
        np.testing.assert_allclose(q, p.detach().numpy(), rtol=1e-12)


def test_codes_are_e4m3_and_right_on_average():
    x = np.linspace(0, 448, 1001)
    total = np.zeros_like(x)
    for b in range(0, 65536, 512):
        c, _ = S.codes(x, np.ones_like(x), b, False)
        t = torch.from_numpy(c).to(torch.float8_e4m3fn).double().numpy()
        assert (t == c).all()
        total += c
    # 128 equally spaced chances: at most one of them falls on the wrong side
    assert (np.abs(total / 128 - x) <= S.e4m3_step(x) / 128).all()


def test_words_do_not_lean():
    w = S.words(5, 7, 2, 1 << 16)
    for bits in (w & np.uint64(0xFFFF), w >> np.uint64(16), (w * np.uint64(0x9E3779B1) & np.uint64(0xFFFFFFFF)) >> np.uint64(16)):
        # the mean of 2^16 uniform 16-bit numbers has a standard deviation of 74
        assert abs(bits.astype(float).mean() - 32767.5) < 5 * 74
    assert (S.words(5, 7, 2, 100, 2 ** 32) != S.words(5, 7, 2, 100)).any()
    assert (S.words(5, 8, 2, 100) != S.words(5, 7, 2, 100)).any() and (S.words(5, 7, 3, 100) != S.words(5, 7, 2, 100)).any()


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
def test_balance_refuses(lib):
    need = L.lrmoe_balance_workspace_bytes(100, 16, 3)
    assert need > 0 and L.lrmoe_balance_workspace_bytes(0, 16, 1) == 0
    assert L.lrmoe_balance_workspace_bytes(100, 2000, 1) == 0
    ok = [FAKE, 100, 16, 1, FAKE, 2, 0, FAKE, 3, 1.0, 0.0, FAKE, FAKE, FAKE, FAKE, FAKE, need, NULL, NULL]

    def refused(at, value, word, code=L.LRMOE_ERR_INVALID_ARG):
        a = list(ok)
        a[at] = value
        assert lib.lrmoe_balance(*a) == code, (at, value)
        assert word in lib.lrmoe_last_error(), lib.lrmoe_last_error()

    for at, word in ((0, b"logits"), (4, b"topk_idx"), (11, b"counts"), (12, b"stats"), (13, b"mean_score"), (14, b"loss")):
        refused(at, NULL, word)
        refused(at, ODD, word)
    refused(7, NULL, b"seq_offsets")          # three sequences without bounds
    refused(7, ODD, b"seq_offsets")
    for at, value in ((1, 0), (1, -1), (2, 0), (5, 0), (5, 33), (3, 7), (6, 2), (8, 0), (9, float("inf")), (9, float("nan")),
                      (10, float("inf")), (8, 2 ** 28)):
        refused(at, value, b"")
    one = list(ok)
    one[1], one[5] = 2 ** 30 + 1, 1
    assert lib.lrmoe_balance(*one) == L.LRMOE_ERR_INVALID_ARG and b"2^30" in lib.lrmoe_last_error()
    refused(2, 1025, b"1024", L.LRMOE_ERR_UNSUPPORTED)
    refused(15, NULL, b"workspace", L.LRMOE_ERR_WORKSPACE)
    refused(16, need - 1, b"workspace", L.LRMOE_ERR_WORKSPACE)
    refused(15, ODD, b"workspace")


def test_balance_grad_refuses(lib):
    ok = [FAKE, 100, 16, 1, FAKE, 2, 0, NULL, 1, 1.0, 0.0, FAKE, FAKE, NULL, NULL, ctypes.c_void_p(0x20000), NULL, NULL]

    def refused(at, value, word, code=L.LRMOE_ERR_INVALID_ARG):
        a = list(ok)
        a[at] = value
        assert lib.lrmoe_balance_grad(*a) == code, (at, value)
        assert word in lib.lrmoe_last_error(), lib.lrmoe_last_error()

    for at, word in ((0, b"logits"), (4, b"topk_idx"), (11, b"counts"), (12, b"stats"), (15, b"dlogits")):
        refused(at, NULL, word)
        refused(at, ODD, word)
    refused(13, UNEVEN, b"dloss")
    refused(14, ODD, b"add")
    refused(15, FAKE, b"dlogits")             # the logits themselves
    refused(8, 2, b"seq_offsets")
    refused(2, 1025, b"1024", L.LRMOE_ERR_UNSUPPORTED)
    for at, value in ((1, 0), (5, 33), (3, 7), (6, 2), (9, float("nan")), (10, float("inf"))):
        refused(at, value, b"")


def _c_list(n=2, **change):
    a = (L.lrmoe_tensor * n)()
    for i in range(n):
        for j, name in enumerate(("param", "grad", "m", "v", "m_scale", "v_scale")):
            setattr(a[i], name, 0x10000 * (10 * i + j + 1))
        a[i].n = 100
    for name, v in change.items():
        setattr(a[n - 1], name, v)
    return a


def test_grad_norm_refuses(lib):
    need = L.lrmoe_grad_norm_workspace_bytes(2)
    assert need > 0 and L.lrmoe_grad_norm_workspace_bytes(0) == 0
    ok = [_c_list(), 2, 0, 1.0, FAKE, FAKE, need, NULL, NULL]

    def refused(at, value, word, code=L.LRMOE_ERR_INVALID_ARG):
        a = list(ok)
        a[at] = value
        assert lib.lrmoe_grad_norm(*a) == code, (at, value)
        assert word in lib.lrmoe_last_error(), lib.lrmoe_last_error()

    refused(0, None, b"tensors")
    refused(1, 0, b"count")
    refused(2, 5, b"dtype")
    for v in (0.0, -1.0, float("nan")):
        refused(3, v, b"max_norm")
    refused(4, NULL, b"out")
    refused(5, NULL, b"workspace", L.LRMOE_ERR_WORKSPACE)
    refused(6, need - 1, b"workspace", L.LRMOE_ERR_WORKSPACE)
    refused(5, ODD, b"workspace")
    refused(0, _c_list(n=2, grad=None), b"tensor 1: grad")
    refused(0, _c_list(n=2, grad=0x10004), b"tensor 1: grad")
    a = _c_list()
    a[1].n = -1
    refused(0, a, b"tensor 1: n")


def test_adamw_refuses(lib):
    ok = [_c_list(), 2, 0, 0, 32, 0.1, NULL, 0.9, 0.99, 1e-8, 1, NULL, NULL, 0, NULL, NULL]

    def refused(at, value, word, **more):
        a = list(ok)
        a[at] = value
        for i, v in more.items():
            a[int(i[1:])] = v
        assert lib.lrmoe_adamw(*a) == L.LRMOE_ERR_INVALID_ARG, (at, value)
        assert word in lib.lrmoe_last_error(), lib.lrmoe_last_error()

    nan, inf = float("nan"), float("inf")
    refused(0, None, b"tensors")
    refused(1, 0, b"count")
    refused(2, 2, b"dtype")
    refused(3, 2, b"dtype")
    refused(4, 16, b"state_bits")
    for v in (-0.1, nan, inf):
        refused(5, v, b"lr")
    for at in (7, 8):
        for v in (-0.1, 1.0, nan):
            refused(at, v, b"beta")
    for v in (0.0, -1.0, nan, inf):
        refused(9, v, b"eps")
    refused(10, 0, b"step")
    for at in (6, 11, 12):
        refused(at, UNEVEN, b"4-byte")
    for name in ("param", "grad", "m", "v"):
        refused(0, _c_list(**{name: None}), b"tensor 1")
        refused(0, _c_list(**{name: 0x10008}), b"tensor 1")
    for name in ("m_scale", "v_scale"):
        refused(0, _c_list(**{name: None}), b"tensor 1", a4=8)
        refused(0, _c_list(**{name: 0x10002}), b"tensor 1", a4=8)
    for v in (-0.1, nan, inf):
        refused(0, _c_list(weight_decay=v), b"weight_decay")
    refused(0, _c_list(master=0x900000), b"some tensors", a2=1)
    one = _c_list(n=1, master=0x900000)
    refused(0, one, b"bf16", a1=1)


def test_tensor_list_refuses():
    z = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype)  # noqa: E731
    p, g, m, v = z(3, 5), z(3, 5), z(3, 5), z(3, 5)
    L.TensorList([g], [p], [m], [v], weight_decay=[0.1])
    bad = [
        (dict(grads=[]), "no tensors"),
        (dict(grads=[g], params=[p]), "go together"),
        (dict(grads=[g], m_scale=[z(1)]), "go with"),
        (dict(grads=[g], params=[p], m=[m, m], v=[v]), "2 tensors"),
        (dict(grads=[g, z(2)], params=[p, z(2)], m=[m, z(2)], v=[v, z(3)]), "v 1"),
        (dict(grads=[g.t()], params=[p], m=[m], v=[v]), "grad 0"),
        (dict(grads=[g.double()]), "dtype"),
        (dict(grads=[g, g.bfloat16()]), "grad 1"),
        (dict(grads=[g], params=[p], m=[m], v=[v], master=[z(3, 5)]), "bf16"),
        (dict(grads=[g], params=[p.bfloat16()], m=[m], v=[v], master=[p.bfloat16()]), "master 0"),
        (dict(grads=[g], params=[p], m=[m], v=[v], m_scale=[z(1)], v_scale=[z(1)]), "8-bit"),
        (dict(grads=[g], params=[p], m=[m.to(torch.float8_e4m3fn)], v=[v.to(torch.float8_e4m3fn)]), "8-bit"),
        (dict(grads=[g], params=[p], m=[m.to(torch.float8_e4m3fn)], v=[v.to(torch.float8_e4m3fn)], m_scale=[z(2)],
              v_scale=[z(1)]), "m_scale 0"),
        (dict(grads=[g], params=[p], m=[m.half()], v=[v.half()], m_scale=[z(1)], v_scale=[z(1)]), "state dtype"),
        (dict(grads=[g], params=[p], m=[m], v=[m]), "overlap"),
        (dict(grads=[g, z(3, 5)], params=[p, p], m=[m, z(3, 5)], v=[v, z(3, 5)]), "overlap"),
        (dict(grads=[p], params=[p], m=[m], v=[v]), "overlap"),
        (dict(grads=[g], params=[p], m=[m], v=[v], weight_decay=[0.1, 0.2]), "weight_decay"),
    ]
    for how, word in bad:
        with pytest.raises(ValueError, match=word):
            L.TensorList(**how)
    with pytest.raises(ValueError, match="gradients only"):
        L.lrmoe_adamw(L.TensorList([g]), lr=0.1, step=1)
    with pytest.raises(ValueError, match="CUDA"):
        L.lrmoe_adamw(L.TensorList([g], [p], [m], [v]), lr=0.1, step=1)
    with pytest.raises(ValueError, match="state_bits"):
        L.alloc_adamw([p], state_bits=16)


def test_balance_binding_refuses():
    i32 = dict(dtype=torch.int32)
    z, idx, ws = torch.zeros(4, 6), torch.zeros(4, 2, **i32), torch.zeros(10, dtype=torch.uint8)
    good = dict(counts=torch.zeros(2, 6, **i32), stats=torch.zeros(3, 2, **i32), mean_score=torch.zeros(2, 6),
                loss=torch.zeros(2), workspace=ws, seq_offsets=torch.zeros(3, **i32))
    for name, t in (("counts", torch.zeros(1, 6, **i32)), ("stats", torch.zeros(2, 2, **i32)), ("mean_score", torch.zeros(6)),
                    ("loss", torch.zeros(1)), ("workspace", torch.zeros(10)), ("seq_offsets", torch.zeros(3))):
        with pytest.raises(ValueError, match=name):
            L.lrmoe_balance(z, idx, **{**good, name: t})
    with pytest.raises(ValueError, match="CUDA"):
        L.lrmoe_balance(z, idx, **good)
    c, st = torch.zeros(1, 6, **i32), torch.zeros(2, 2, **i32)
    for more, word in ((dict(add=torch.zeros(4, 5)), "add"), (dict(dloss=torch.zeros(1)), "dloss"),
                       (dict(seq_offsets=torch.zeros(3, **i32)), "counts")):
        with pytest.raises(ValueError, match=word):
            L.lrmoe_balance_grad(z, idx, c, st, torch.zeros(4, 6), **more)
