"""The forward operators without a GPU: the 64-bit forms that the GPU tests compare with are pinned
to worked examples, brute force and differences, and the entry points refuse what they cannot do."""
import ctypes

import numpy as np
import pytest
import torch

from pruned_expert_backward_lrmoe_b200 import build as B
from pruned_expert_backward_lrmoe_b200 import lrmoe as L
from tests import forward_ref as R

NULL, FAKE = ctypes.c_void_p(0), ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10004)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


# ---------------------------------------------------------------------------
# the 64-bit forms
# ---------------------------------------------------------------------------
def test_route_worked_example():
    z = np.log(np.array([[4.0, 1.0, 2.0, 1.0]]))          # softmax 1/2, 1/8, 1/4, 1/8
    idx, w, _ = R.route(z, 3, renorm=False)
    assert idx.tolist() == [[0, 2, 1]]                     # the tie 1, 3 goes to 1
    np.testing.assert_allclose(w, [[0.5, 0.25, 0.125]], rtol=1e-14)
    idx, w, _ = R.route(z, 2, renorm=True, scale=3.0)
    np.testing.assert_allclose(w, [[2.0, 1.0]], rtol=1e-14)
    # a bias moves the selection, not the weights: keys 0.5, 0.525, 0.25, 0.125
    idx, w, _ = R.route(z, 2, bias=np.array([0, 0.4, 0, 0]), renorm=False)
    assert idx.tolist() == [[1, 0]]
    np.testing.assert_allclose(w, [[0.125, 0.5]], rtol=1e-14)
    # groups {0,1}, {2,3} count 0.625 and 0.375; the second stays out
    idx, _, _ = R.route(z, 2, n_group=2, topk_group=1, renorm=False)
    assert idx.tolist() == [[0, 1]]


def test_route_masks():
    inf = np.inf
    idx, w, st = R.route(np.array([[-inf, 0.0, -inf], [-inf] * 3, [np.nan, 1.0, inf]]), 2)
    assert idx.tolist() == [[1, -1], [-1, -1], [1, -1]] and st == R.NONFINITE
    np.testing.assert_allclose(w, [[1, 0], [0, 0], [1, 0]])


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_grad_is_the_difference_of_the_weights(kind, renorm):
    rng = np.random.default_rng(0)
    T, E, k, h = 5, 7, 3, 1e-6
    z = rng.standard_normal((T, E))
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    idx[1, 2] = -1
    idx[2, 1] = idx[2, 0]                                  # the same expert twice
    idx[3] = -1
    dw = rng.standard_normal((T, k))
    got, _ = R.route_grad(z, idx, dw, kind, renorm, 2.5)
    for t in range(T):
        for e in range(E):
            zp, zm = z.copy(), z.copy()
            zp[t, e] += h
            zm[t, e] -= h
            d = ((R.weights(zp, idx, kind, renorm, 2.5) - R.weights(zm, idx, kind, renorm, 2.5))
                 * np.where(idx >= 0, dw, 0)).sum() / (2 * h)
            assert abs(d - got[t, e]) < 1e-7


def test_products_and_sums():
    rng = np.random.default_rng(1)
    off = np.array([1, 3, 3, 6])
    rows, W, b = rng.standard_normal((7, 4)), rng.standard_normal((3, 5, 4)), rng.standard_normal((3, 5))
    out, _ = R.product(rows, W, off, b)
    for r, e in ((1, 0), (2, 0), (3, 2), (5, 2)):
        for n in range(5):
            assert abs(out[r, n] - (sum(rows[r, i] * W[e, n, i] for i in range(4)) + b[e, n])) < 1e-12
    assert np.isnan(out[[0, 6]]).all()
    db, _ = R.bias_grad(rows, off, 3)
    np.testing.assert_allclose(db[0], rows[1] + rows[2])
    assert (db[1] == 0).all()
    y, idx = rng.standard_normal((4, 3)), np.array([[1, -1], [9, 0]], np.int32)
    Y, _ = R.combine(y, idx, np.array([[0.5, 9.0], [9.0, 2.0]]), 3, residual=np.ones((2, 3)))
    np.testing.assert_allclose(Y, [1 + 0.5 * y[0], 1 + 2 * y[3]])


# ---------------------------------------------------------------------------
# refusals of the C ABI
# ---------------------------------------------------------------------------
def refuse(f, args, at, value, code=L.LRMOE_ERR_INVALID_ARG):
    bad = list(args)
    bad[at] = value
    assert f(*bad) == code, (at, value)


ROUTE = [FAKE, 4, 16, 0, NULL, 4, 0, 4, 2, 1, 1.0, FAKE, FAKE, NULL, NULL]


@pytest.mark.parametrize("at,value,code", [
    (0, NULL, 1), (0, ODD, 1), (1, 0, 1), (2, 0, 1), (3, 7, 1), (4, ODD, 1), (5, 0, 1), (5, 17, 1), (5, 9, 1),
    (6, 2, 1), (7, 0, 1), (7, 3, 1), (8, 0, 1), (8, 5, 1), (10, float("inf"), 1), (10, float("nan"), 1),
    (11, NULL, 1), (12, ODD, 1), (2, 2048, 2)])
def test_route_refuses(lib, at, value, code):
    refuse(lib.lrmoe_route, ROUTE, at, value, code)


def test_route_refuses_wide_tops_and_many_groups(lib):
    a = list(ROUTE)
    a[2], a[5], a[7], a[8] = 64, 33, 1, 1
    assert lib.lrmoe_route(*a) == L.LRMOE_ERR_INVALID_ARG          # k > 32
    a[5], a[7], a[8] = 4, 64, 64
    assert lib.lrmoe_route(*a) == L.LRMOE_ERR_UNSUPPORTED          # 64 groups
    a[1], a[5], a[7], a[8] = 2 ** 30, 4, 1, 1
    assert lib.lrmoe_route(*a) == L.LRMOE_ERR_INVALID_ARG          # T*k past int32


ROUTE_GRAD = [FAKE, 4, 16, 0, FAKE, 4, 0, 1, 1.0, FAKE, ctypes.c_void_p(0x20000), NULL, NULL]


@pytest.mark.parametrize("at,value,code", [
    (0, NULL, 1), (1, 0, 1), (2, 2048, 2), (3, 2, 1), (4, NULL, 1), (5, 33, 1), (6, 5, 1), (8, float("nan"), 1),
    (9, ODD, 1), (10, NULL, 1), (10, FAKE, 1)])
def test_route_grad_refuses(lib, at, value, code):
    refuse(lib.lrmoe_route_grad, ROUTE_GRAD, at, value, code)


SWIGLU = [FAKE, 8, 2, FAKE, FAKE, 16, FAKE, NULL, 4, 64, 64, 1, FAKE, NULL, NULL, NULL, NULL, NULL]


@pytest.mark.parametrize("at,value,code", [
    (0, NULL, 1), (1, 0, 1), (2, 0, 1), (3, NULL, 1), (3, ODD, 1), (4, NULL, 1), (5, 0, 1), (6, ODD, 1),
    (7, ODD, 1), (8, 0, 1), (8, 1025, 2), (9, 60, 1), (10, 4, 1), (11, 3, 1), (12, NULL, 1), (13, ODD, 1),
    (14, ODD, 1), (15, ODD, 1), (2, 2 ** 29, 1)])
def test_swiglu_refuses(lib, at, value, code):
    refuse(lib.lrmoe_grouped_swiglu, SWIGLU, at, value, code)


def test_swiglu_without_perm_needs_all_rows(lib):
    a = list(SWIGLU)
    a[2], a[3] = 1, NULL
    assert lib.lrmoe_grouped_swiglu(*a) == L.LRMOE_ERR_INVALID_ARG  # 8 source rows, 16 packed ones


LINEAR = [FAKE, 16, FAKE, NULL, FAKE, 4, 64, 64, 1, NULL, FAKE, 20, ctypes.c_void_p(0x20000), NULL, NULL]


@pytest.mark.parametrize("at,value,code", [
    (0, NULL, 1), (1, 0, 1), (2, NULL, 1), (3, ODD, 1), (4, NULL, 1), (5, -1, 1), (5, 5000, 2), (6, 12, 1),
    (7, 0, 1), (8, 9, 1), (9, ODD, 1), (10, ODD, 1), (11, 0, 1), (12, NULL, 1), (12, FAKE, 1)])
def test_linear_refuses(lib, at, value, code):
    refuse(lib.lrmoe_grouped_linear, LINEAR, at, value, code)


def test_linear_without_perm_needs_all_rows(lib):
    a = list(LINEAR)
    a[10], a[11] = NULL, 15
    assert lib.lrmoe_grouped_linear(*a) == L.LRMOE_ERR_INVALID_ARG


@pytest.mark.parametrize("at,value,code", [
    (0, NULL, 1), (1, 0, 1), (2, ODD, 1), (3, 0, 1), (3, 1025, 2), (4, 12, 1), (5, 2, 1), (6, NULL, 1)])
def test_bias_grad_refuses(lib, at, value, code):
    refuse(lib.lrmoe_grouped_bias_grad, [FAKE, 16, FAKE, 4, 64, 1, FAKE, 0, NULL, NULL], at, value, code)


@pytest.mark.parametrize("at,value,code", [
    (0, NULL, 1), (1, ODD, 1), (2, NULL, 1), (3, 0, 1), (4, 33, 1), (5, 0, 1), (6, 4, 1), (7, 4, 1), (8, ODD, 1),
    (9, NULL, 1), (9, FAKE, 1)])
def test_combine_refuses(lib, at, value, code):
    refuse(lib.lrmoe_combine, [FAKE, FAKE, FAKE, 4, 2, 8, 64, 1, NULL, ctypes.c_void_p(0x20000), NULL, NULL],
           at, value, code)


# ---------------------------------------------------------------------------
# refusals of the binding: types, shapes and devices the C ABI cannot see
# ---------------------------------------------------------------------------
def test_binding_refuses_types_and_shapes(lib):
    z = torch.zeros(4, 16)
    i, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)

    def refused(what, f, *args, **kw):
        with pytest.raises(ValueError, match=what):
            f(*args, **kw)

    class Cuda(torch.Tensor):
        """A CPU tensor that says it is on cuda:0: no call gets past the checks with it."""

        def get_device(self):
            return 0

    c = lambda t: t.as_subclass(Cuda)  # noqa: E731
    z, i, w = c(z), c(i), c(w)
    refused("topk_idx", L.lrmoe_route, z, c(i.long()), w)
    refused("topk_w", L.lrmoe_route, z, i, c(w[:3]))
    refused("bias", L.lrmoe_route, z, i, w, bias=c(torch.zeros(15)))
    refused("status", L.lrmoe_route, z, i, w, status=c(torch.zeros(1)))
    refused("contiguous", L.lrmoe_route, c(torch.zeros(16, 4)).t(), i, w)
    refused("one device", L.lrmoe_route, torch.zeros(4, 16), i, w)
    refused("one device", L.lrmoe_route, z, i, torch.zeros(4, 2))
    refused("CUDA tensors", L.lrmoe_route, torch.zeros(4, 16), torch.zeros(4, 2, dtype=torch.int32),
            torch.zeros(4, 2))
    refused("dlogits", L.lrmoe_route_grad, z, i, w, c(z.bfloat16()))
    x, W, off = c(torch.zeros(4, 64)), c(torch.zeros(3, 32, 64)), c(torch.zeros(4, dtype=torch.int32))
    perm, new = c(torch.zeros(8, dtype=torch.int32)), lambda *s: c(torch.zeros(*s))
    refused("perm has 8 entries for 9", L.lrmoe_grouped_swiglu, x, W, off, new(9, 16), perm=perm, src_div=2)
    refused("perm: expected", L.lrmoe_grouped_swiglu, x, W, off, new(8, 16), perm=c(perm.long()), src_div=2)
    refused("u: expected", L.lrmoe_grouped_swiglu, x, W, off, new(8, 16), perm=perm, src_div=2, u=new(4, 16))
    refused("offsets", L.lrmoe_grouped_swiglu, x, W, c(off[:3]), new(8, 16), perm=perm, src_div=2)
    refused("W_gu", L.lrmoe_grouped_swiglu, x, new(3, 33, 64), off, new(8, 16), perm=perm, src_div=2)
    refused("residual", L.lrmoe_grouped_linear, x, W, off, new(4, 32), residual=new(4, 64))
    refused("W: expected", L.lrmoe_grouped_linear, x, c(W.bfloat16()), off, new(4, 32))
    refused("db", L.lrmoe_grouped_bias_grad, x, off, c(torch.zeros(3, 64, dtype=torch.float64)))
    refused("y: expected", L.lrmoe_combine, new(7, 64), i, w, 8, new(4, 64))


def test_binding_refuses_tensors_of_another_device(monkeypatch):
    class Far(torch.Tensor):
        def get_device(self):
            return 1

    far = torch.zeros(4, 2).as_subclass(Far)
    with pytest.raises(ValueError, match="one device"):
        L._arg("w", far, torch.float32, (4, 2), 0)
    assert L._arg("w", far, torch.float32, (4, 2), 1) == far.data_ptr()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="cuda:1"):
        L._launch(1, None)
