"""The experts' forward products against the 64-bit forms: expert sizes around every tile edge
(empty experts, 1 to 5 rows, 31-33, 127-130, 255-257, 383-385), ragged K and N, gathered and packed
rows, every optional operand, rows that no call may read or write.

Tolerances.  A product of 16-bit operands is exact in fp32; K of them are summed in fp32, each step off
by at most one step of the partial sum (the tensor cores may truncate): below (K + 2) 2^-23 times the
sum of magnitudes, the bias and residual among them.  silu(g) u moves with g by at most 1.1 |u| and with u
by at most |silu(g)|; the fast exponential and the division are good to 2^-18 relative for the |g| < 64 of
these tests.  Each output is rounded once: half a step of its type.
"""
import numpy as np
import pytest
import torch

from pruned_expert_backward_lrmoe_b200 import lrmoe as L
from tests import forward_ref as R

pytestmark = pytest.mark.gpu

TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
SENTINEL = -77.0

SIZES = {
    "edges": [0, 1, 2, 3, 4, 5, 31, 32, 33, 0, 64, 127, 128, 129, 130, 255, 256, 257, 383, 384, 385, 0],
    "one": [1],
    "dense": [300],
    "small": [3, 0, 60, 7],
    "none": [0, 0, 0],
    # long experts, with and without a last tile of at most 128 rows, an empty one between
    "long": [700, 1029, 0, 2050, 257, 3841, 512, 1153, 640, 4100],
}


def normal(shape, dt, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(TYPE[dt])


def offsets_of(sizes, first=0):
    return np.concatenate([[first], first + np.cumsum(sizes)]).astype(np.int32)


def bound_product(K, mag, ref, dt):
    return (K + 2) * 2.0 ** -23 * mag + R.HALF[dt] * np.abs(ref)


def near(got, ref, tol, what):
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4])


def np64(t):
    return None if t is None else t.double().cpu().numpy()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("K,N", [(64, 256), (8, 8), (72, 136), (136, 264), (520, 120)])
@pytest.mark.parametrize("extras", ["plain", "all", "in place"])
def test_linear(sizes, K, N, extras, dt):
    sz = SIZES[sizes]
    E, M, first = len(sz), sum(sz), 2
    rows_cap, n_out = first + M + 6, first + M + 40
    off = offsets_of(sz, first)
    rows = normal((rows_cap, K), dt, 1)
    rows[:first] = float("nan")
    rows[first + M:] = float("nan")
    W = normal((E, N, K), dt, 2, 0.3)
    bias = res = perm = None
    out = torch.full((n_out, N), SENTINEL, dtype=TYPE[dt], device="cuda")
    dest = np.arange(rows_cap)
    if extras != "plain":
        bias = normal((E, N), dt, 3)
        dest = np.random.default_rng(M).permutation(n_out)[:rows_cap]
        perm = torch.from_numpy(dest.astype(np.int32)).cuda()
        res = normal((n_out, N), dt, 4)
        if extras == "in place":
            out.copy_(res)
    ref, mag = R.product(np64(rows), np64(W), off, np64(bias))
    before = np64(out)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.lrmoe_grouped_linear(rows, W, torch.from_numpy(off).cuda(), out, bias=bias,
                           residual=out if extras == "in place" else res, perm=perm, status=st)
    got = np64(out)
    live = slice(first, first + M)
    want, size = ref[live], mag[live]
    if res is not None:
        want = want + np64(res)[dest[live]]
        size = size + np.abs(np64(res)[dest[live]])
    near(got[dest[live]], want, bound_product(K, size, want, dt), "out")
    rest = np.setdiff1d(np.arange(n_out), dest[live])
    np.testing.assert_array_equal(got[rest], before[rest])
    assert int(st.item()) == 0


def swiglu_case(sz, H, I, dt, T=None, k=1, bias=False, seed=0):
    """Gathered rows: every pair of T tokens belongs to at most one expert."""
    E, M = len(sz), sum(sz)
    T = T or -(-M // k) + 3
    P = T * k
    rng = np.random.default_rng(seed + M)
    pairs = rng.permutation(P)[:M].astype(np.int32)
    x = normal((T, H), dt, seed + 1)
    W = normal((E, 2 * I, H), dt, seed + 2, 1.5 / H ** 0.5)
    b = normal((E, 2 * I), dt, seed + 3) if bias else None
    return P, pairs, x, W, b


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("H,I", [(64, 128), (8, 8), (72, 136), (200, 264), (520, 40)])
@pytest.mark.parametrize("k,bias,outputs", [(1, False, "gua"), (4, True, "gua"), (2, True, "g"), (3, False, "")])
def test_swiglu_gathered(sizes, H, I, k, bias, outputs, dt):
    sz = SIZES[sizes]
    P, pairs, x, W, b = swiglu_case(sz, H, I, dt, k=k, bias=bias)
    M, cap = sum(sz), sum(sz) + 5
    off = offsets_of(sz)
    perm = torch.full((cap,), 10 ** 8, dtype=torch.int32)     # entries past the last row are not used
    perm[:M] = torch.from_numpy(pairs)
    new = lambda n: torch.full((n, I), SENTINEL, dtype=TYPE[dt], device="cuda")  # noqa: E731
    Ap, outs = new(cap), {n: new(P) for n in outputs}
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.lrmoe_grouped_swiglu(x, W, torch.from_numpy(off).cuda(), Ap, perm=perm.cuda(), src_div=k, bias=b, status=st,
                           **outs)
    assert int(st.item()) == 0
    ref, mag = R.product(np64(x)[pairs // k], np64(W), off, np64(b))
    g, u, mg, mu = ref[:, :I], ref[:, I:], mag[:, :I], mag[:, I:]
    a = R.silu(g) * u
    step = (H + 2) * 2.0 ** -23
    tol_a = 1.1 * np.abs(u) * step * mg + np.abs(R.silu(g)) * step * mu + 2 * step ** 2 * mg * mu \
        + (2.0 ** -18 + R.HALF[dt]) * np.abs(a)
    if dt == "f32":
        assert np.abs(g).max(initial=0) < 64
    near(np64(Ap)[:M], a, tol_a, "Ap")
    assert (np64(Ap)[M:] == SENTINEL).all()
    rest = np.setdiff1d(np.arange(P), pairs)
    for n, t in outs.items():
        want, tol = {"g": (g, bound_product(H, mg, g, dt)), "u": (u, bound_product(H, mu, u, dt)),
                     "a": (a, tol_a)}[n]
        near(np64(t)[pairs], want, tol, n)
        assert (np64(t)[rest] == SENTINEL).all()


@pytest.mark.parametrize("I", [128, 136, 264, 392])
@pytest.mark.parametrize("H", [2048, 2056, 4104])
def test_swiglu_gathered_long_rows(H, I):
    """Long K (wide tiles): one, two and three column blocks."""
    test_swiglu_gathered("edges", H, I, 4, True, "gua", "bf16")


@pytest.mark.parametrize("H,I", [(64, 1160), (2048, 1160), (136, 2184)])
def test_swiglu_long_experts(H, I):
    test_swiglu_gathered("long", H, I, 4, True, "gua", "bf16")


@pytest.mark.parametrize("K,N", [(64, 2056), (136, 4104)])
@pytest.mark.parametrize("extras", ["plain", "all", "in place"])
def test_linear_long_experts(K, N, extras):
    test_linear("long", K, N, extras, "bf16")


@pytest.mark.parametrize("K,N", [(72, 2056), (520, 1032), (4, 4100)])
@pytest.mark.parametrize("extras", ["plain", "all", "in place"])
def test_linear_long_experts_f32(K, N, extras):
    """Wide tiles, several to a block."""
    test_linear("long", K, N, extras, "f32")


@pytest.mark.parametrize("H,I", [(68, 1160), (136, 2188)])
def test_swiglu_long_experts_f32(H, I):
    test_swiglu_gathered("long", H, I, 4, True, "gua", "f32")


@pytest.mark.parametrize("sizes", [[4096] * 4, [4097] * 4, [16500], [3, 20000, 5]])
def test_linear_with_uneven_last_tiles(sizes):
    """No last tile at all, one in every expert, one expert that holds nearly all rows."""
    SIZES["here"] = sizes
    test_linear("here", 72, 2056, "all", "bf16")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_swiglu_packed_rows_equal_gathered_ones(dt):
    sz, H, I, k = SIZES["edges"], 136, 72, 4
    P, pairs, x, W, b = swiglu_case(sz, H, I, dt, k=k, bias=True)
    off = torch.from_numpy(offsets_of(sz)).cuda()
    M = sum(sz)
    new = lambda n: torch.full((n, I), SENTINEL, dtype=TYPE[dt], device="cuda")  # noqa: E731
    p = torch.from_numpy(pairs).cuda()
    A1, G1 = new(M), new(P)
    L.lrmoe_grouped_swiglu(x, W, off, A1, perm=p, src_div=k, bias=b, g=G1)
    A2, G2 = new(M), new(M)
    L.lrmoe_grouped_swiglu(x[p.long() // k].contiguous(), W, off, A2, bias=b, g=G2)
    assert torch.equal(A1, A2) and torch.equal(G1[p.long()], G2)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("op", ["swiglu", "linear"])
def test_bad_perm_entries_are_flagged_and_skipped(op, dt):
    """A perm entry outside its range leaves that row's outputs alone; all other rows are unchanged."""
    sz, H, I = [5, 140, 300], 72, 136
    M, P = sum(sz), 500
    off = torch.from_numpy(offsets_of(sz)).cuda()
    pairs = torch.from_numpy(np.random.default_rng(1).permutation(P)[:M].astype(np.int32)).cuda()
    broken = pairs.clone()
    at = [0, 7, 144, 260, M - 1]
    broken[at] = torch.tensor([-1, P, 2 ** 31 - 1, -2 ** 31, P + 3], dtype=torch.int32, device="cuda")
    got = []
    for p in (pairs, broken):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        if op == "swiglu":
            x, W = normal((P, H), dt, 1), normal((3, 2 * I, H), dt, 2, 0.1)
            Ap = torch.full((M, I), SENTINEL, dtype=TYPE[dt], device="cuda")
            a = torch.full((P, I), SENTINEL, dtype=TYPE[dt], device="cuda")
            L.lrmoe_grouped_swiglu(x, W, off, Ap, perm=p, a=a, status=st)
            got.append((Ap, a, int(st.item())))
        else:
            rows, W = normal((M, H), dt, 1), normal((3, I, H), dt, 2, 0.1)
            a = torch.full((P, I), SENTINEL, dtype=TYPE[dt], device="cuda")
            L.lrmoe_grouped_linear(rows, W, off, a, perm=p, status=st)
            got.append((a, a, int(st.item())))
    (A1, a1, s1), (A2, a2, s2) = got
    assert s1 == 0 and s2 == R.BAD_INDEX
    gone = pairs[at].long()
    a1[gone] = SENTINEL
    assert torch.equal(a1, a2)
    if op == "swiglu":
        A1[at] = SENTINEL
        assert torch.equal(A1, A2)


def test_many_experts_and_repeat():
    """1024 experts, most of them empty or with one row; two runs give the same bits."""
    E, K, N = 1024, 64, 264
    rng = np.random.default_rng(0)
    sz = np.where(rng.random(E) < 0.3, rng.integers(1, 4, E), 0)
    sz[5], sz[1023] = 200, 130
    M, off = int(sz.sum()), offsets_of(sz)
    rows, W = normal((M, K), "bf16", 1), normal((E, N, K), "bf16", 2, 0.3)
    a = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    b = torch.empty_like(a)
    o = torch.from_numpy(off).cuda()
    L.lrmoe_grouped_linear(rows, W, o, a)
    L.lrmoe_grouped_linear(rows, W, o, b)
    assert torch.equal(a, b)
    ref, mag = R.product(np64(rows), np64(W), off)
    near(np64(a), ref, bound_product(K, mag, ref, "bf16"), "out")


def test_nan_rows_stay_in_their_rows():
    """NaN and infinities in one row, or in another expert's rows and weights, reach no other row."""
    sz, K, N = [40, 100, 130], 64, 128
    rows, W = normal((270, K), "bf16", 1), normal((3, N, K), "bf16", 2)
    off = torch.from_numpy(offsets_of(sz)).cuda()
    clean, dirty = (torch.empty(270, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    L.lrmoe_grouped_linear(rows, W, off, clean)
    rows[17], rows[60, 3], W[2] = float("nan"), float("inf"), float("nan")
    L.lrmoe_grouped_linear(rows, W, off, dirty)
    keep = torch.ones(270, dtype=torch.bool, device="cuda")
    keep[17] = keep[60] = False
    keep[140:] = False
    assert torch.equal(clean[keep], dirty[keep])
    assert bool(torch.isnan(dirty[17]).all()) and bool(torch.isnan(dirty[140:]).all())


def test_outputs_past_32_bits():
    """More than 2^31 output elements: the last rows land where they belong."""
    M, K, N = 1048583, 8, 2056
    rows = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    rows[-300:, 0] = torch.arange(1, 301, device="cuda").clamp(max=256).to(torch.bfloat16)
    W = torch.ones(1, N, K, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    L.lrmoe_grouped_linear(rows, W, off, out)
    assert torch.equal(out[-300:], rows[-300:, :1].expand(300, N))
    assert not bool(out[:-300].any())
