"""Child of test_forward_gpu.py: the forward operators on the checked-index library (LRMOE_CHECKED=1)."""
import torch

from pruned_expert_backward_lrmoe_b200 import lrmoe as L
from tests.test_forward_gpu import Layer, TOL

assert L.LIB_PATH.endswith("liblrmoe_checked.so")
for dt in ("bf16", "f32"):
    la = Layer(301, 8, 2, 136, 264, dt)
    la.out["status"].zero_()
    la.forward()
    la.backward()
    assert int(la.out["status"].item()) == 0
    got, ref = la.results(), la.reference()
    for n, r in ref.items():
        assert (got[n].double() - r).norm() <= TOL[dt] * (4 if n == "dz" else 1) * r.norm(), n

for dt in (torch.bfloat16, torch.float32):
    # views into larger buffers: even an unchecked read would stay in owned memory
    rows = torch.randn(4096, 64, device="cuda").to(dt)[:100]
    W = torch.randn(2, 64, 64, device="cuda").to(dt)
    big = torch.full((4096, 64), 7.0, device="cuda", dtype=dt)
    for off in ([0, 120, 90], [0, 60, 101], [-1, 60, 100]):
        off = torch.tensor(off, dtype=torch.int32, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        L.lrmoe_grouped_linear(rows, W, off, big[:100], status=st)
        assert int(st.item()) == L.ST_BAD_INDEX and bool((big == 7).all())
        st.zero_()
        L.lrmoe_grouped_swiglu(rows, W, off, big.view(-1, 32)[:100], status=st)
        assert int(st.item()) == L.ST_BAD_INDEX and bool((big == 7).all())
        st.zero_()
        db = torch.empty(2, 64, device="cuda")
        L.lrmoe_grouped_bias_grad(rows, off, db, status=st)
        assert int(st.item()) == L.ST_BAD_INDEX and bool(torch.isfinite(db).all())
print("ok")
