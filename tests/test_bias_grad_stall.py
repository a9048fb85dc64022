"""The bias gradient's way out of a wait that runs out: the status word says so, only copies that are in
flight are waited for, and the context stays usable."""
import ctypes

import pytest
import torch

from pruned_expert_backward_lrmoe_b200 import build as B
from pruned_expert_backward_lrmoe_b200 import lrmoe as L

NULL, FAKE, ODD = ctypes.c_void_p(0), ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10002)


def test_refusals():
    B.build()
    f = L.load().lrmoe_selftest_bias_grad_stall
    bad = L.LRMOE_ERR_INVALID_ARG
    assert f(FAKE, 8, FAKE, 2, 8, FAKE, 0, FAKE, NULL) == bad            # no limit
    assert f(FAKE, 8, FAKE, 2, 8, FAKE, 2_000_000, FAKE, NULL) == bad    # too long a one
    assert f(FAKE, 8, FAKE, 2, 8, FAKE, 100, NULL, NULL) == bad          # no status word
    assert f(FAKE, 8, FAKE, 2, 8, FAKE, 100, ODD, NULL) == bad
    assert f(FAKE, 8, FAKE, 2, 7, FAKE, 100, FAKE, NULL) == bad          # N % 8
    assert f(FAKE, 0, FAKE, 2, 8, FAKE, 100, FAKE, NULL) == bad
    assert f(FAKE, 8, FAKE, 0, 8, FAKE, 100, FAKE, NULL) == bad
    assert f(NULL, 8, FAKE, 2, 8, FAKE, 100, FAKE, NULL) == bad
    assert f(FAKE, 8, NULL, 2, 8, FAKE, 100, FAKE, NULL) == bad
    assert f(FAKE, 8, FAKE, 2, 8, NULL, 100, FAKE, NULL) == bad
    with pytest.raises(ValueError):
        L.lrmoe_selftest_bias_grad_stall(torch.zeros(8, 8), torch.zeros(3, dtype=torch.int32), torch.zeros(2, 8), 100,
                                         None)


# rows over clusters, one CTA to an expert and chunk (up to three turns of an SM), more boxes than slots
@pytest.mark.gpu
@pytest.mark.parametrize("E,N,m", [(2, 256, 2048), (40, 2048, 500), (1, 64, 60)])
def test_a_stalled_copy_times_out_without_further_waits(E, N, m):
    rows = torch.randn(E * m, N, generator=torch.Generator("cuda").manual_seed(1), device="cuda").bfloat16()
    off = torch.arange(0, E * m + 1, m, dtype=torch.int32, device="cuda")
    db, st = torch.empty(E, N, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    L.lrmoe_grouped_bias_grad(rows, off, db, status=st)
    want = db.clone()
    assert int(st.item()) == 0
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    L.lrmoe_selftest_bias_grad_stall(rows, off, db, 5000, st)            # 5 ms a wait
    b.record()
    torch.cuda.synchronize()
    assert int(st.item()) == L.ST_TIMEOUT
    assert 4 < a.elapsed_time(b) < 150                                   # a phase that cannot come would cost 200
    st.zero_()
    L.lrmoe_grouped_bias_grad(rows, off, db, status=st)
    assert int(st.item()) == 0 and torch.equal(db, want)
