"""How many launches a call of the sequence block's operators takes, where the cut of its work counts on it."""
import pytest
import torch

import block_ref as R
from test_gpu_block import attn_inputs, run_attn
from test_gpu_mixer import ROUND, near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hc():
    assert torch.cuda.is_available()
    from spatially_sharded_cnn_gb300 import build
    build.build()
    from spatially_sharded_cnn_gb300 import hc as mod
    return mod


@pytest.mark.parametrize("Dk,Dv,main", [(96, 128, 1), (40, 64, 1), (128, 72, 1), (56, 24, 1), (128, 128, 1), (64, 128, 2)])
def test_gradient_passes_of_one_kernel_are_one_launch(hc, Dk, Dv, main):
    """Segments are counted for three gradient passes at once where the head sizes need the same kernel, equal or not."""
    t, L, H = torch.bfloat16, 1300, 2
    a = attn_inputs(21, t, 1, L, H, Dk, Dv, 0, None, True, True)
    d = hc.linear_attn_desc(1, L, H, Dk, Dv, t)
    run = lambda: run_attn(hc, d, a, 1, L, H, Dk, Dv, t, 0, None)
    run()
    hc.hc_trace_collect()
    hc.check(hc.hc_trace_enable(True))
    try:
        o = run()
    finally:
        hc.check(hc.hc_trace_enable(False))
    torch.cuda.synchronize()
    st, table = hc.hc_trace_collect()
    hc.check(st)
    # one of the forward pass, and those of the backward pass
    assert table["attn_tc_kernel"][0] == 1 + main and table["attn_tc_carry_kernel"][0] == 1 + main, table
    ref = R.linear_attn(a["q"][1], a["k"][1], a["v"][1], H, d.scale, a["decay"][1], a["h0"][1], None, a["gy"][1], a["ghT"][1])
    for name, out in o.items():
        near(name, out, ref[name], 1e-5 + (ROUND[t] if out.t.dtype == t else 0.0))
