"""What the mixer operators' entry points refuse, and what they take, at the edges (no GPU: errors come
before any launch)."""
import ctypes as C

import pytest

from test_mixer_abi import rows


@pytest.fixture(scope="module")
def hc():
    from spatially_sharded_cnn_gb300 import build
    build.build()
    from spatially_sharded_cnn_gb300 import hc as mod
    return mod


@pytest.mark.parametrize("state_in,gstate_out,gstate_in", [(0, 16384, 16384), (16384, 0, 16384), (16384, 32768, 32768)])
def test_conv_gradient_state_over_one_that_is_read(hc, state_in, gstate_out, gstate_in):
    """Runs of a sequence in other blocks read state_in and gstate_out while the first run writes gstate_in."""
    d = hc.causal_conv_desc(B=2, L=8, D=8, K=4, dtype=hc.HC_DTYPE_F32)
    # no workspace: a call that is not refused for its states ends before any launch all the same
    got = hc._lib.hc_causal_conv_bwd(C.byref(d), rows(hc), 4096, 0, rows(hc), rows(hc, 8192), 4096, 0, state_in, gstate_out,
                                     gstate_in, 0, 0, 0, None)
    assert got == hc.HC_ERR_INVALID_ARG
    ok = hc._lib.hc_causal_conv_bwd(C.byref(d), rows(hc), 4096, 0, rows(hc), rows(hc, 8192), 4096, 0, state_in, gstate_out,
                                    65536, 0, 0, 0, None)
    assert ok == hc.HC_ERR_WORKSPACE
