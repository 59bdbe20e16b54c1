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


def test_scan_takes_as_many_sequences_as_a_map_has_pixels(hc):
    """128 x 1024 pixels are 131072 sequences; the limit is that of channels over all sequences, 2^31."""
    F = hc.HC_DTYPE_BF16
    for d in (hc.selective_scan_desc(131072, 16, 512, 16, F), hc.selective_scan_desc(1 << 30, 1, 1, 16, F)):
        assert hc.hc_selective_scan_workspace_size(d, 0) == (0, 0)  # uncut: nothing to join
        st, nb = hc.hc_selective_scan_workspace_size(d, 1)
        assert st == 0 and nb >= 4 * d.B * d.D * (d.d_state + 2)
        assert hc.hc_selective_scan_saved_size(d)[0] == 0
    for bad in (hc.selective_scan_desc(1 << 22, 16, 512, 16, F), hc.selective_scan_desc(1 << 30, 1, 2, 16, F),
                hc.selective_scan_desc(1, 16, 1 << 21, 16, F), hc.selective_scan_desc(1, 0x7fffffff, 1, 16, F)):
        assert hc.hc_selective_scan_workspace_size(bad, 0)[0] == hc.HC_ERR_UNSUPPORTED


def test_many_sequences_stay_uncut_under_any_sm_count(hc):
    """Segments are joined with a grid of 65535 sequences at most."""
    hc.check(hc.hc_set_sm_count(1 << 20))
    try:
        few = hc.selective_scan_desc(65535, 400, 4, 16, hc.HC_DTYPE_F32)
        many = hc.selective_scan_desc(65536, 400, 4, 16, hc.HC_DTYPE_F32)
        assert hc.hc_selective_scan_workspace_size(few, 0)[1] > 0
        assert hc.hc_selective_scan_workspace_size(many, 0) == (0, 0)
    finally:
        hc.check(hc.hc_set_sm_count(0))
