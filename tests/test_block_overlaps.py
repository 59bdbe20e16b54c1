"""Outputs of the sequence block's operators that lie over what the same call reads or writes: refused before anything is
launched (no GPU needed).  Calls that are not refused here stop at a workspace that is not there."""
import ctypes as C

import pytest

from test_mixer_abi import rows


@pytest.fixture(scope="module")
def hc():
    from spatially_sharded_cnn_gb300 import build
    build.build()
    from spatially_sharded_cnn_gb300 import hc as mod
    return mod


M, CH, F = 16, 32, 24
X, GY, GX, WI, WO, GI, GO = (i << 20 for i in range(1, 8))
IN, OUT, ROWS = 2 * CH * F * 2, CH * F * 2, M * CH * 2  # bytes


@pytest.fixture
def backward(hc):
    d = hc.gated_ffn_desc(M, CH, F, hc.HC_DTYPE_BF16)

    def call(x=X, gy=GY, gx=GX, wi=WI, wo=WO, gi=GI, go=GO, row=CH, d=d):
        r = lambda p: rows(hc, p, row=row, dtype=1)
        return hc._lib.hc_gated_ffn_bwd(C.byref(d), r(x), wi, wo, r(gy), r(gx) if gx else None, gi, go, 0, 0, None)

    return call


def test_gated_ffn_gradients_over_inputs(hc, backward):
    INV, OK = hc.HC_ERR_INVALID_ARG, hc.HC_ERR_WORKSPACE
    assert backward() == OK and backward(gi=0, go=0) == OK and backward(gx=0) == OK
    assert backward(gi=WI) == INV and backward(go=WO) == INV         # a gradient in its weights' place
    assert backward(gi=WO) == INV and backward(go=WI) == INV         # in the other weights'
    assert backward(gi=GI, go=GI) == INV                             # two gradients in one place
    for at, n in ((X, ROWS), (GY, ROWS), (GX, ROWS), (WI, IN), (WO, OUT)):
        for name, own in (("gi", IN), ("go", OUT)):
            for p in (at, at + n - 16, at - own + 16):
                assert backward(**{name: p}) == INV, (name, p - at)
            for p in (at + n, at - own):                             # just behind it, just ahead of it
                assert backward(**{name: p}) == OK, (name, p - at)
    assert backward(gi=GI, go=GI + IN) == OK and backward(gi=GI, go=GI + IN - 16) == INV
    assert backward(gx=WI) == INV and backward(gx=WO + OUT - 16) == INV and backward(gx=WO + OUT) == OK
    # with no gradient of x its place is free
    assert backward(gx=0, gi=GX) == OK


def test_gated_ffn_gradients_between_rows(hc, backward):
    """Rows far apart leave room between them."""
    INV, OK = hc.HC_ERR_INVALID_ARG, hc.HC_ERR_WORKSPACE
    row = 4096
    far = dict(x=1 << 30, gy=2 << 30, gx=3 << 30, row=row)
    for k in ("x", "gy", "gx"):
        for r in (0, 5, M - 1):
            at = far[k] + 2 * row * r
            assert backward(**far, gi=at + 2 * CH) == OK and backward(**far, gi=at + 2 * CH - 16) == INV
            assert backward(**far, go=at - OUT) == OK and backward(**far, go=at - OUT + 16) == INV
        assert backward(**far, gi=far[k] + 2 * row * M) == OK
    one = hc.gated_ffn_desc(1, CH, F, hc.HC_DTYPE_BF16)  # one row has no stride
    assert backward(d=one, row=0, gi=X + 2 * CH) == OK and backward(d=one, row=0, gi=X) == INV


def test_gated_ffn_rows_over_weights(hc):
    d = hc.gated_ffn_desc(M, CH, F, hc.HC_DTYPE_BF16)
    fwd = lambda y: hc._lib.hc_gated_ffn_fwd(C.byref(d), rows(hc, X, row=CH, dtype=1), WI, WO, rows(hc, y, row=CH, dtype=1), 0, 0,
                                             None)
    for y in (WI, WO, WI + IN - 16, WO - ROWS + 16):
        assert fwd(y) == hc.HC_ERR_INVALID_ARG
    for y in (WI + IN, WO - ROWS, GX):
        assert fwd(y) == hc.HC_ERR_WORKSPACE


def test_layernorm_two_outputs_in_one_place(hc):
    INV = hc.HC_ERR_INVALID_ARG
    d = hc.layernorm_desc(2, 8, 8, hc.HC_DTYPE_F32)
    assert hc._lib.hc_layernorm_fwd(C.byref(d), rows(hc), 4096, 4096, rows(hc, 8192), 1 << 20, 1 << 20, 0, None) == INV
    bwd = lambda gg, gb: hc._lib.hc_layernorm_bwd(C.byref(d), rows(hc), 4096, 4096, 4096, rows(hc, 16384), rows(hc, 8192), gg, gb,
                                                 0, 0, 0, None)
    assert bwd(1 << 20, 1 << 20) == INV
    assert bwd(1 << 20, 2 << 20) == hc.HC_ERR_WORKSPACE and bwd(1 << 20, 0) == hc.HC_ERR_WORKSPACE
