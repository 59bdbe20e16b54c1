"""Host-side checks of the channels-last mixer operators' entry points (no GPU needed): what they
refuse, before anything is launched, and the sizes they ask for."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def hc():
    from spatially_sharded_cnn_gb300 import build
    build.build()
    from spatially_sharded_cnn_gb300 import hc as mod
    return mod


def rows(hc, p=4096, batch=64, row=8, dtype=0):
    return hc._pack_rows(p, batch, row, dtype)


def test_groupnorm_refusals(hc):
    ok = dict(N=2, P=8, C=8, groups=2, dtype=hc.HC_DTYPE_F32, eps=1e-5, act=hc.HC_PW_SILU)
    INV = hc.HC_ERR_INVALID_ARG
    call = lambda d, x, y, g=4096, b=4096, ws=4096, nb=1 << 20: hc._lib.hc_groupnorm_fwd(C.byref(d), x, g, b, y, 0, 0, ws,
                                                                                      nb, None)
    for bad in (dict(N=0), dict(P=0), dict(C=0), dict(groups=0), dict(groups=3), dict(eps=-1.0), dict(act=7),
                dict(dtype=5), dict(eps=float("nan"))):
        d = hc.groupnorm_desc(**dict(ok, **bad))
        assert call(d, rows(hc), rows(hc, 8192)) == INV, bad
        assert hc.hc_groupnorm_workspace_size(d, 0)[0] == INV, bad
    d = hc.groupnorm_desc(**ok)
    st, nb = hc.hc_groupnorm_workspace_size(d, 1)
    assert st == 0 and nb > 0
    assert hc.hc_groupnorm_workspace_size(d, 2)[0] == INV
    out = rows(hc, 8192)
    assert call(d, rows(hc, 0), out) == INV                   # absent
    assert call(d, rows(hc, 4098), out) == INV                # not aligned to its elements
    assert call(d, rows(hc, dtype=1), out) == INV             # another element type
    assert call(d, rows(hc, row=-8), out) == INV
    assert call(d, rows(hc), rows(hc, 8192, row=7)) == INV    # output rows overlap
    assert call(d, rows(hc), rows(hc, 8192, batch=63)) == INV
    assert call(d, rows(hc), rows(hc)) == INV                 # in place
    assert call(d, rows(hc), out, g=0) == INV and call(d, rows(hc), out, b=4100) == INV
    assert call(d, rows(hc), out, ws=0) == hc.HC_ERR_WORKSPACE
    assert call(d, rows(hc), out, nb=hc.hc_groupnorm_workspace_size(d, 0)[1] - 1) == hc.HC_ERR_WORKSPACE
    bwd = lambda gx, mean=4096, ws=4096, n=nb: hc._lib.hc_groupnorm_bwd(C.byref(d), rows(hc), 4096, 4096, mean, 4096,
                                                                     rows(hc), gx, 0, 0, ws, n, None)
    assert bwd(rows(hc)) == INV and bwd(out, mean=0) == INV
    assert bwd(out, n=nb - 1) == hc.HC_ERR_WORKSPACE
    big = hc.groupnorm_desc(**dict(ok, N=70000))
    assert call(big, rows(hc), out) == hc.HC_ERR_UNSUPPORTED


def test_causal_conv_refusals(hc):
    ok = dict(B=2, L=8, D=8, K=4, dtype=hc.HC_DTYPE_F32, act=hc.HC_PW_SILU)
    INV = hc.HC_ERR_INVALID_ARG
    call = lambda d, x, y, w=4096, bias=0, si=0, so=0, lens=0: hc._lib.hc_causal_conv_fwd(C.byref(d), x, w, bias, y, si,
                                                                                       so, lens, None)
    out = rows(hc, 8192)
    for bad in (dict(B=0), dict(L=-1), dict(D=0), dict(K=0), dict(act=hc.HC_PW_GELU), dict(dtype=-1)):
        assert call(hc.causal_conv_desc(**dict(ok, **bad)), rows(hc), out) == INV, bad
    for bad in (dict(K=1), dict(K=9), dict(D=1 << 21)):
        d = hc.causal_conv_desc(**dict(ok, **bad))
        assert call(d, rows(hc), out) == hc.HC_ERR_UNSUPPORTED, bad
        assert hc.hc_causal_conv_workspace_size(d)[0] == hc.HC_ERR_UNSUPPORTED, bad
    d = hc.causal_conv_desc(**ok)
    assert call(d, rows(hc, 0), out) == INV and call(d, rows(hc), rows(hc)) == INV
    assert call(d, rows(hc), rows(hc, 8192, row=4)) == INV
    assert call(d, rows(hc), out, w=0) == INV and call(d, rows(hc), out, w=4100) == INV
    assert call(d, rows(hc), out, si=4104) == INV and call(d, rows(hc), out, si=4096, so=4096) == INV
    assert call(d, rows(hc), out, lens=4098) == INV
    st, nb = hc.hc_causal_conv_workspace_size(d)
    assert st == 0 and nb > 0
    bwd = lambda gx, gw=4096, ws=4096, n=nb: hc._lib.hc_causal_conv_bwd(C.byref(d), rows(hc), 4096, 0, rows(hc), gx, gw, 0,
                                                                     0, 0, 0, 0, ws, n, None)
    assert bwd(rows(hc)) == INV
    assert bwd(out, n=nb - 1) == hc.HC_ERR_WORKSPACE and bwd(out, ws=0) == hc.HC_ERR_WORKSPACE
    step = lambda y, state=4096: hc._lib.hc_causal_conv_step(C.byref(d), rows(hc), 4096, 0, state, y, None)
    assert step(rows(hc)) == INV and step(out, state=0) == INV and step(out, state=4100) == INV


def test_selective_scan_refusals(hc):
    ok = dict(B=2, L=8, D=8, d_state=4, dtype=hc.HC_DTYPE_F32, groups=2, softplus=1)
    INV = hc.HC_ERR_INVALID_ARG

    def inputs(A=4096, **kw):
        f = {k: (4096, 64, 8, 0) for k in ("u", "dt", "Bm", "Cm", "z")}
        f.update(kw)
        return hc._pack_scan_in(*(v for k in ("u", "dt", "Bm", "Cm", "z") for v in f[k]), A, 0, 0)

    out = rows(hc, 8192)
    fwd = lambda d, i, y=out, h0=0, hT=0, saved=0: hc._lib.hc_selective_scan_fwd(C.byref(d), i, h0, 0, y, hT, saved, 4096,
                                                                              1 << 30, None)
    for bad in (dict(B=0), dict(L=-1), dict(D=0), dict(groups=0), dict(groups=3), dict(d_state=0), dict(softplus=2),
                dict(dtype=3)):
        d = hc.selective_scan_desc(**dict(ok, **bad))
        assert fwd(d, inputs()) == INV, bad
        assert hc.hc_selective_scan_workspace_size(d, 0)[0] == INV and hc.hc_selective_scan_saved_size(d)[0] == INV
    big = hc.selective_scan_desc(**dict(ok, d_state=65))
    assert fwd(big, inputs()) == hc.HC_ERR_UNSUPPORTED
    assert hc.hc_selective_scan_workspace_size(big, 1)[0] == hc.HC_ERR_UNSUPPORTED
    d = hc.selective_scan_desc(**ok)
    none = (0, 0, 0, 0)
    for k in ("u", "dt", "Bm", "Cm"):
        assert fwd(d, inputs(**{k: none})) == INV, k
        assert fwd(d, inputs(**{k: (4096, 64, 8, 1)})) == INV, k
        assert fwd(d, inputs(**{k: (4097, 64, 8, 0)})) == INV, k
    assert fwd(d, inputs(z=(4097, 64, 8, 0))) == INV
    assert fwd(d, inputs(A=0)) == INV and fwd(d, inputs(A=4100)) == INV
    assert fwd(d, inputs(), y=rows(hc)) == INV                    # in place
    assert fwd(d, inputs(), y=rows(hc, 8192, row=7)) == INV
    assert fwd(d, inputs(), h0=4104) == INV and fwd(d, inputs(), h0=4096, hT=4096) == INV
    assert fwd(d, inputs(), saved=4104) == INV
    st, nb = hc.hc_selective_scan_workspace_size(d, 1)
    assert st == 0 and nb > 0 and hc.hc_selective_scan_workspace_size(d, 2)[0] == INV

    def bwd(saved=4096, gA=4096, n=nb, **kw):
        f = {k: (8192, 64, 8, 0) for k in ("u", "dt", "Bm", "Cm", "z")}
        f.update(kw)
        g = hc._pack_scan_grad(*(v for k in ("u", "dt", "Bm", "Cm", "z") for v in f[k]), gA, 0, 0, 0)
        return hc._lib.hc_selective_scan_bwd(C.byref(d), inputs(), 0, 0, saved, rows(hc), 0, g, 4096, n, None)

    assert bwd(saved=0) == INV and bwd(gA=0) == INV
    assert bwd(z=none) == INV                                     # a gate without its gradient
    assert bwd(u=(4096, 64, 8, 0)) == INV                         # over an input
    assert bwd(Bm=(8192, 64, 7, 0)) == INV                        # rows of 8 that overlap
    assert bwd(n=nb - 1) == hc.HC_ERR_WORKSPACE
    step = lambda y, state=4096: hc._lib.hc_selective_scan_step(C.byref(d), inputs(), state, y, None)
    assert step(rows(hc)) == INV and step(out, state=0) == INV and step(out, state=4100) == INV


def test_binding_checks_shapes_and_channels(hc):
    import torch
    d = hc.causal_conv_desc(B=2, L=8, D=8, K=4, dtype=torch.float32)
    x = torch.zeros(2, 8, 8)
    for bad in (torch.zeros(2, 8, 9), torch.zeros(2, 7, 8), x.transpose(1, 2)):
        with pytest.raises(hc.HcError):
            hc.hc_causal_conv_fwd(d, bad, x, None, x)
    assert hc._dtype(torch.float64) == -1
    assert hc._view(x.half(), 2, 8, 8)[3] == hc.HC_DTYPE_F16
    assert hc._view(x[:, 0], 2, 8) == (x.data_ptr(), 64, 0, hc.HC_DTYPE_F32)


def test_binding_checks_lengths(hc):
    import torch
    assert hc._lens(None) == 0
    ok = torch.tensor([1, 2], dtype=torch.int32)
    assert hc._lens(ok) == ok.data_ptr()
    for bad in (torch.tensor([1, 2]), torch.zeros(4, dtype=torch.int32)[::2]):
        with pytest.raises(hc.HcError):
            hc._lens(bad)
