"""Host-side checks of the sequence block operators' entry points (no GPU needed): what they refuse,
before anything is launched, the sizes they ask for, and what the binding refuses."""
import ctypes as C

import pytest

from test_mixer_abi import rows
from test_mixer_sources import kernels


@pytest.fixture(scope="module")
def hc():
    from spatially_sharded_cnn_gb300 import build
    build.build()
    from spatially_sharded_cnn_gb300 import hc as mod
    return mod


def test_layernorm_refusals(hc):
    ok = dict(B=2, L=8, C=8, dtype=hc.HC_DTYPE_F32, eps=1e-5)
    INV, UNS = hc.HC_ERR_INVALID_ARG, hc.HC_ERR_UNSUPPORTED
    out = rows(hc, 8192)
    fwd = lambda d, x, y, g=4096, b=4096, mean=0, lens=0: hc._lib.hc_layernorm_fwd(C.byref(d), x, g, b, y, mean, 0, lens,
                                                                                 None)
    for bad in (dict(B=0), dict(L=-1), dict(C=0), dict(eps=-1.0), dict(eps=float("nan")), dict(dtype=3)):
        d = hc.layernorm_desc(**dict(ok, **bad))
        assert fwd(d, rows(hc), out) == INV, bad
        assert hc.hc_layernorm_workspace_size(d)[0] == INV, bad
    for bad in (dict(C=(1 << 20) + 1), dict(B=1 << 16, L=1 << 15)):
        d = hc.layernorm_desc(**dict(ok, **bad))
        assert fwd(d, rows(hc), out) == UNS and hc.hc_layernorm_workspace_size(d)[0] == UNS, bad
    d = hc.layernorm_desc(**ok)
    assert fwd(d, rows(hc, 0), out) == INV                    # absent
    assert fwd(d, rows(hc, 4098), out) == INV                 # not aligned to its elements
    assert fwd(d, rows(hc, dtype=1), out) == INV              # another element type
    assert fwd(d, rows(hc, row=-8), out) == INV
    assert fwd(d, rows(hc), rows(hc, 8192, row=7)) == INV     # output rows overlap
    assert fwd(d, rows(hc), rows(hc)) == INV                  # in place
    assert fwd(d, rows(hc), out, g=0) == INV and fwd(d, rows(hc), out, b=4100) == INV
    assert fwd(d, rows(hc), out, mean=4100) == INV and fwd(d, rows(hc), out, lens=4098) == INV
    st, nb = hc.hc_layernorm_workspace_size(d)
    assert st == 0 and nb > 0
    bwd = lambda gx, mean=4096, gg=4096, ws=4096, n=nb: hc._lib.hc_layernorm_bwd(
        C.byref(d), rows(hc), 4096, mean, 4096, rows(hc, 16384), gx, gg, 0, 0, ws, n, None)
    assert bwd(rows(hc)) == INV and bwd(rows(hc, 16384)) == INV and bwd(out, mean=0) == INV and bwd(out, gg=4100) == INV
    assert bwd(out, n=nb - 1) == hc.HC_ERR_WORKSPACE and bwd(out, ws=0) == hc.HC_ERR_WORKSPACE


def test_linear_attn_refusals(hc):
    ok = dict(B=2, L=8, H=2, Dk=4, Dv=4, dtype=hc.HC_DTYPE_F32, scale=0.5)
    INV, UNS = hc.HC_ERR_INVALID_ARG, hc.HC_ERR_UNSUPPORTED
    out = rows(hc, 8192)
    fwd = lambda d, q=rows(hc), k=rows(hc), v=rows(hc), y=out, a=0, h0=0, hT=0, lens=0, ws=4096, n=1 << 40: \
        hc._lib.hc_linear_attn_fwd(C.byref(d), q, k, v, a, y, h0, hT, lens, ws, n, None)
    for bad in (dict(B=0), dict(L=-1), dict(H=0), dict(Dk=0), dict(Dv=0), dict(dtype=5), dict(scale=float("nan")),
                dict(scale=float("inf"))):
        d = hc.linear_attn_desc(**dict(ok, **bad))
        assert fwd(d) == INV, bad
        assert hc.hc_linear_attn_workspace_size(d, 0)[0] == INV, bad
    for bad in (dict(Dk=129), dict(Dv=129), dict(L=0x7fffffff), dict(H=1 << 19, Dk=4), dict(B=1 << 30)):
        d = hc.linear_attn_desc(**dict(ok, **bad))
        assert hc.hc_linear_attn_workspace_size(d, 1)[0] == UNS, bad
        assert fwd(d) == UNS, bad
    d = hc.linear_attn_desc(**ok)
    assert hc.hc_linear_attn_workspace_size(d, 2)[0] == INV
    for k in ("q", "k", "v"):
        for bad in (rows(hc, 0), rows(hc, 4098), rows(hc, dtype=1), rows(hc, row=-8)):
            assert fwd(d, **{k: bad}) == INV, k
    assert fwd(d, y=rows(hc)) == INV and fwd(d, y=rows(hc, 8192, row=7)) == INV
    assert fwd(d, a=4100) == INV and fwd(d, h0=4104) == INV and fwd(d, hT=4104) == INV
    assert fwd(d, h0=4096, hT=4096) == INV and fwd(d, lens=4098) == INV
    long = hc.linear_attn_desc(**dict(ok, B=1, L=4096))
    hc.check(hc.hc_set_sm_count(152))
    try:
        st, nb = hc.hc_linear_attn_workspace_size(long, 1)
        assert st == 0 and nb > 0
        big = dict(q=rows(hc, batch=1 << 20), k=rows(hc, batch=1 << 20), v=rows(hc, batch=1 << 20))
        assert fwd(long, **big, ws=0) == hc.HC_ERR_WORKSPACE and fwd(long, **big, n=0) == hc.HC_ERR_WORKSPACE
    finally:
        hc.check(hc.hc_set_sm_count(0))

    def bwd(h0=0, ghT=0, gh0=0, **kw):
        g = dict(gq=rows(hc, 8192), gk=rows(hc, 16384), gv=rows(hc, 32768))
        g.update(kw)
        return hc._lib.hc_linear_attn_bwd(C.byref(d), rows(hc), rows(hc), rows(hc), 0, h0, rows(hc), ghT, g["gq"], g["gk"],
                                          g["gv"], gh0, 0, 0, 0, None)

    assert bwd(ghT=65536, gh0=65536) == INV and bwd(h0=65536, gh0=65536) == INV and bwd(gh0=65540) == INV
    for k in ("gq", "gk", "gv"):
        for bad in (rows(hc), rows(hc, 0), rows(hc, 8192 * 8, row=7)):  # over an input, absent, rows that overlap
            assert bwd(**{k: bad}) == INV, k
    assert bwd(gk=rows(hc, 8192)) == INV                      # two gradients in one place
    step = lambda y=out, state=4096, q=rows(hc): hc._lib.hc_linear_attn_step(C.byref(d), q, rows(hc), rows(hc), 0, state, y,
                                                                            None)
    assert step(y=rows(hc)) == INV and step(state=0) == INV and step(state=4100) == INV and step(q=rows(hc, 0)) == INV


def test_gated_ffn_refusals(hc):
    ok = dict(M=16, C=16, F=24, dtype=hc.HC_DTYPE_BF16, act=hc.HC_PW_SILU)
    INV, UNS = hc.HC_ERR_INVALID_ARG, hc.HC_ERR_UNSUPPORTED
    x, out = rows(hc, row=16, dtype=1), rows(hc, 8192, row=16, dtype=1)
    fwd = lambda d, x=x, y=out, wi=4096, wo=4096, ws=4096, n=1 << 40: hc._lib.hc_gated_ffn_fwd(C.byref(d), x, wi, wo, y, ws,
                                                                                             n, None)
    for bad in (dict(M=-1), dict(C=0), dict(F=0), dict(act=3), dict(act=-1), dict(dtype=7)):
        d = hc.gated_ffn_desc(**dict(ok, **bad))
        assert fwd(d) == INV and hc.hc_gated_ffn_workspace_size(d, 0)[0] == INV, bad
    for bad in (dict(C=12), dict(F=20), dict(C=1 << 17), dict(F=1 << 17), dict(M=0x7fffffff), dict(dtype=hc.HC_DTYPE_F32)):
        d = hc.gated_ffn_desc(**dict(ok, **bad))
        assert fwd(d) == UNS and hc.hc_gated_ffn_workspace_size(d, 1)[0] == UNS, bad
    d = hc.gated_ffn_desc(**ok)
    assert hc.hc_gated_ffn_workspace_size(d, 2)[0] == INV
    assert fwd(d, x=rows(hc, 0, row=16, dtype=1)) == INV and fwd(d, x=rows(hc, row=16, dtype=2)) == INV
    assert fwd(d, x=rows(hc, 4097, row=16, dtype=1)) == INV
    assert fwd(d, x=rows(hc, 4098, row=16, dtype=1)) == UNS and fwd(d, x=rows(hc, row=17, dtype=1)) == UNS
    assert fwd(d, x=rows(hc, row=0, dtype=1)) == UNS          # one row for all
    assert fwd(d, y=rows(hc, 8200, row=16, dtype=1)) == UNS and fwd(d, y=rows(hc, 8192, row=20, dtype=1)) == UNS
    assert fwd(d, y=rows(hc, 8192, row=8, dtype=1)) == INV and fwd(d, y=x) == INV
    assert fwd(d, wi=0) == INV and fwd(d, wo=4104) == INV
    st, nb = hc.hc_gated_ffn_workspace_size(d, 1)
    assert st == 0 and nb >= 16 * 24 * 2 * 3
    assert fwd(d, ws=0) == hc.HC_ERR_WORKSPACE and fwd(d, n=16 * 24 * 2 - 1) == hc.HC_ERR_WORKSPACE
    bwd = lambda gx, gw=0, n=nb: hc._lib.hc_gated_ffn_bwd(C.byref(d), x, 4096, 4096, rows(hc, 16384, row=16, dtype=1), gx,
                                                         gw, 0, 4096, n, None)
    assert bwd(x) == INV and bwd(rows(hc, 16384, row=16, dtype=1)) == INV and bwd(out, gw=4104) == INV
    assert bwd(rows(hc, 8192, row=17, dtype=1)) == UNS and bwd(out, n=nb - 1) == hc.HC_ERR_WORKSPACE
    assert hc.hc_gated_ffn_workspace_size(hc.gated_ffn_desc(**dict(ok, M=0)), 0) == (0, 0)
    # one row has no row stride
    one = hc.gated_ffn_desc(**dict(ok, M=1))
    assert fwd(one, x=rows(hc, row=1, dtype=1), y=rows(hc, 8192, row=3, dtype=1), ws=0) == hc.HC_ERR_WORKSPACE


def test_binding_checks(hc):
    import torch
    x = torch.zeros(2, 8, 8)
    with pytest.raises(hc.HcError):  # not on the device
        hc.hc_layernorm_fwd(hc.layernorm_desc(2, 8, 8, torch.float32), x, None, None, x)
    d = hc.linear_attn_desc(2, 8, 2, 4, 4, torch.float32)
    assert d.scale == 0.5
    with pytest.raises(hc.HcError):
        hc.hc_linear_attn_fwd(d, x, x, x, x)
    with pytest.raises(hc.HcError):
        hc.hc_gated_ffn_fwd(hc.gated_ffn_desc(16, 8, 8, torch.bfloat16), x[0], x, x, x[0])


@pytest.mark.parametrize("source", ["layernorm.cu", "attn.cu", "attn_fp32.cu", "attn_tc.cu", "ffn.cu"])
def test_reads_stay_behind_the_wait(source):
    """As test_mixer_sources.py, for the kernels of this set."""
    found = kernels(source)
    assert found
    for name, params, body in found:
        assert body.lstrip("{ \n").startswith("grid_begin();"), f"{name} acts before its wait"
        assert "__restrict__" not in params + body, f"{name} has a __restrict__ pointer"
        assert "__ldg" not in body and "global.nc" not in body, f"{name} reads through the read-only path"
