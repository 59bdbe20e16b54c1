"""GPU parity of the operators of a channels-last sequence block (layer norm, linear attention with a
decay for each head, gated feed-forward product: forward, backward, one token) with their 64-bit
formulas (block_ref.py), through the binding.

Tolerances, of the largest value of each output: 1e-5 for fp32 outputs, input gradients and states,
1e-4 for parameter gradients (the bars of the other kernels), and for elements stored in 16 bits half
a step more (2^-8 of the value for bf16, 2^-11 for fp16).  Operators that round something to 16 bits
inside (scores and states that are read, h and the gradients of a and u) get half a step of that type
more for each such rounding: the rounded values enter sums of products whose other factor is exact, so
that the sum is off by at most half a step of the sum of magnitudes, which for the inputs here (random
signs, n terms) is at most about sqrt(n) times their root mean square sum while the errors add up like
the terms themselves; the largest value of an output lies above its root mean square.  Held to 2 such
half steps in all (one inside at its worst case, one for the output)."""
import numpy as np
import pytest
import torch

import block_ref as R
from test_gpu_mixer import DT, ROUND, Data, Out, lens_of, near, space

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hc():
    assert torch.cuda.is_available()
    from spatially_sharded_cnn_gb300 import build
    build.build()
    from spatially_sharded_cnn_gb300 import hc as mod
    return mod


# ---------------------------------------------------------------- layer norm

LN = [(1, 1, 1, "f32", 0, False), (2, 3, 8, "f32", 0, False), (3, 7, 33, "bf16", 0, True), (2, 50, 64, "bf16", 0, False),
      (5, 19, 100, "f16", 4, True), (2, 31, 128, "f32", 0, False), (4, 9, 250, "f16", 0, False), (1, 300, 256, "bf16", 8, False),
      (5, 40, 330, "f32", 2, True), (3, 21, 512, "bf16", 0, True), (2, 11, 1000, "f32", 0, False), (1, 17, 1025, "bf16", 7, False),
      (2, 5, 2048, "f16", 0, True), (1, 9, 4100, "f32", 0, False), (1, 6, 9000, "bf16", 0, False), (1, 3, 20001, "f32", 0, False),
      (1, 4, 40000, "f16", 0, False), (700, 5, 48, "bf16", 0, True),
      (40, 60, 96, "bf16", 0, False), (4, 50, 768, "bf16", 0, False), (3, 40, 1024, "f16", 0, False),
      (2, 700, 1536, "bf16", 0, False), (2, 9, 3000, "bf16", 0, True), (6, 33, 330, "bf16", 0, False),
      (2, 20, 333, "f16", 1, False), (900, 3, 20, "f16", 0, False), (2, 11, 1389, "bf16", 0, False)]


@pytest.mark.parametrize("B,L,C,dt,wide,ragged", LN)
def test_layernorm(hc, B, L, C, dt, wide, ragged):
    t = DT[dt]
    lens, lens_t = lens_of(ragged, B, L)
    s = Data(1, t, wide, lens)
    x, xr = s.rows(B, L, C, 1.5, 0.7)
    gy, gyr = s.rows(B, L, C)
    gamma, gr = s.param(C, scale=0.2, shift=1.0)
    beta, br = s.param(C, scale=0.2)
    ref = R.layernorm(xr, gr, br, 1e-5, lens, gyr)
    d = hc.layernorm_desc(B, L, C, t)
    y, mean, rstd, gx = Out((B, L, C), t, wide), Out((B, L)), Out((B, L)), Out((B, L, C), t, wide)
    gg, gb = Out((C,)), Out((C,))
    hc.check(hc.hc_layernorm_fwd(d, x, gamma, beta, y.t, mean.t, rstd.t, lens=lens_t))
    ws, nb = space(hc, hc.hc_layernorm_workspace_size(d))
    hc.check(hc.hc_layernorm_bwd(d, x, gamma, mean.t, rstd.t, gy, gx.t, gg.t, gb.t, lens=lens_t, ws=ws, ws_bytes=nb))
    for name, o, bar in (("y", y, 1e-5), ("mean", mean, 1e-5), ("rstd", rstd, 1e-5), ("gx", gx, 1e-5)):
        near(name, o, ref[name], bar)
    if C > 1:
        near("ggamma", gg, ref["ggamma"], 1e-4)
    near("gbeta", gb, ref["gbeta"], 1e-4)
    # without statistics, and without the parameters' gradients
    y2, gx2 = Out((B, L, C), t), Out((B, L, C), t)
    hc.check(hc.hc_layernorm_fwd(d, x, gamma, beta, y2.t, lens=lens_t))
    hc.check(hc.hc_layernorm_bwd(d, x, gamma, mean.t, rstd.t, gy, gx2.t, lens=lens_t))
    assert torch.equal(y2.t, y.t) and torch.equal(gx2.t, gx.t)


def test_layernorm_of_no_rows(hc):
    d = hc.layernorm_desc(3, 0, 8, torch.float32)
    x, g = torch.empty(3, 0, 8, device="cuda"), torch.ones(8, device="cuda")
    gg, gb = Out((8,)), Out((8,))
    hc.check(hc.hc_layernorm_fwd(d, x, g, g, x))
    hc.check(hc.hc_layernorm_bwd(d, x, g, None, None, x, x, gg.t, gb.t))
    assert (gg.numpy() == 0).all() and (gb.numpy() == 0).all()


def test_layernorm_far_offset(hc):
    """An offset of 4096 standard deviations: the deviations are taken from the mean, not from sums of squares."""
    r = np.random.default_rng(3)
    x = torch.from_numpy(r.normal(size=(1, 64, 512)) + 4096).float().cuda()
    g, b = torch.ones(512, device="cuda"), torch.zeros(512, device="cuda")
    y = Out((1, 64, 512))
    hc.check(hc.hc_layernorm_fwd(hc.layernorm_desc(1, 64, 512, torch.float32), x, g, b, y.t))
    ref = R.layernorm(x.double().cpu().numpy(), np.ones(512), np.zeros(512), 1e-5)["y"]
    # the mean is rounded once at 4096 (half a step: 2.4e-4 of a standard deviation) and its sum carries a few more
    near("y", y, ref, 1e-3)


# ---------------------------------------------------------------- linear attention

AT = [(1, 1, 1, 1, 1, "f32", 0, False, True, True), (2, 5, 2, 3, 7, "f32", 0, True, True, True),
      (5, 33, 3, 41, 82, "f32", 2, True, True, True), (2, 64, 2, 64, 64, "f32", 0, False, False, True),
      (1, 700, 2, 32, 96, "f32", 4, False, True, True), (3, 257, 1, 128, 128, "f32", 0, True, True, False),
      (2, 100, 2, 16, 16, "bf16", 0, False, True, True), (5, 130, 2, 64, 64, "bf16", 8, True, True, True),
      (1, 129, 1, 64, 64, "bf16", 0, False, False, False), (2, 300, 3, 40, 80, "bf16", 0, False, True, True),
      (2, 1000, 1, 128, 128, "bf16", 8, False, True, True), (5, 515, 2, 128, 64, "bf16", 0, True, True, True),
      (1, 2500, 1, 64, 128, "bf16", 0, False, True, True), (2, 400, 2, 96, 24, "bf16", 3, True, True, True),
      (5, 9, 2, 64, 64, "bf16", 0, True, True, True), (2, 1, 1, 128, 128, "bf16", 0, False, True, True),
      (5, 3, 2, 72, 16, "bf16", 8, True, True, True), (1, 10, 1, 64, 8, "bf16", 0, False, False, True),
      (5, 300, 2, 64, 64, "f16", 0, True, True, True), (2, 200, 1, 128, 120, "f16", 0, False, True, True),
      (1, 77, 3, 31, 9, "f16", 0, False, False, True),
      (5, 400, 2, 41, 82, "f32", 0, True, True, True), (1, 900, 1, 128, 40, "f16", 0, False, True, True),
      (2, 610, 1, 30, 100, "f32", 0, True, True, True)]


def attn_inputs(seed, t, B, L, H, Dk, Dv, wide, lens, state, decays):
    s = Data(seed, t, wide, lens)
    a = dict(q=s.rows(B, L, H * Dk), k=s.rows(B, L, H * Dk), v=s.rows(B, L, H * Dv), gy=s.rows(B, L, H * Dv))
    a["h0"] = s.param(B, H, Dk, Dv, scale=2.0) if state else (None, None)
    a["ghT"] = s.param(B, H, Dk, Dv) if state else (None, None)
    # heads that remember about 100 rows, 3, a few thousand and nothing
    values = np.array([(-0.01, -0.3, -0.0004, -40.0)[h % 4] for h in range(H)])
    a["decay"] = s.param(H, value=values) if decays else (None, None)
    return a


def run_attn(hc, d, a, B, L, H, Dk, Dv, t, wide, lens_t, stream=None):
    st = a["h0"][0] is not None
    o = dict(y=Out((B, L, H * Dv), t, wide), state=Out((B, H, Dk, Dv)), gq=Out((B, L, H * Dk), t, wide),
             gk=Out((B, L, H * Dk), t, wide), gv=Out((B, L, H * Dv), t, wide))
    if st:
        o["gstate"] = Out((B, H, Dk, Dv))
    ws, nb = space(hc, hc.hc_linear_attn_workspace_size(d, 0))
    hc.check(hc.hc_linear_attn_fwd(d, a["q"][0], a["k"][0], a["v"][0], o["y"].t, a["decay"][0], a["h0"][0], o["state"].t,
                                   lens_t, ws, nb, stream))
    ws, nb = space(hc, hc.hc_linear_attn_workspace_size(d, 1))
    hc.check(hc.hc_linear_attn_bwd(d, a["q"][0], a["k"][0], a["v"][0], a["gy"][0], o["gq"].t, o["gk"].t, o["gv"].t,
                                   a["decay"][0], a["h0"][0], a["ghT"][0], o["gstate"].t if st else None, lens_t, ws, nb,
                                   stream))
    return o


@pytest.mark.parametrize("B,L,H,Dk,Dv,dt,wide,ragged,state,decays", AT)
def test_linear_attn(hc, B, L, H, Dk, Dv, dt, wide, ragged, state, decays):
    t = DT[dt]
    lens, lens_t = lens_of(ragged, B, L)
    a = attn_inputs(2, t, B, L, H, Dk, Dv, wide, lens, state, decays)
    d = hc.linear_attn_desc(B, L, H, Dk, Dv, t, scale=0.5 * Dk ** -0.5)
    o = run_attn(hc, d, a, B, L, H, Dk, Dv, t, wide, lens_t)
    ref = R.linear_attn(a["q"][1], a["k"][1], a["v"][1], H, d.scale, a["decay"][1], a["h0"][1], lens, a["gy"][1], a["ghT"][1])
    assert hc.hc_sync_check(None) == hc.HC_OK
    for name, out in o.items():
        near(name, out, ref[name], 1e-5 + (ROUND[t] if out.t.dtype == t and t != torch.float32 else 0.0))


def test_linear_attn_forgets_all(hc):
    """A log decay of minus infinity: y_t = scale (q_t . k_t) v_t, and states end at the last row's product."""
    t = torch.float32
    a = attn_inputs(4, t, 2, 40, 2, 8, 8, 0, None, True, True)
    a["decay"] = (torch.tensor([-float("inf"), -0.1], device="cuda"), np.array([-np.inf, float(np.float32(-0.1))]))
    d = hc.linear_attn_desc(2, 40, 2, 8, 8, t)
    o = run_attn(hc, d, a, 2, 40, 2, 8, 8, t, 0, None)
    ref = R.linear_attn(a["q"][1], a["k"][1], a["v"][1], 2, d.scale, a["decay"][1], a["h0"][1], None, a["gy"][1], a["ghT"][1])
    for name, out in o.items():
        near(name, out, ref[name], 1e-5)


def test_linear_attn_of_no_rows(hc):
    d = hc.linear_attn_desc(2, 0, 3, 4, 5, torch.float32)
    q, v = torch.empty(2, 0, 12, device="cuda"), torch.empty(2, 0, 15, device="cuda")
    h0, gh = torch.randn(2, 3, 4, 5, device="cuda"), torch.randn(2, 3, 4, 5, device="cuda")
    hT, g0 = Out((2, 3, 4, 5)), Out((2, 3, 4, 5))
    hc.check(hc.hc_linear_attn_fwd(d, q, q, v, torch.empty_like(v), h0=h0, hT=hT.t))
    e = lambda x: torch.empty_like(x)
    hc.check(hc.hc_linear_attn_bwd(d, q, q, v, v, e(q), e(q), e(v), h0=h0, ghT=gh, gh0=g0.t))
    assert torch.equal(hT.t, h0) and torch.equal(g0.t, gh)
    hc.check(hc.hc_linear_attn_fwd(d, q, q, v, torch.empty_like(v), hT=hT.t))
    assert (hT.numpy() == 0).all()


@pytest.mark.parametrize("D", [64, 128])
def test_linear_attn_of_no_rows_bf16(hc, D):
    """Sizes that tensor cores take when there are rows."""
    d = hc.linear_attn_desc(2, 0, 1, D, D, torch.bfloat16)
    q = torch.empty(2, 0, D, device="cuda", dtype=torch.bfloat16)
    h0, gh = torch.randn(2, 1, D, D, device="cuda"), torch.randn(2, 1, D, D, device="cuda")
    hT, g0 = Out((2, 1, D, D)), Out((2, 1, D, D))
    e = lambda: torch.empty_like(q)
    hc.check(hc.hc_linear_attn_fwd(d, q, q, q, e(), h0=h0, hT=hT.t))
    hc.check(hc.hc_linear_attn_bwd(d, q, q, q, q, e(), e(), e(), h0=h0, ghT=gh, gh0=g0.t))
    assert torch.equal(hT.t, h0) and torch.equal(g0.t, gh)


@pytest.mark.parametrize("B,H,Dk,Dv,dt,wide", [(1, 1, 1, 1, "f32", 0), (3, 2, 41, 82, "f32", 3), (64, 4, 64, 64, "bf16", 8),
                                               (5, 3, 128, 128, "f16", 0), (2, 5, 16, 100, "bf16", 1)])
def test_linear_attn_step(hc, B, H, Dk, Dv, dt, wide):
    """Single tokens one after another give the rows that the sequence gives."""
    t, L = DT[dt], 4
    a = attn_inputs(5, t, B, L, H, Dk, Dv, wide, None, True, True)
    d = hc.linear_attn_desc(B, 1, H, Dk, Dv, t)
    ref = R.linear_attn(a["q"][1], a["k"][1], a["v"][1], H, d.scale, a["decay"][1], a["h0"][1])
    state = a["h0"][0].clone()
    for i in range(L):
        y = Out((B, H * Dv), t, wide)
        hc.check(hc.hc_linear_attn_step(d, a["q"][0][:, i], a["k"][0][:, i], a["v"][0][:, i], state, y.t, a["decay"][0]))
        near(f"y {i}", y, ref["y"][:, i], 1e-5)
    near("state", state, ref["state"], 1e-5)


# ---------------------------------------------------------------- gated feed-forward

FF = [(1, 8, 8, "bf16", "none", 0), (3, 64, 64, "bf16", "silu", 0), (64, 128, 256, "bf16", "silu", 8), (129, 72, 200, "f16", "gelu", 0),
      (300, 328, 872, "f16", "gelu", 16), (1000, 256, 128, "bf16", "gelu", 0), (2000, 136, 264, "bf16", "silu", 0),
      (5, 1024, 2816, "bf16", "silu", 0), (3000, 64, 40, "f16", "none", 0), (257, 512, 1408, "bf16", "silu", 0)]


@pytest.mark.parametrize("M,C,F,dt,kind,wide", FF)
def test_gated_ffn(hc, M, C, F, dt, kind, wide):
    t = DT[dt]
    s = Data(6, t, wide)
    x, xr = (v[0] for v in s.rows(1, M, C))
    gy, gyr = (v[0] for v in s.rows(1, M, C))
    s.wide = 0
    w_in, wir = (v[0] for v in s.rows(1, C, 2 * F, C ** -0.5))
    w_out, wor = (v[0] for v in s.rows(1, F, C, F ** -0.5))
    act = {"none": hc.HC_PW_NONE, "silu": hc.HC_PW_SILU, "gelu": hc.HC_PW_GELU}[kind]
    d = hc.gated_ffn_desc(M, C, F, t, act)
    y, gx, gwi, gwo = Out((M, C), t, wide), Out((M, C), t, wide), Out((C, 2 * F), t), Out((F, C), t)
    ws, nb = space(hc, hc.hc_gated_ffn_workspace_size(d, 0))
    hc.check(hc.hc_gated_ffn_fwd(d, x, w_in, w_out, y.t, ws, nb))
    ws, nb = space(hc, hc.hc_gated_ffn_workspace_size(d, 1))
    hc.check(hc.hc_gated_ffn_bwd(d, x, w_in, w_out, gy, gx.t, gwi.t, gwo.t, ws, nb))
    ref = R.gated_ffn(xr, wir, wor, kind, gyr)
    assert hc.hc_sync_check(None) == hc.HC_OK
    for name, out in (("y", y), ("gx", gx), ("gw_in", gwi), ("gw_out", gwo)):
        near(name, out, ref[name], 1e-5 + ROUND[t])


def test_gated_ffn_of_no_rows(hc):
    d = hc.gated_ffn_desc(0, 16, 24, torch.bfloat16)
    x = torch.empty(0, 16, device="cuda", dtype=torch.bfloat16)
    w_in, w_out = (torch.ones(*s, device="cuda", dtype=torch.bfloat16) for s in ((16, 48), (24, 16)))
    gwi, gwo = Out((16, 48), torch.bfloat16), Out((24, 16), torch.bfloat16)
    hc.check(hc.hc_gated_ffn_fwd(d, x, w_in, w_out, torch.empty_like(x)))
    ws, nb = space(hc, hc.hc_gated_ffn_workspace_size(d, 1))
    hc.check(hc.hc_gated_ffn_bwd(d, x, w_in, w_out, torch.empty_like(x), torch.empty_like(x), gwi.t, gwo.t, ws, nb))
    assert (gwi.numpy() == 0).all() and (gwo.numpy() == 0).all()
