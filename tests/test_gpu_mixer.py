"""GPU parity of the channels-last mixer operators (group norm with an activation, short causal
convolution, selective state-space scan: forward, backward, one token) with their 64-bit formulas
(mixer_ref.py), through the binding.

Tolerances, of the largest value of each output: 1e-5 for outputs, input gradients and states, 1e-4
for parameter gradients (the bars of the other kernels), and for elements stored in 16 bits half a
unit in the last place more (2^-8 for bf16, 2^-11 for fp16) -- the inputs are rounded to the type
before the reference reads them, and each output is rounded once."""
import numpy as np
import pytest
import torch

import mixer_ref as M

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ROUND = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
PAD = 64


@pytest.fixture(scope="module")
def hc():
    assert torch.cuda.is_available()
    from spatially_sharded_cnn_gb300 import build
    build.build()
    from spatially_sharded_cnn_gb300 import hc as mod
    return mod


class Out:
    """An output: NaN-filled, guard elements on both sides; `wide` adds columns to each row that must stay as they are."""

    def __init__(self, shape, dtype=torch.float32, wide=0):
        self.shape, self.wide = tuple(shape), wide
        n = int(np.prod(self.shape[:-1])) * (self.shape[-1] + wide)
        self.buf = torch.full((n + 2 * PAD,), 7.0, dtype=dtype, device="cuda")
        rows = self.buf[PAD:PAD + n].view(self.shape[:-1] + (self.shape[-1] + wide,))
        self.t = rows[..., :self.shape[-1]]
        self.t.fill_(float("nan"))
        self.rest = rows[..., self.shape[-1]:]

    def numpy(self):
        torch.cuda.synchronize()
        assert (self.buf[:PAD] == 7).all() and (self.buf[-PAD:] == 7).all() and (self.rest == 7).all(), \
            "written outside the output"
        return self.t.double().cpu().numpy()


def near(name, out, ref, bar):
    got = out.numpy() if isinstance(out, Out) else out.double().cpu().numpy()
    r = ROUND[out.t.dtype if isinstance(out, Out) else out.dtype]
    assert got.shape == ref.shape, name
    assert np.isfinite(got).all(), f"{name}: not finite"
    top = np.abs(ref).max() if ref.size else 0.0
    err = np.abs(got - ref).max() if ref.size else 0.0
    assert err <= (bar + r) * top, f"{name}: {err / top if top else err:.2e} of the largest value, {bar + r:.2e} allowed"


class Data:
    """Seeded inputs: device tensors of the type (rows `wide` elements longer than their channels) and the same values in
    64 bits.  Rows past a sequence's length hold NaN and infinities on the device."""

    def __init__(self, seed, dtype, wide=0, lens=None):
        self.r, self.dtype, self.wide, self.lens = np.random.default_rng(seed), dtype, wide, lens

    def rows(self, b, l, c, scale=1.0, shift=0.0):
        v = torch.from_numpy(self.r.normal(size=(b, l, c)) * scale + shift).to(self.dtype).cuda()
        ref = v.double().cpu().numpy()
        buf = torch.full((b, l, c + self.wide), 3.0, dtype=self.dtype, device="cuda")
        buf[..., :c] = v
        if self.lens is not None:
            for i, n in enumerate(self.lens):
                buf[i, n:] = float("nan")
                buf[i, n + 1:] = float("inf")
        return buf[..., :c], ref

    def param(self, *shape, scale=1.0, shift=0.0, value=None):
        v = torch.from_numpy((self.r.normal(size=shape) * scale + shift) if value is None else value).float().cuda()
        return v, v.double().cpu().numpy()


def lens_of(ragged, b, l):
    if not ragged:
        return None, None
    v = [(l, 0, min(1, l), l // 2, max(l - 1, 0))[i % 5] for i in range(b)]
    return v, torch.tensor(v, dtype=torch.int32, device="cuda")


def space(hc, got):
    hc.check(got[0])
    return torch.full((max(got[1], 16),), 0xFF, dtype=torch.uint8, device="cuda"), got[1]  # NaNs in every float


# ---------------------------------------------------------------- group norm

GN = [(1, 1, 1, 1, "f32", "none", 0), (2, 1, 8, 8, "f32", "silu", 0), (2, 37, 24, 3, "f32", "gelu", 0),
      (3, 100, 256, 32, "bf16", "silu", 0), (1, 1000, 40, 5, "f16", "gelu", 0), (2, 257, 120, 24, "bf16", "none", 3),
      (2, 65, 64, 4, "f32", "silu", 5), (1, 50, 1100, 1, "f32", "silu", 0), (1, 33, 2056, 257, "bf16", "silu", 8),
      (5, 2000, 16, 2, "f16", "silu", 0), (40, 19, 32, 32, "f32", "silu", 4)]


@pytest.mark.parametrize("N,P,C,G,dt,kind,wide", GN)
def test_groupnorm(hc, N, P, C, G, dt, kind, wide):
    t = DT[dt]
    s = Data(1, t, wide)
    x, xr = s.rows(N, P, C, 1.5, 0.7)
    gy, gyr = s.rows(N, P, C)
    gamma, gr = s.param(C, scale=0.2, shift=1.0)
    beta, br = s.param(C, scale=0.2)
    act = dict(none=hc.HC_PW_NONE, silu=hc.HC_PW_SILU, gelu=hc.HC_PW_GELU)[kind]
    d = hc.groupnorm_desc(N, P, C, G, t, 1e-5, act)
    ref = M.groupnorm(xr, gr, br, G, 1e-5, kind, gyr)
    ws, nb = space(hc, hc.hc_groupnorm_workspace_size(d, 1))
    y, mean, rstd = Out((N, P, C), t, wide), Out((N, G)), Out((N, G))
    hc.check(hc.hc_groupnorm_fwd(d, x, gamma, beta, y.t, mean.t, rstd.t, ws, nb))
    near("y", y, ref["y"], 1e-5)
    near("mean", mean, ref["mean"], 1e-5)
    near("rstd", rstd, ref["rstd"], 1e-5)
    y2 = Out((N, P, C), t)
    hc.check(hc.hc_groupnorm_fwd(d, x, gamma, beta, y2.t, ws=ws, ws_bytes=nb))  # keeping no statistics
    assert np.array_equal(y.numpy(), y2.numpy())
    gx, gg, gb = Out((N, P, C), t, wide), Out((C,)), Out((C,))
    bwd = lambda a, b, c: hc.check(hc.hc_groupnorm_bwd(d, x, gamma, beta, mean.t, rstd.t, gy, a, b, c, ws, nb))
    bwd(gx.t, gg.t, gb.t)
    if P * C // G > 2:  # two values of a group leave nothing but rounding
        # gx is what is left of q after its projections on 1 and xhat: held to the size of rstd * q
        top = np.abs(ref["rstd"]).max() * np.abs(gyr).max() * np.abs(gr).max()
        assert np.abs(gx.numpy() - ref["gx"]).max() <= 1e-5 * top + ROUND[t] * np.abs(ref["gx"]).max()
    near("ggamma", gg, ref["ggamma"], 1e-4)
    near("gbeta", gb, ref["gbeta"], 1e-4)
    again = Out((N, P, C), t), Out((C,)), Out((C,))
    bwd(*(o.t for o in again))
    for a, b in zip((gx, gg, gb), again):
        assert np.array_equal(a.numpy(), b.numpy())
    only = Out((N, P, C), t)
    bwd(only.t, None, None)
    assert np.array_equal(only.numpy(), gx.numpy())


def test_groupnorm_large_offset(hc):
    """A common offset of 1000 standard deviations: squares of the values themselves would lose the variance."""
    N, P, C, G = 1, 4096, 32, 4
    s = Data(2, torch.float32)
    x, xr = s.rows(N, P, C, 1.0, 1000.0)
    gamma, gr = s.param(C, shift=1.0)
    beta, br = s.param(C)
    d = hc.groupnorm_desc(N, P, C, G, torch.float32, 1e-5, hc.HC_PW_NONE)
    ws, nb = space(hc, hc.hc_groupnorm_workspace_size(d, 0))
    y, mean, rstd = Out((N, P, C)), Out((N, G)), Out((N, G))
    hc.check(hc.hc_groupnorm_fwd(d, x, gamma, beta, y.t, mean.t, rstd.t, ws, nb))
    ref = M.groupnorm(xr, gr, br, G, 1e-5, "none")
    near("rstd", rstd, ref["rstd"], 1e-5)
    # mean is held to its last bit, 2^-24 * 1000 = 6e-5 of a standard deviation
    assert np.abs(y.numpy() - ref["y"]).max() <= 2e-4


# ---------------------------------------------------------------- causal convolution

CC = [(1, 1, 1, 2, "f32", "none", False, False, 0), (2, 0, 8, 4, "f32", "silu", True, False, 0),
      (3, 1, 16, 4, "bf16", "silu", True, True, 0), (5, 33, 24, 4, "f32", "silu", True, True, 0),
      (5, 70, 40, 3, "f16", "silu", False, True, 0), (2, 129, 264, 4, "bf16", "silu", True, False, 8),
      (2, 61, 17, 5, "f32", "silu", True, True, 3), (1, 300, 12, 8, "f32", "none", True, False, 0),
      (2, 40, 16, 7, "bf16", "silu", False, False, 0), (2, 45, 8, 6, "f16", "none", True, True, 0),
      (1, 3, 2050, 4, "f32", "silu", True, False, 0), (70, 5, 8, 4, "bf16", "silu", True, True, 0)]


@pytest.mark.parametrize("B,L,D,K,dt,kind,state,ragged,wide", CC)
def test_causal_conv(hc, B, L, D, K, dt, kind, state, ragged, wide):
    t = DT[dt]
    lens, lens_d = lens_of(ragged, B, L)
    s = Data(3, t, wide, lens)
    x, xr = s.rows(B, L, D)
    gy, gyr = s.rows(B, L, D)
    w, wr = s.param(D, K, scale=0.5)
    bias, br = s.param(D, scale=0.5)
    whole = Data(4, t)
    (si, sir), (gso, gsor) = whole.rows(B, K - 1, D), whole.rows(B, K - 1, D)
    if not state:
        si = sir = gso = gsor = None
    act = hc.HC_PW_SILU if kind == "silu" else hc.HC_PW_NONE
    d = hc.causal_conv_desc(B, L, D, K, t, act)
    ref = M.causal_conv(xr, wr, br, kind, sir, lens, gyr, gsor)
    y, so = Out((B, L, D), t, wide), Out((B, K - 1, D), t)
    hc.check(hc.hc_causal_conv_fwd(d, x, w, bias, y.t, si, so.t, lens_d))
    near("y", y, ref["y"], 1e-5)
    assert np.array_equal(so.numpy(), ref["state"])
    ws, nb = space(hc, hc.hc_causal_conv_workspace_size(d))
    gx, gw, gb, gs = Out((B, L, D), t, wide), Out((D, K)), Out((D,)), Out((B, K - 1, D), t)
    hc.check(hc.hc_causal_conv_bwd(d, x, w, bias, gy, gx.t, gw.t, gb.t, si, gso, gs.t, lens_d, ws, nb))
    near("gx", gx, ref["gx"], 1e-5)
    near("gw", gw, ref["gw"], 1e-4)
    near("gb", gb, ref["gb"], 1e-4)
    near("gstate", gs, ref["gstate"], 1e-5)
    gx2, gw2 = Out((B, L, D), t), Out((D, K))
    hc.check(hc.hc_causal_conv_bwd(d, x, w, bias, gy, gx2.t, gw2.t, None, si, gso, None, lens_d, ws, nb))
    assert np.array_equal(gx.numpy(), gx2.numpy()) and np.array_equal(gw.numpy(), gw2.numpy())


@pytest.mark.parametrize("dt,D,K,T", [("f32", 24, 4, 9), ("bf16", 40, 3, 5), ("f16", 7, 2, 4)])
def test_causal_conv_step_by_step(hc, dt, D, K, T):
    """T one-token calls give the prompt call's rows and state, bit for bit."""
    t, B = DT[dt], 3
    s = Data(5, t)
    x, _ = s.rows(B, T, D)
    w, _ = s.param(D, K)
    bias, _ = s.param(D)
    si, _ = s.rows(B, K - 1, D)
    d = hc.causal_conv_desc(B, T, D, K, t, hc.HC_PW_SILU)
    y, so = Out((B, T, D), t), Out((B, K - 1, D), t)
    hc.check(hc.hc_causal_conv_fwd(d, x, w, bias, y.t, si, so.t))
    state = si.contiguous().clone()
    for i in range(T):
        o = Out((B, D), t)
        hc.check(hc.hc_causal_conv_step(d, x[:, i], w, bias, state, o.t))
        assert np.array_equal(o.numpy(), y.numpy()[:, i]), i
    assert np.array_equal(state.double().cpu().numpy(), so.numpy())


# ---------------------------------------------------------------- selective scan

#      B  L    D  G  N  type  gate  state  ragged wide
SC = [(1, 1, 1, 1, 1, "f32", False, False, False, 0), (2, 0, 8, 1, 16, "f32", True, True, False, 0),
      (1, 15, 64, 1, 16, "f32", True, False, False, 0), (2, 16, 132, 1, 16, "f32", True, True, False, 4),
      (5, 50, 40, 2, 7, "f32", True, True, True, 0), (1, 100, 256, 1, 16, "bf16", True, True, False, 0),
      (3, 33, 36, 4, 4, "f16", False, True, True, 0), (2, 40, 24, 1, 33, "f32", True, True, True, 3),
      (1, 70, 20, 1, 64, "f32", True, True, False, 0), (2, 48, 300, 2, 13, "bf16", True, True, True, 0),
      (2, 31, 70, 1, 8, "f32", False, True, False, 1), (1, 64, 520, 1, 3, "f32", True, True, False, 0),
      (6, 130, 16, 1, 32, "f16", True, False, True, 0), (1, 1100, 48, 1, 16, "f32", True, True, False, 0),
      (2, 2050, 136, 1, 16, "bf16", True, True, True, 0), (3, 5, 1030, 1, 16, "f32", True, True, True, 0)]


def scan_data(B, L, D, G, N, t, gate, state, lens, wide, seed=6):
    s = Data(seed, t, wide, lens)
    x = {}
    x["u"], x["dt"], x["gy"] = s.rows(B, L, D), s.rows(B, L, D, 0.5), s.rows(B, L, D)
    x["z"] = s.rows(B, L, D) if gate else (None, None)
    x["Bm"], x["Cm"] = s.rows(B, L, G * N), s.rows(B, L, G * N)
    x["A"] = s.param(D, N, value=-np.arange(1, N + 1) * np.exp(s.r.normal(size=(D, N)) * 0.2))
    x["D"] = s.param(D, scale=0.3, shift=1.0)
    x["bias"] = s.param(D, scale=1.0, shift=-3.0)
    x["h0"], x["ghT"] = (s.param(B, D, N), s.param(B, D, N)) if state else ((None, None), (None, None))
    return {k: v[0] for k, v in x.items()}, {k: v[1] for k, v in x.items()}


@pytest.mark.parametrize("B,L,D,G,N,dt,gate,state,ragged,wide", SC)
def test_selective_scan(hc, B, L, D, G, N, dt, gate, state, ragged, wide):
    t = DT[dt]
    lens, lens_d = lens_of(ragged, B, L)
    x, r = scan_data(B, L, D, G, N, t, gate, state, lens, wide)
    ref = M.scan(r["u"], r["dt"], r["A"], r["Bm"], r["Cm"], G, True, r["D"], r["z"], r["bias"], r["h0"], lens, r["gy"],
                 r["ghT"])
    d = hc.selective_scan_desc(B, L, D, N, t, G)
    ws, nb = space(hc, hc.hc_selective_scan_workspace_size(d, 1))
    saved, _ = space(hc, hc.hc_selective_scan_saved_size(d))
    kw = dict(D=x["D"], z=x["z"], dt_bias=x["bias"], h0=x["h0"], lens=lens_d, ws=ws, ws_bytes=nb)
    args = (x["u"], x["dt"], x["A"], x["Bm"], x["Cm"])
    y, hT = Out((B, L, D), t, wide), Out((B, D, N))
    hc.check(hc.hc_selective_scan_fwd(d, *args, y.t, hT=hT.t, saved=saved, **kw))
    near("y", y, ref["y"], 1e-5)
    near("hT", hT, ref["state"], 1e-5)
    y2, hT2 = Out((B, L, D), t), Out((B, D, N))
    hc.check(hc.hc_selective_scan_fwd(d, *args, y2.t, hT=hT2.t, **kw))  # keeping nothing for a backward pass
    assert np.array_equal(y.numpy(), y2.numpy()) and np.array_equal(hT.numpy(), hT2.numpy())

    def backward():
        o = dict(gu=Out((B, L, D), t, wide), gdt=Out((B, L, D), t, wide), gA=Out((D, N)), gB=Out((B, L, G * N), t, wide),
                 gC=Out((B, L, G * N), t, wide), gD=Out((D,)), gdt_bias=Out((D,)))
        if gate:
            o["gz"] = Out((B, L, D), t, wide)
        if state:
            o["gstate"] = Out((B, D, N))
        g = {k: v.t for k, v in o.items()}
        hc.check(hc.hc_selective_scan_bwd(d, *args, x["gy"], saved, g["gu"], g["gdt"], g["gA"], g["gB"], g["gC"],
                                          ghT=x["ghT"], gD=g["gD"], gz=g.get("gz"), gdt_bias=g["gdt_bias"],
                                          gh0=g.get("gstate"), **kw))
        return o

    o = backward()
    for k, v in o.items():
        near(k, v, ref[k], 1e-4 if k in ("gA", "gD", "gdt_bias") else 1e-5)
    for (k, a), b in zip(o.items(), backward().values()):
        assert np.array_equal(a.numpy(), b.numpy()), k


def test_selective_scan_bare(hc):
    """No softplus, D, gate, bias, states or lengths: the plain recurrence."""
    B, L, D, N = 2, 37, 12, 5
    s = Data(7, torch.float32)
    u, ur = s.rows(B, L, D)
    dt, dtr = s.rows(B, L, D, 0.01, 0.1)
    Bm, Br = s.rows(B, L, N)
    Cm, Cr = s.rows(B, L, N)
    gy, gyr = s.rows(B, L, D)
    A, Ar = s.param(D, N, scale=0.2, shift=-2.0)
    ref = M.scan(ur, dtr, Ar, Br, Cr, 1, False, gy=gyr)
    d = hc.selective_scan_desc(B, L, D, N, torch.float32, 1, 0)
    ws, nb = space(hc, hc.hc_selective_scan_workspace_size(d, 1))
    saved, _ = space(hc, hc.hc_selective_scan_saved_size(d))
    y = Out((B, L, D))
    hc.check(hc.hc_selective_scan_fwd(d, u, dt, A, Bm, Cm, y.t, saved=saved, ws=ws, ws_bytes=nb))
    near("y", y, ref["y"], 1e-5)
    o = dict(gu=Out((B, L, D)), gdt=Out((B, L, D)), gA=Out((D, N)), gB=Out((B, L, N)), gC=Out((B, L, N)))
    hc.check(hc.hc_selective_scan_bwd(d, u, dt, A, Bm, Cm, gy, saved, *(v.t for v in o.values()), ws=ws, ws_bytes=nb))
    for k, v in o.items():
        near(k, v, ref[k], 1e-4 if k == "gA" else 1e-5)


@pytest.mark.parametrize("dt,D,G,N,gate", [("f32", 24, 2, 16, True), ("bf16", 40, 1, 7, True), ("f16", 9, 1, 64, False),
                                           ("f32", 130, 1, 3, True)])
def test_selective_scan_step_by_step(hc, dt, D, G, N, gate):
    t, B, T = DT[dt], 3, 6
    x, r = scan_data(B, T, D, G, N, t, gate, True, None, 0, seed=8)
    ref = M.scan(r["u"], r["dt"], r["A"], r["Bm"], r["Cm"], G, True, r["D"], r["z"], r["bias"], r["h0"])
    d = hc.selective_scan_desc(B, T, D, N, t, G)
    state = Out((B, D, N))
    state.t.copy_(x["h0"])
    for i in range(T):
        y = Out((B, D), t, 3)
        hc.check(hc.hc_selective_scan_step(d, x["u"][:, i], x["dt"][:, i], x["A"], x["Bm"][:, i], x["Cm"][:, i], state.t,
                                           y.t, D=x["D"], z=x["z"][:, i] if gate else None, dt_bias=x["bias"]))
        near(f"y {i}", y, ref["y"][:, i], 1e-5)
    near("state", state, ref["state"], 1e-5)


# ---------------------------------------------------------------- shared hazards

def test_offsets_past_32_bits(hc):
    """Two sequences 2^31 + 8 elements apart in one buffer."""
    far = (1 << 31) + 8
    L, C = 40, 16
    buf = torch.empty(far + L * C, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((2, L, C), (far, C, 1))
    g = torch.Generator(device="cuda").manual_seed(1)
    x.copy_(torch.randn(2, L, C, generator=g, device="cuda"))
    out = torch.empty(far + L * C, dtype=torch.bfloat16, device="cuda")
    y = out.as_strided((2, L, C), (far, C, 1))
    xr = x.double().cpu().numpy()
    s = Data(9, torch.bfloat16)
    w, wr = s.param(C, 4)
    hc.check(hc.hc_causal_conv_fwd(hc.causal_conv_desc(2, L, C, 4, x.dtype, hc.HC_PW_SILU), x, w, None, y))
    near("conv", y, M.causal_conv(xr, wr, None, "silu")["y"], 1e-5)
    gamma, gr = s.param(C)
    beta, br = s.param(C)
    d = hc.groupnorm_desc(2, L, C, 4, x.dtype)
    ws, nb = space(hc, hc.hc_groupnorm_workspace_size(d, 0))
    hc.check(hc.hc_groupnorm_fwd(d, x, gamma, beta, y, ws=ws, ws_bytes=nb))
    near("norm", y, M.groupnorm(xr, gr, br, 4, 1e-5, "none")["y"], 1e-5)
    A, Ar = s.param(C, 16, scale=0.1, shift=-1.0)
    d = hc.selective_scan_desc(2, L, C, 16, x.dtype)
    ws, nb = space(hc, hc.hc_selective_scan_workspace_size(d, 0))
    hc.check(hc.hc_selective_scan_fwd(d, x, x, A, x, x, y, ws=ws, ws_bytes=nb))
    near("scan", y, M.scan(xr, xr, Ar, xr, xr, 1)["y"], 1e-5)


def test_on_another_stream(hc):
    """Every call of a short chain on a side stream that waits for the inputs' stream."""
    B, L, D, N = 2, 200, 64, 16
    x, r = scan_data(B, L, D, 1, N, torch.float32, True, False, None, 0, seed=10)
    side = torch.cuda.Stream()
    y, c = torch.empty(B, L, D, device="cuda"), torch.empty(B, L, D, device="cuda")
    w, wr = Data(11, torch.float32).param(D, 4)
    d, dc = hc.selective_scan_desc(B, L, D, N, torch.float32), hc.causal_conv_desc(B, L, D, 4, torch.float32)
    ws, nb = space(hc, hc.hc_selective_scan_workspace_size(d, 0))
    side.wait_stream(torch.cuda.current_stream())
    hc.check(hc.hc_causal_conv_fwd(dc, x["u"], w, None, c, stream=side))
    hc.check(hc.hc_selective_scan_fwd(d, c, x["dt"], x["A"], x["Bm"], x["Cm"], y, z=x["z"], ws=ws, ws_bytes=nb,
                                      stream=side))
    side.synchronize()
    cr = M.causal_conv(r["u"], wr, None, "none")["y"]
    near("y", y, M.scan(cr, r["dt"], r["A"], r["Bm"], r["Cm"], 1, z=r["z"])["y"], 1e-5)
