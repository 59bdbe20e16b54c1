"""The mixer operators over a sequence cut into blocks (W shards) with carried states, over SM counts
that cut the work differently, and back to back in a stream.  Tolerances as in test_gpu_mixer.py."""
import numpy as np
import pytest
import torch

import mixer_ref as M
from test_gpu_mixer import DT, Data, Out, near, scan_data, space

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hc():
    assert torch.cuda.is_available()
    from spatially_sharded_cnn_gb300 import build
    build.build()
    from spatially_sharded_cnn_gb300 import hc as mod
    yield mod
    mod.hc_set_sm_count(0)


@pytest.mark.parametrize("dt,L,cut", [("f32", 70, 32), ("f32", 41, 3), ("bf16", 300, 150)])
def test_convolution_in_two_blocks(hc, dt, L, cut):
    """Two blocks, rows and gradients handed over, against the whole sequence in 64 bits."""
    t, B, D, K = DT[dt], 2, 24, 4
    s = Data(20, t)
    (x, xr), (gy, gyr) = s.rows(B, L, D), s.rows(B, L, D)
    (w, wr), (bias, br) = s.param(D, K, scale=0.5), s.param(D)
    ref = M.causal_conv(xr, wr, br, "silu", gy=gyr)
    y, gx = Out((B, L, D), t), Out((B, L, D), t)
    state, gstate = Out((B, K - 1, D), t), Out((B, K - 1, D), t)
    gw, gb = [], []
    parts = slice(0, cut), slice(cut, L)
    descs = [hc.causal_conv_desc(B, p.stop - p.start, D, K, t, hc.HC_PW_SILU) for p in parts]
    hc.check(hc.hc_causal_conv_fwd(descs[0], x[:, parts[0]], w, bias, y.t[:, parts[0]], None, state.t))
    hc.check(hc.hc_causal_conv_fwd(descs[1], x[:, parts[1]], w, bias, y.t[:, parts[1]], state.t, None))
    for i, (si, gso, gsi) in ((1, (state.t, None, gstate.t)), (0, (None, gstate.t, None))):
        ws, nb = space(hc, hc.hc_causal_conv_workspace_size(descs[i]))
        gw.append(Out((D, K)))
        gb.append(Out((D,)))
        hc.check(hc.hc_causal_conv_bwd(descs[i], x[:, parts[i]], w, bias, gy[:, parts[i]], gx.t[:, parts[i]], gw[-1].t,
                                       gb[-1].t, si, gso, gsi, None, ws, nb))
    near("y", y, ref["y"], 1e-5)
    if dt == "f32":  # in 16 bits the carried gradient is rounded between the blocks
        near("gx", gx, ref["gx"], 1e-5)
        near("gw", gw[0].t + gw[1].t, ref["gw"], 1e-4)
        near("gb", gb[0].t + gb[1].t, ref["gb"], 1e-4)


@pytest.mark.parametrize("L,cut", [(70, 32), (41, 3), (600, 304)])
def test_scan_in_two_blocks(hc, L, cut):
    B, D, N, t = 2, 40, 16, torch.float32
    x, r = scan_data(B, L, D, 1, N, t, True, False, None, 0, seed=21)
    ref = M.scan(r["u"], r["dt"], r["A"], r["Bm"], r["Cm"], 1, True, r["D"], r["z"], r["bias"], None, None, r["gy"])
    parts = slice(0, cut), slice(cut, L)
    descs = [hc.selective_scan_desc(B, p.stop - p.start, D, N, t) for p in parts]
    y, hT, g0 = Out((B, L, D)), Out((B, D, N)), Out((B, D, N))
    o = {k: Out((B, L, D)) for k in ("gu", "gdt", "gz")}
    o.update({k: Out((B, L, N)) for k in ("gB", "gC")})
    saved, sums = [], []
    args = lambda p: tuple(x[k][:, p] if k != "A" else x[k] for k in ("u", "dt", "A", "Bm", "Cm"))
    for i, (h0, out) in enumerate(((None, hT.t), (hT.t, None))):
        p = parts[i]
        ws, nb = space(hc, hc.hc_selective_scan_workspace_size(descs[i], 1))
        saved.append(space(hc, hc.hc_selective_scan_saved_size(descs[i]))[0])
        hc.check(hc.hc_selective_scan_fwd(descs[i], *args(p), y.t[:, p], D=x["D"], z=x["z"][:, p], dt_bias=x["bias"], h0=h0,
                                          hT=out, saved=saved[i], ws=ws, ws_bytes=nb))
    for i, (h0, gh0, ghT) in ((1, (hT.t, g0.t, None)), (0, (None, None, g0.t))):
        p = parts[i]
        ws, nb = space(hc, hc.hc_selective_scan_workspace_size(descs[i], 1))
        sums.append({"gA": Out((D, N)), "gD": Out((D,)), "gdt_bias": Out((D,))})
        hc.check(hc.hc_selective_scan_bwd(descs[i], *args(p), x["gy"][:, p], saved[i], o["gu"].t[:, p], o["gdt"].t[:, p],
                                          sums[-1]["gA"].t, o["gB"].t[:, p], o["gC"].t[:, p], D=x["D"], z=x["z"][:, p],
                                          dt_bias=x["bias"], h0=h0, ghT=ghT, gD=sums[-1]["gD"].t, gz=o["gz"].t[:, p],
                                          gdt_bias=sums[-1]["gdt_bias"].t, gh0=gh0, ws=ws, ws_bytes=nb))
    near("y", y, ref["y"], 1e-5)
    for k, v in o.items():
        near(k, v, ref[k], 1e-5)
    for k in sums[0]:
        near(k, sums[0][k].t + sums[1][k].t, ref[k], 1e-4)


@pytest.mark.parametrize("sms", [0, 37, 1, 1000])
def test_sm_counts(hc, sms):
    """Grids, chunks and segments sized for other SM counts: the same results within the bars, the same bits twice."""
    hc.check(hc.hc_set_sm_count(sms))
    try:
        B, L, D, N, t = 2, 400, 72, 16, torch.float32
        x, r = scan_data(B, L, D, 1, N, t, True, True, [L, 150], 0, seed=22)
        lens = torch.tensor([L, 150], dtype=torch.int32, device="cuda")
        ref = M.scan(r["u"], r["dt"], r["A"], r["Bm"], r["Cm"], 1, True, r["D"], r["z"], r["bias"], r["h0"], [L, 150],
                     r["gy"], r["ghT"])
        d = hc.selective_scan_desc(B, L, D, N, t)
        ws, nb = space(hc, hc.hc_selective_scan_workspace_size(d, 1))
        saved = space(hc, hc.hc_selective_scan_saved_size(d))[0]
        kw = dict(D=x["D"], z=x["z"], dt_bias=x["bias"], h0=x["h0"], lens=lens, ws=ws, ws_bytes=nb)
        args = (x["u"], x["dt"], x["A"], x["Bm"], x["Cm"])
        got = []
        for _ in range(2):
            y, hT = Out((B, L, D)), Out((B, D, N))
            hc.check(hc.hc_selective_scan_fwd(d, *args, y.t, hT=hT.t, saved=saved, **kw))
            o = dict(gu=Out((B, L, D)), gdt=Out((B, L, D)), gA=Out((D, N)), gB=Out((B, L, N)), gC=Out((B, L, N)))
            gz = Out((B, L, D))
            hc.check(hc.hc_selective_scan_bwd(d, *args, x["gy"], saved, *(v.t for v in o.values()), ghT=x["ghT"], gz=gz.t,
                                              **kw))
            got.append(dict(o, y=y, state=hT, gz=gz))
        for k, v in got[0].items():
            near(k, v, ref[k], 1e-4 if k == "gA" else 1e-5)
            assert np.array_equal(v.numpy(), got[1][k].numpy()), k
        n, p, c, g = 2, 3000, 96, 12
        s = Data(23, t)
        (f, fr), (gy, gyr), (gamma, gr), (beta, br) = s.rows(n, p, c), s.rows(n, p, c), s.param(c, shift=1.0), s.param(c)
        d = hc.groupnorm_desc(n, p, c, g, t, 1e-5, hc.HC_PW_SILU)
        ws, nb = space(hc, hc.hc_groupnorm_workspace_size(d, 1))
        y, gx, mean, rstd, gg, gb = Out((n, p, c)), Out((n, p, c)), Out((n, g)), Out((n, g)), Out((c,)), Out((c,))
        hc.check(hc.hc_groupnorm_fwd(d, f, gamma, beta, y.t, mean.t, rstd.t, ws, nb))
        hc.check(hc.hc_groupnorm_bwd(d, f, gamma, beta, mean.t, rstd.t, gy, gx.t, gg.t, gb.t, ws, nb))
        ref = M.groupnorm(fr, gr, br, g, 1e-5, "silu", gyr)
        for k, v, bar in (("y", y, 1e-5), ("gx", gx, 1e-5), ("ggamma", gg, 1e-4), ("gbeta", gb, 1e-4)):
            near(k, v, ref[k], bar)
    finally:
        hc.check(hc.hc_set_sm_count(0))


def test_large_map_takes_the_three_launches(hc):
    """A map past what L2 keeps, against torch's 64-bit group norm on the device."""
    n, p, c, g = 2, 40000, 256, 32
    x = torch.randn(n, p, c, device="cuda", generator=torch.Generator(device="cuda").manual_seed(24)) * 2 + 3
    gy = torch.randn(n, p, c, device="cuda", generator=torch.Generator(device="cuda").manual_seed(25))
    gamma, beta = torch.rand(c, device="cuda") + 0.5, torch.rand(c, device="cuda")
    d = hc.groupnorm_desc(n, p, c, g, x.dtype, 1e-5, hc.HC_PW_GELU)
    ws, nb = space(hc, hc.hc_groupnorm_workspace_size(d, 1))
    y, gx, mean, rstd, gg, gb = Out((n, p, c)), Out((n, p, c)), Out((n, g)), Out((n, g)), Out((c,)), Out((c,))
    hc.hc_trace_collect()
    hc.hc_trace_enable(True)
    hc.check(hc.hc_groupnorm_fwd(d, x, gamma, beta, y.t, mean.t, rstd.t, ws, nb))
    hc.check(hc.hc_groupnorm_bwd(d, x, gamma, beta, mean.t, rstd.t, gy, gx.t, gg.t, gb.t, ws, nb))
    hc.hc_trace_enable(False)
    assert "gn_stats_kernel" in hc.hc_trace_collect()[1]
    xd, gd, bd = x.double().requires_grad_(), gamma.double().requires_grad_(), beta.double().requires_grad_()
    out = torch.nn.functional.gelu(torch.nn.functional.group_norm(xd.transpose(1, 2), g, gd, bd, 1e-5)).transpose(1, 2)
    ref = torch.autograd.grad(out, (xd, gd, bd), gy.double())
    for k, v, r, bar in (("y", y, out.detach(), 1e-5), ("gx", gx, ref[0], 1e-5), ("ggamma", gg, ref[1], 1e-4),
                         ("gbeta", gb, ref[2], 1e-4)):
        near(k, v, r.cpu().numpy(), bar)


def test_calls_back_to_back_see_each_other(hc):
    """Convolution into scan into norm, a hundred times over the same buffers without a wait: every kernel starts
    while the one before it ends, and reads what that one wrote."""
    B, L, D, N = 4, 64, 32, 8
    x, r = scan_data(B, L, D, 1, N, torch.float32, False, False, None, 0, seed=26)
    w, wr = Data(27, torch.float32).param(D, 4, scale=0.4)
    gamma, gr = Data(28, torch.float32).param(D, shift=1.0)
    beta, br = Data(29, torch.float32).param(D)
    dc, ds = hc.causal_conv_desc(B, L, D, 4, torch.float32), hc.selective_scan_desc(B, L, D, N, torch.float32)
    dn = hc.groupnorm_desc(B, L, D, 4, torch.float32)
    ws, nb = space(hc, hc.hc_groupnorm_workspace_size(dn, 0))
    a, b = (torch.empty(B, L, D, device="cuda") for _ in range(2))
    cur = x["u"].clone()
    want, got = r["u"], []
    for i in range(100):
        hc.check(hc.hc_causal_conv_fwd(dc, cur, w, None, a))
        hc.check(hc.hc_selective_scan_fwd(ds, a, x["dt"], x["A"], x["Bm"], x["Cm"], b))
        hc.check(hc.hc_groupnorm_fwd(dn, b, gamma, beta, cur, ws=ws, ws_bytes=nb))
    first = cur.clone()
    cur.copy_(x["u"])
    for i in range(100):
        for f in (lambda: hc.hc_causal_conv_fwd(dc, cur, w, None, a),
                  lambda: hc.hc_selective_scan_fwd(ds, a, x["dt"], x["A"], x["Bm"], x["Cm"], b),
                  lambda: hc.hc_groupnorm_fwd(dn, b, gamma, beta, cur, ws=ws, ws_bytes=nb)):
            hc.check(f())
            torch.cuda.synchronize()
        if i == 0:
            want = M.groupnorm(M.scan(M.causal_conv(want, wr, None, "none")["y"], r["dt"], r["A"], r["Bm"], r["Cm"], 1)["y"],
                               gr, br, 4, 1e-5, "none")["y"]
            near("one round", cur, want, 1e-4)  # the norm divides by what the scan leaves
    assert torch.equal(first, cur)


@pytest.mark.parametrize("D", [47, 1, 5, 130])
@pytest.mark.parametrize("N", [4, 8, 16, 32, 64])
def test_scan_odd_channels_many_sequences(hc, D, N):
    """Channel counts whose rows of partial sums start off 16 bytes from the second sequence on."""
    B, L, t, lens = 5, 6, torch.float32, [6, 0, 1, 3, 5]
    x, r = scan_data(B, L, D, 1, N, t, True, True, lens, 0, seed=30)
    ref = M.scan(r["u"], r["dt"], r["A"], r["Bm"], r["Cm"], 1, True, r["D"], r["z"], r["bias"], r["h0"], lens, r["gy"],
                 r["ghT"])
    d = hc.selective_scan_desc(B, L, D, N, t)
    ws, nb = space(hc, hc.hc_selective_scan_workspace_size(d, 1))
    saved = space(hc, hc.hc_selective_scan_saved_size(d))[0]
    kw = dict(D=x["D"], z=x["z"], dt_bias=x["bias"], h0=x["h0"], ws=ws, ws_bytes=nb,
              lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    args = (x["u"], x["dt"], x["A"], x["Bm"], x["Cm"])
    y, hT = Out((B, L, D)), Out((B, D, N))
    hc.check(hc.hc_selective_scan_fwd(d, *args, y.t, hT=hT.t, saved=saved, **kw))
    o = dict(gu=Out((B, L, D)), gdt=Out((B, L, D)), gA=Out((D, N)), gB=Out((B, L, N)), gC=Out((B, L, N)))
    rest = dict(gz=Out((B, L, D)), gD=Out((D,)), gdt_bias=Out((D,)), gh0=Out((B, D, N)))
    hc.check(hc.hc_selective_scan_bwd(d, *args, x["gy"], saved, *(v.t for v in o.values()), ghT=x["ghT"],
                                      **{k: v.t for k, v in rest.items()}, **kw))
    for k, v in dict(o, y=y, state=hT, gstate=rest.pop("gh0"), **rest).items():
        near(k, v, ref[k], 1e-4 if k in ("gA", "gD", "gdt_bias") else 1e-5)


def test_captured_into_a_graph(hc):
    """Convolution, scan in segments and norm (a cluster and a cooperative grid) replayed from a CUDA graph."""
    B, L, D, N, t = 1, 512, 64, 16, torch.float32
    x, _ = scan_data(B, L, D, 1, N, t, True, False, None, 0, seed=31)
    w = Data(32, t).param(D, 4)[0]
    gamma, beta = Data(33, t).param(D, shift=1.0)[0], Data(34, t).param(D)[0]
    dc, ds = hc.causal_conv_desc(B, L, D, 4, t, hc.HC_PW_SILU), hc.selective_scan_desc(B, L, D, N, t)
    big, small = hc.groupnorm_desc(B, L, D, 4, t), hc.groupnorm_desc(B, 32, D, 4, t)
    ws, nb = space(hc, hc.hc_selective_scan_workspace_size(ds, 0))
    ns, nn = space(hc, hc.hc_groupnorm_workspace_size(big, 0))
    ms, nm = space(hc, hc.hc_groupnorm_workspace_size(small, 0))
    a, b, c = (torch.empty(B, L, D, device="cuda") for _ in range(3))
    e = torch.empty(B, 32, D, device="cuda")

    def chain(stream=None):
        hc.check(hc.hc_causal_conv_fwd(dc, x["u"], w, None, a, stream=stream))
        hc.check(hc.hc_selective_scan_fwd(ds, a, x["dt"], x["A"], x["Bm"], x["Cm"], b, z=x["z"], ws=ws, ws_bytes=nb,
                                          stream=stream))
        hc.check(hc.hc_groupnorm_fwd(big, b, gamma, beta, c, ws=ns, ws_bytes=nn, stream=stream))
        hc.check(hc.hc_groupnorm_fwd(small, c[:, :32], gamma, beta, e, ws=ms, ws_bytes=nm, stream=stream))

    chain()
    torch.cuda.synchronize()
    want = [v.clone() for v in (a, b, c, e)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(torch.cuda.current_stream())
    for v in (a, b, c, e):
        v.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    for v, r in zip((a, b, c, e), want):
        assert torch.equal(v, r)
