"""The sequence block's operators in the uses between the single calls: sequences cut into blocks with
carried states, calls back to back, graphs, other streams, SM counts, many sequences, broadcast and
unaligned rows, rows behind 2^31 elements."""
import numpy as np
import pytest
import torch

import block_ref as R
from test_gpu_block import attn_inputs, run_attn
from test_gpu_mixer import DT, ROUND, Data, Out, lens_of, near, space

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def hc():
    assert torch.cuda.is_available()
    from spatially_sharded_cnn_gb300 import build
    build.build()
    from spatially_sharded_cnn_gb300 import hc as mod
    return mod


def rnd(*shape, dtype=BF, seed=0, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda") * scale).to(dtype)


def attn(hc, d, q, k, v, decay, h0=None, lens=None, ws=None, stream=None, y=None):
    y = torch.empty(d.B, d.L, d.H * d.Dv, dtype=q.dtype, device="cuda") if y is None else y
    hT = torch.empty(d.B, d.H, d.Dk, d.Dv, device="cuda")
    ws = space(hc, hc.hc_linear_attn_workspace_size(d, 1)) if ws is None else ws
    hc.check(hc.hc_linear_attn_fwd(d, q, k, v, y, decay, h0, hT, lens, *ws, stream))
    return y, hT


@pytest.mark.parametrize("dt,D,cut", [("f32", 41, 100), ("bf16", 64, 333), ("bf16", 128, 128), ("f16", 32, 77)])
def test_attention_in_blocks(hc, dt, D, cut):
    """Two blocks of a sequence, the state handed on, against the whole; backwards with the state's gradient."""
    t, B, L, H = DT[dt], 2, 700, 2
    a = attn_inputs(7, t, B, L, H, D, D, 0, None, True, True)
    x = {k: v[0] for k, v in a.items()}
    ref = R.linear_attn(a["q"][1], a["k"][1], a["v"][1], H, D ** -0.5, a["decay"][1], a["h0"][1], None, a["gy"][1],
                        a["ghT"][1])
    part = lambda s: {k: x[k][:, s] for k in ("q", "k", "v", "gy")}
    first, second = part(slice(0, cut)), part(slice(cut, L))
    d1, d2 = (hc.linear_attn_desc(B, n, H, D, D, t) for n in (cut, L - cut))
    y1, mid = attn(hc, d1, first["q"], first["k"], first["v"], x["decay"], x["h0"])
    y2, end = attn(hc, d2, second["q"], second["k"], second["v"], x["decay"], mid)
    bar = 1e-5 + (ROUND[t] if t != torch.float32 else 0.0)
    near("y", torch.cat([y1, y2], 1), ref["y"], bar)
    near("state", end, ref["state"], 1e-5)

    def back(d, s, h0, ghT):
        o = [torch.empty_like(s[k]).contiguous() for k in ("q", "k", "v")]
        g0 = torch.empty_like(ghT)
        ws = space(hc, hc.hc_linear_attn_workspace_size(d, 1))
        hc.check(hc.hc_linear_attn_bwd(d, s["q"], s["k"], s["v"], s["gy"], *o, x["decay"], h0, ghT, g0, None, *ws))
        return o, g0

    o2, gmid = back(d2, second, mid, x["ghT"])
    o1, g0 = back(d1, first, x["h0"], gmid)
    for name, p, q in zip(("gq", "gk", "gv"), o1, o2):
        near(name, torch.cat([p, q], 1), ref[name], bar)
    near("gstate", g0, ref["gstate"], 1e-5)


@pytest.mark.parametrize("sms", [1, 7, 76, 152])
def test_attention_at_other_sm_counts(hc, sms):
    """Other cuts of the sequence: the same values within the bars, the same bits when called again."""
    B, L, H, D = 1, 2700, 2, 64
    a = attn_inputs(8, BF, B, L, H, D, D, 0, None, True, True)
    ref = R.linear_attn(a["q"][1], a["k"][1], a["v"][1], H, D ** -0.5, a["decay"][1], a["h0"][1], None, a["gy"][1],
                        a["ghT"][1])
    d = hc.linear_attn_desc(B, L, H, D, D, BF)
    hc.check(hc.hc_set_sm_count(sms))
    try:
        o = run_attn(hc, d, a, B, L, H, D, D, BF, 0, None)
        again = run_attn(hc, d, a, B, L, H, D, D, BF, 0, None)
    finally:
        hc.check(hc.hc_set_sm_count(0))
    for name, out in o.items():
        near(name, out, ref[name], 1e-5 + (ROUND[BF] if out.t.dtype == BF else 0.0))
        assert torch.equal(out.t, again[name].t), name


@pytest.mark.parametrize("sms", [1, 2, 9, 152])
def test_ffn_and_norm_at_other_sm_counts(hc, sms):
    M, C, F = 700, 136, 264
    x, gy, wi, wo = rnd(M, C, seed=1), rnd(M, C, seed=2), rnd(C, 2 * F, seed=3, scale=C ** -0.5), rnd(F, C, seed=4, scale=F ** -0.5)
    n = lambda t: t.double().cpu().numpy()
    ref = R.gated_ffn(n(x), n(wi), n(wo), "gelu", n(gy))
    d, dn = hc.gated_ffn_desc(M, C, F, BF, hc.HC_PW_GELU), hc.layernorm_desc(1, M, C, BF)
    g = torch.ones(C, device="cuda")
    hc.check(hc.hc_set_sm_count(sms))
    try:
        runs = []
        for _ in range(2):
            y, gx, gwi, gwo = (torch.empty_like(v) for v in (x, x, wi, wo))
            ws = space(hc, hc.hc_gated_ffn_workspace_size(d, 1))
            hc.check(hc.hc_gated_ffn_fwd(d, x, wi, wo, y, *ws))
            hc.check(hc.hc_gated_ffn_bwd(d, x, wi, wo, gy, gx, gwi, gwo, *ws))
            yn, gn, mean, rstd = torch.empty_like(x), torch.empty_like(x), *(torch.empty(M, device="cuda") for _ in range(2))
            gg, gb = torch.empty_like(g), torch.empty_like(g)
            wn = space(hc, hc.hc_layernorm_workspace_size(dn))
            hc.check(hc.hc_layernorm_fwd(dn, x[None], g, g, yn[None], mean, rstd))
            hc.check(hc.hc_layernorm_bwd(dn, x[None], g, mean, rstd, gy[None], gn[None], gg, gb, None, *wn))
            runs.append([y, gx, gwi, gwo, yn, gn, gg, gb])
    finally:
        hc.check(hc.hc_set_sm_count(0))
    assert all(torch.equal(a, b) for a, b in zip(*runs))
    for name, out in zip(("y", "gx", "gw_in", "gw_out"), runs[0]):
        near(name, out, ref[name], 1e-5 + ROUND[BF])
    ln = R.layernorm(n(x)[None], np.ones(C), np.ones(C), 1e-5, None, n(gy)[None])
    for name, out, bar in (("y", runs[0][4][None], 1e-5), ("gx", runs[0][5][None], 1e-5), ("ggamma", runs[0][6], 1e-4)):
        near(name, out, ln[name], bar)


def test_back_to_back_with_parameters_written_between(hc):
    """Each call takes what the kernel just before it wrote (weights, decays, states), whatever overlaps."""
    B, H, D, C, F = 64, 4, 64, 256, 512
    q, x = rnd(B, H * D, seed=1), rnd(B, C, seed=2)
    wi, wo = rnd(C, 2 * F, seed=3, scale=C ** -0.5), rnd(F, C, seed=4, scale=F ** -0.5)
    d, df = hc.linear_attn_desc(B, 1, H, D, D, BF), hc.gated_ffn_desc(B, C, F, BF)
    ws = space(hc, hc.hc_gated_ffn_workspace_size(df, 0))

    def go(wait):
        state, decay, w, h = torch.zeros(B, H, D, D, device="cuda"), torch.zeros(H, device="cuda"), wi.clone(), x.clone()
        out = []
        for i in range(6):
            decay.fill_(-0.1 * i)
            y = torch.empty_like(q)
            hc.check(hc.hc_linear_attn_step(d, q, q, q, state, y, decay))
            wait()
            w.mul_(0.9)
            f = torch.empty_like(h)
            hc.check(hc.hc_gated_ffn_fwd(df, h, w, wo, f, *ws))
            wait()
            h = f
            out += [y, f]
        return out + [state]

    a, b = go(lambda: None), go(torch.cuda.synchronize)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_two_graphs_and_streams_at_once(hc):
    """Two captured calls with workspaces of their own, replayed on two streams at once."""
    d = hc.linear_attn_desc(1, 3000, 2, 64, 64, BF)
    df = hc.gated_ffn_desc(1500, 256, 512, BF)
    jobs = []
    for i in range(2):
        q, k, v = (rnd(1, 3000, 128, seed=10 * i + j) for j in range(3))
        x, wi, wo = rnd(1500, 256, seed=50 + i), rnd(256, 1024, seed=60 + i, scale=0.06), rnd(512, 256, seed=70 + i, scale=0.05)
        decay = torch.full((2,), -0.01 * (i + 1), device="cuda")
        y, f = torch.empty_like(q), torch.empty_like(x)
        ws, wf = space(hc, hc.hc_linear_attn_workspace_size(d, 0)), space(hc, hc.hc_gated_ffn_workspace_size(df, 0))

        def run(q=q, k=k, v=v, y=y, decay=decay, ws=ws, x=x, wi=wi, wo=wo, f=f, wf=wf):
            st = torch.cuda.current_stream()
            attn(hc, d, q, k, v, decay, ws=ws, stream=st, y=y)
            hc.check(hc.hc_gated_ffn_fwd(df, x, wi, wo, f, *wf, stream=st))

        run()
        torch.cuda.synchronize()
        want = (y.clone(), f.clone())
        y.zero_(), f.zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        jobs.append((g, torch.cuda.Stream(), (y, f), want, run))  # (run holds the tensors that the graph uses)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s, *_ in jobs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, _, got, want, _ in jobs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert hc.hc_sync_check(None) == hc.HC_OK


def test_many_sequences(hc):
    """70000 sequences of three rows, two heads; every one by itself."""
    B, L, H, D = 70000, 3, 2, 8
    q, k, v = (rnd(B, L, H * D, seed=i) for i in range(3))
    decay = torch.tensor([-0.1, -1.0], device="cuda")
    d = hc.linear_attn_desc(B, L, H, D, D, BF)
    y, hT = attn(hc, d, q, k, v, decay)
    for lo in (0, 34999, 69990):
        n = lambda t: t[lo:lo + 10].double().cpu().numpy()
        ref = R.linear_attn(n(q), n(k), n(v), H, D ** -0.5, decay.double().cpu().numpy())
        near("y", y[lo:lo + 10], ref["y"], 1e-5)
        near("state", hT[lo:lo + 10], ref["state"], 1e-5)


def test_broadcast_and_unaligned_rows(hc):
    """Rows that the copy engine does not take (a stride of 0, one that is no multiple of 16 bytes, an odd
    address) run in fp32 and give the same values."""
    B, L, H, D = 3, 200, 2, 32
    decay = torch.tensor([-0.02, -0.2], device="cuda")
    d = hc.linear_attn_desc(B, L, H, D, D, BF)
    q, k, v = rnd(1, L, H * D, seed=1), rnd(B, L, H * D, seed=2), rnd(B, L, H * D, seed=3)
    n = lambda t: t.double().cpu().numpy()
    ref = R.linear_attn(n(q.expand(B, -1, -1)), n(k), n(v), H, D ** -0.5, n(decay))
    y, _ = attn(hc, d, q.expand(B, -1, -1), k, v, decay)
    near("broadcast", y, ref["y"], 1e-5)
    wide = torch.zeros(B, L, H * D + 3, dtype=BF, device="cuda")
    wide[..., 1:1 + H * D] = k
    y, _ = attn(hc, d, q.expand(B, -1, -1).contiguous(), wide[..., 1:1 + H * D], v, decay)
    near("unaligned", y, ref["y"], 1e-5)
    x = torch.zeros(5, 7, 131, dtype=BF, device="cuda")
    x[..., 3:] = rnd(5, 7, 128, seed=9)
    g, y = torch.ones(128, device="cuda"), torch.empty(5, 7, 128, dtype=BF, device="cuda")
    hc.check(hc.hc_layernorm_fwd(hc.layernorm_desc(5, 7, 128, BF), x[..., 3:], g, g, y))
    near("norm", y, R.layernorm(n(x[..., 3:]), np.ones(128), np.ones(128), 1e-5)["y"], 1e-5)


@pytest.mark.parametrize("D", [64, 24])
def test_rows_behind_2_31_elements(hc, D):
    """Rows 40000 elements apart, 60000 of them: offsets past 2^31 elements and 2^32 bytes."""
    L, row = 60000, 40000
    buf = torch.empty(1, L, row, dtype=BF, device="cuda")
    q, k, v, y = (buf[..., i * D:(i + 1) * D] for i in range(4))
    for i, t in enumerate((q, k, v)):
        t.copy_(rnd(1, L, D, seed=i))
    decay = torch.tensor([-0.5], device="cuda")
    d = hc.linear_attn_desc(1, L, 1, D, D, BF)
    attn(hc, d, q, k, v, decay, y=y)
    # the decay leaves nothing of rows 200 back (e^-100)
    n = lambda t: t[:, -300:].double().cpu().numpy()
    ref = R.linear_attn(n(q), n(k), n(v), 1, D ** -0.5, np.array([-0.5]))
    near("y", y[:, -100:].contiguous(), ref["y"][:, -100:], 1e-5 + ROUND[BF])
    g = torch.ones(D, device="cuda")
    hc.check(hc.hc_layernorm_fwd(hc.layernorm_desc(1, L, D, BF), q, g, g, y))
    near("norm", y[:, -20:].contiguous(), R.layernorm(n(q)[:, -20:], np.ones(D), np.ones(D), 1e-5)["y"], 1e-5)
    if D == 64:
        f = hc.gated_ffn_desc(L, D, 32, BF)
        wi, wo = rnd(D, 64, seed=5, scale=0.1), rnd(32, D, seed=6, scale=0.1)
        hc.check(hc.hc_gated_ffn_fwd(f, q[0], wi, wo, y[0], *space(hc, hc.hc_gated_ffn_workspace_size(f, 0))))
        one = lambda t: t.double().cpu().numpy()
        near("feed-forward", y[0, -20:].contiguous(), R.gated_ffn(one(q[0, -20:]), one(wi), one(wo), "silu")["y"],
             1e-5 + ROUND[BF])


def test_lengths_out_of_range_are_taken_as_the_ends(hc):
    B, L, H, D = 3, 150, 1, 64
    q, k, v = (rnd(B, L, D, seed=i) for i in range(3))
    d = hc.linear_attn_desc(B, L, H, D, D, BF)
    lens = torch.tensor([-5, 1000, 70], dtype=torch.int32, device="cuda")
    ends = torch.tensor([0, L, 70], dtype=torch.int32, device="cuda")
    a, b = attn(hc, d, q, k, v, None, lens=lens), attn(hc, d, q, k, v, None, lens=ends)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert (a[0][0] == 0).all() and (a[0][2, 70:] == 0).all()
