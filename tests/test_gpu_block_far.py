"""The sequence block's backward calls on rows whose offsets pass 2^31 elements and 2^32 bytes, in batches and in rows,
and captured calls that use one workspace."""
import numpy as np
import pytest
import torch

import block_ref as R
from test_gpu_block_uses import attn, rnd
from test_gpu_mixer import ROUND, Out, near, space

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
n64 = lambda t: t.double().cpu().numpy()


@pytest.fixture(scope="module")
def hc():
    assert torch.cuda.is_available()
    from spatially_sharded_cnn_gb300 import build
    build.build()
    from spatially_sharded_cnn_gb300 import hc as mod
    return mod


def far_rows(B, L, row, D, count):
    """`count` (B, L, D) slices of rows `row` elements apart; the first half of them inputs."""
    buf = torch.empty(B, L, row, dtype=BF, device="cuda")
    s = [buf[..., i * D:(i + 1) * D] for i in range(count)]
    assert s[-1].stride(0) * (B - 1) + s[-1].stride(1) * (L - 1) > 1 << 31
    return s


@pytest.mark.parametrize("D", [64, 24])
def test_attention_backward(hc, D):
    """The last sequence ends behind 2^31 elements; its last rows against the recurrence over its last 300 (a decay of
    -0.5 leaves e^-100 of what lies 200 rows back)."""
    B, L = 2, 30000
    q, k, v, gy, gq, gk, gv = far_rows(B, L, 40000, D, 7)
    for i, t in enumerate((q, k, v, gy)):
        t.copy_(rnd(B, L, D, seed=i))
    for t in (gq, gk, gv):
        t.fill_(float("nan"))
    decay = torch.tensor([-0.5], device="cuda")
    d = hc.linear_attn_desc(B, L, 1, D, D, BF)
    ws, nb = space(hc, hc.hc_linear_attn_workspace_size(d, 1))
    hc.check(hc.hc_linear_attn_bwd(d, q, k, v, gy, gq, gk, gv, decay, ws=ws, ws_bytes=nb))
    ref = R.linear_attn(*(n64(t[1:, -300:]) for t in (q, k, v)), 1, d.scale, np.array([-0.5]), gy=n64(gy[1:, -300:]))
    for name, t in (("gq", gq), ("gk", gk), ("gv", gv)):
        near(name, t[1:, -100:].contiguous(), ref[name][:, -100:], 1e-5 + ROUND[BF])
        assert torch.isfinite(t).all()


@pytest.mark.parametrize("D", [64, 24, 333])
def test_norm_backward(hc, D):
    B, L = 2, 30000
    x, gy, gx = far_rows(B, L, 40000, D, 3)
    x.copy_(rnd(B, L, D, seed=1))
    gy.copy_(rnd(B, L, D, seed=2))
    gx.fill_(float("nan"))
    g, mean, rstd = torch.ones(D, device="cuda"), torch.empty(B, L, device="cuda"), torch.empty(B, L, device="cuda")
    d = hc.layernorm_desc(B, L, D, BF)
    gg, gb = Out((D,)), Out((D,))
    hc.check(hc.hc_layernorm_fwd(d, x, g, g, torch.empty(B, L, D, dtype=BF, device="cuda"), mean, rstd))
    ws, nb = space(hc, hc.hc_layernorm_workspace_size(d))
    hc.check(hc.hc_layernorm_bwd(d, x, g, mean, rstd, gy, gx, gg.t, gb.t, ws=ws, ws_bytes=nb))
    one = np.ones(D)
    near("gx", gx[1:, -50:].contiguous(), R.layernorm(n64(x[1:, -50:]), one, one, 1e-5, None, n64(gy[1:, -50:]))["gx"], 1e-5)
    assert torch.isfinite(gx).all()
    x, gy = x.double(), gy.double()
    xh = (x - x.mean(-1, keepdim=True)) * (x.var(-1, unbiased=False, keepdim=True) + 1e-5).rsqrt()
    near("ggamma", gg, n64((gy * xh).sum((0, 1))), 1e-4)
    near("gbeta", gb, n64(gy.sum((0, 1))), 1e-4)


def test_ffn_backward(hc):
    M, C, F = 60000, 64, 32
    x, gy, gx = (t[0] for t in far_rows(1, M, 40000, C, 3))
    x.copy_(rnd(M, C, seed=1))
    gy.copy_(rnd(M, C, seed=2))
    gx.fill_(float("nan"))
    wi, wo = rnd(C, 2 * F, seed=3, scale=C ** -0.5), rnd(F, C, seed=4, scale=F ** -0.5)
    d = hc.gated_ffn_desc(M, C, F, BF)
    gwi, gwo = Out((C, 2 * F), BF), Out((F, C), BF)
    ws, nb = space(hc, hc.hc_gated_ffn_workspace_size(d, 1))
    hc.check(hc.hc_gated_ffn_bwd(d, x, wi, wo, gy, gx, gwi.t, gwo.t, ws, nb))
    ref = R.gated_ffn(n64(x), n64(wi), n64(wo), "silu", n64(gy))
    for name, t in (("gx", gx.contiguous()), ("gw_in", gwi), ("gw_out", gwo)):
        near(name, t, ref[name], 1e-5 + ROUND[BF])


def test_graphs_that_share_a_workspace(hc):
    """Captured calls of all three operators over one workspace, replayed one behind another in several orders."""
    d = hc.linear_attn_desc(1, 3000, 2, 64, 64, BF)
    df, dn = hc.gated_ffn_desc(1500, 256, 512, BF), hc.layernorm_desc(1, 1500, 256, BF)
    sizes = [hc.hc_linear_attn_workspace_size(d, 1), hc.hc_gated_ffn_workspace_size(df, 1), hc.hc_layernorm_workspace_size(dn)]
    ws, nb = space(hc, (max(s for s, _ in sizes), max(n for _, n in sizes)))
    jobs = []
    for i in range(2):
        q, k, v, gy = (rnd(1, 3000, 128, seed=10 * i + j) for j in range(4))
        x, gx = rnd(1500, 256, seed=50 + i), rnd(1500, 256, seed=55 + i)
        wi, wo = rnd(256, 1024, seed=60 + i, scale=0.06), rnd(512, 256, seed=70 + i, scale=0.05)
        decay, g = torch.full((2,), -0.01 * (i + 1), device="cuda"), torch.ones(256, device="cuda")
        out = [torch.empty_like(t) for t in (q, q, k, v, x, x, wi, wo, x, x, g, g)]
        stats = [torch.empty(1500, device="cuda") for _ in range(2)]

        def run(q=q, k=k, v=v, gy=gy, x=x, gx=gx, wi=wi, wo=wo, decay=decay, g=g, out=out, stats=stats):
            st = torch.cuda.current_stream()
            attn(hc, d, q, k, v, decay, ws=(ws, nb), stream=st, y=out[0])
            hc.check(hc.hc_linear_attn_bwd(d, q, k, v, gy, *out[1:4], decay, ws=ws, ws_bytes=nb, stream=st))
            hc.check(hc.hc_gated_ffn_fwd(df, x, wi, wo, out[4], ws, nb, st))
            hc.check(hc.hc_gated_ffn_bwd(df, x, wi, wo, gx, *out[5:8], ws, nb, st))
            hc.check(hc.hc_layernorm_fwd(dn, x[None], g, g, out[8][None], *stats, stream=st))
            hc.check(hc.hc_layernorm_bwd(dn, x[None], g, *stats, gx[None], out[9][None], *out[10:], ws=ws, ws_bytes=nb,
                                         stream=st))

        run()
        torch.cuda.synchronize()
        want = [t.clone() for t in out]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        jobs.append((graph, out, want, run))  # (run holds the tensors that the graph uses)
    for order in ((0, 1), (1, 0), (1, 1, 0)):
        for _, out, _, _ in jobs:
            for t in out:
                t.zero_()
        ws.fill_(0xFF)
        for i in order:
            jobs[i][0].replay()
        torch.cuda.synchronize()
        for _, out, want, _ in jobs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert hc.hc_sync_check(None) == hc.HC_OK
