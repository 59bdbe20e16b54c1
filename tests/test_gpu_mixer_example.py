"""The temporal mixer (spatially_sharded_cnn_gb300/mixer.py) as a whole, in fp32 on small maps: its
rows against the operators' 64-bit formulas chained with 64-bit projections, its gradients against
central differences of that chain, and a stream of single frames against all frames at once."""
import numpy as np
import pytest
import torch

import mixer_ref as M

pytestmark = pytest.mark.gpu

T, P, C, D, K, N, G = 5, 6, 8, 12, 3, 4, 4


@pytest.fixture(scope="module")
def mixer():
    assert torch.cuda.is_available()
    from spatially_sharded_cnn_gb300 import build
    build.build()
    from spatially_sharded_cnn_gb300.mixer import TemporalMixer
    # the projections in full fp32
    torch.backends.cuda.matmul.allow_tf32 = False
    m = TemporalMixer(C=C, D=D, K=K, N=N, groups=G, dtype=torch.float32, seed=3)
    g = torch.Generator().manual_seed(4)
    for k in ("gamma", "beta", "conv_bias"):
        m.p[k] += 0.1 * torch.randn(m.p[k].shape, generator=g).cuda()
    return m


def chain(m, x, p):
    """The mixer in 64 bits: x (T, P, C)."""
    seq = lambda t: np.swapaxes(t, 0, 1)
    n = M.groupnorm(x, p["gamma"], p["beta"], G, 1e-5, "silu")["y"]
    xz = n @ p["w_in"]
    c = seq(M.causal_conv(seq(xz[..., :D]), p["conv"], p["conv_bias"], "silu")["y"])
    proj = c @ p["w_x"]
    R = m.R
    s = M.scan(seq(c), seq(proj[..., :R] @ p["w_dt"]), p["A"], seq(proj[..., R:R + N]), seq(proj[..., R + N:]), 1, True,
               p["D"], seq(xz[..., D:]), p["dt_bias"])["y"]
    return x + seq(s) @ p["w_out"]


def test_forward_backward_and_stream(mixer):
    r = np.random.default_rng(5)
    x = torch.from_numpy(r.normal(size=(T, P, C))).float().cuda()
    gy = torch.from_numpy(r.normal(size=(T, P, C))).float().cuda()
    p = {k: v.double().cpu().numpy() for k, v in mixer.p.items()}
    xr, gr = x.double().cpu().numpy(), gy.double().cpu().numpy()
    y, kept = mixer.forward(x, train=True)
    ref = chain(mixer, xr, p)
    assert np.abs(y.double().cpu().numpy() - ref).max() <= 1e-5 * np.abs(ref).max()
    assert torch.equal(mixer.forward(x), y)
    states = mixer.states(P)
    rows = torch.stack([mixer.step(x[t], states) for t in range(T)])
    assert float((rows - y).abs().max()) <= 1e-5 * float(y.abs().max())

    gx, g = mixer.backward(gy, kept)
    # differences of the 64-bit chain along random directions: truncation ~ h^2 = 1e-10 of the
    # value, rounding ~ 1e-16 / h = 1e-11; the fp32 gradients are held to 1e-4 of their own size
    h = 1e-5
    for name, grad in dict(g, x=gx).items():
        grad = grad.double().cpu().numpy()
        base = xr if name == "x" else p[name]
        for k in range(3):
            v = np.random.default_rng(10 + k).normal(size=base.shape)
            v /= np.linalg.norm(v)
            f = lambda s: float((gr * (chain(mixer, xr + s * v, p) if name == "x" else
                                       chain(mixer, xr, dict(p, **{name: base + s * v})))).sum())
            want = (f(h) - f(-h)) / (2 * h)
            got = float((grad * v).sum())
            assert abs(got - want) <= 1e-4 * max(np.linalg.norm(grad), 1e-3), (name, got, want)


def test_main_runs(mixer, capsys):
    from spatially_sharded_cnn_gb300 import mixer as mod
    mod.main()
    assert "one frame of a stream" in capsys.readouterr().out
