"""The sequence block (spatially_sharded_cnn_gb300/block.py) as a whole, on small maps: its rows and
gradients against the operators' 64-bit formulas chained with 64-bit projections, a stream of single
frames against all frames at once, and the whole on a side stream and replayed from a CUDA graph.

Tolerances, of the largest value: a row passes eight tensors that are rounded to bf16 on the way (n1,
qkv, s, its projection, y1, n2, h, f) and is rounded itself, a gradient those, and ten of its own; each
rounding is off by at most half a step, 2^-8 of a value, and is handed on by normed or random products,
which do not amplify it: 9 and 20 half steps."""
import numpy as np
import pytest
import torch

import block_ref as R

pytestmark = pytest.mark.gpu

T, P, C, H, F = 37, 6, 32, 2, 40
STEP = 2.0 ** -8


@pytest.fixture(scope="module")
def mod():
    assert torch.cuda.is_available()
    from spatially_sharded_cnn_gb300 import build
    build.build()
    from spatially_sharded_cnn_gb300 import block
    return block


def make(mod, device="cuda"):
    m = mod.AttentionBlock(C=C, H=H, F=F, seed=3)
    g = torch.Generator().manual_seed(4)
    for k in ("gamma1", "beta1", "gamma2", "beta2"):
        m.p[k] += 0.1 * torch.randn(C, generator=g).cuda()
    return m


def chain(p, x, gy):
    """The block in 64 bits, forward and backward: x, gy (T, P, C)."""
    seq = lambda t: np.swapaxes(t, 0, 1)
    flat = lambda t: t.reshape(T * P, -1)
    norm = lambda v, k, g=None: R.layernorm(v, p["gamma" + k], p["beta" + k], 1e-5, None, g)
    n1 = norm(x, "1")["y"]
    qkv = n1 @ p["w_qkv"]
    q, k, v = (seq(qkv[..., i * C:(i + 1) * C]) for i in range(3))
    attn = lambda g=None: R.linear_attn(q, k, v, H, (C // H) ** -0.5, p["log_decay"], gy=g)
    s = seq(attn()["y"])
    y1 = x + s @ p["w_o"]
    n2 = flat(norm(y1, "2")["y"])
    f = R.gated_ffn(n2, p["w_in"], p["w_out"], "silu", flat(gy))
    g = dict(w_in=f["gw_in"], w_out=f["gw_out"])
    b = norm(y1, "2", f["gx"].reshape(T, P, C))
    g["gamma2"], g["beta2"] = b["ggamma"], b["gbeta"]
    g1 = gy + b["gx"]
    g["w_o"] = flat(s).T @ flat(g1)
    a = attn(seq(g1 @ p["w_o"].T))
    gqkv = np.concatenate([seq(a[n]) for n in ("gq", "gk", "gv")], -1)
    g["w_qkv"] = flat(n1).T @ flat(gqkv)
    b = norm(x, "1", gqkv @ p["w_qkv"].T)
    g["gamma1"], g["beta1"] = b["ggamma"], b["gbeta"]
    return y1 + f["y"].reshape(T, P, C), g1 + b["gx"], g


def data():
    r = np.random.default_rng(5)
    return [torch.from_numpy(r.normal(size=(T, P, C))).to(torch.bfloat16).cuda() for _ in range(2)]


def test_forward_backward_and_stream(mod):
    m = make(mod)
    x, gy = data()
    p = {k: v.double().cpu().numpy() for k, v in m.p.items()}
    y, kept = m.forward(x, train=True)
    gx, g = m.backward(gy, kept)
    ry, rgx, rg = chain(p, x.double().cpu().numpy(), gy.double().cpu().numpy())

    def near(got, ref, steps, name):
        got = got.double().cpu().numpy()
        assert got.shape == ref.shape, name
        assert np.abs(got - ref).max() <= steps * STEP * np.abs(ref).max(), (name, np.abs(got - ref).max() / np.abs(ref).max())

    near(y, ry, 9, "y")
    near(gx, rgx, 20, "gx")
    for name, ref in rg.items():
        near(g[name], ref, 20, name)
    assert torch.equal(m.forward(x), y)
    states = m.states(P)
    rows = torch.stack([m.step(x[t], states) for t in range(T)])
    near(rows, ry, 9, "stream")


def test_side_stream_and_graph(mod):
    """On a side stream, and replayed from a graph with other inputs in the same places: the same bits."""
    m = make(mod)
    x, gy = data()
    y, kept = m.forward(x, train=True)
    want = [y, *m.backward(gy, kept)[1].values()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y, kept = m.forward(x, train=True)
        got = [y, *m.backward(gy, kept)[1].values()]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph, xin, gin = torch.cuda.CUDAGraph(), x.clone(), gy.clone()
    with torch.cuda.graph(graph):
        y, kept = m.forward(xin, train=True)
        out = [y, *m.backward(gin, kept)[1].values()]
    xin.zero_(), gin.zero_()
    graph.replay()
    xin.copy_(x), gin.copy_(gy)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, out))


def test_main_runs(mod, capsys):
    mod.main()
    assert "one frame of a stream" in capsys.readouterr().out
