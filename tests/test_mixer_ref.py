"""The 64-bit formulas of the mixer operators (tests/mixer_ref.py) against central differences of
their own forward passes: every gradient, on small ragged inputs with carried states (no GPU)."""
import numpy as np
import pytest

import mixer_ref as M

STEP, BAR = 1e-5, 1e-7  # truncation ~ STEP^2, rounding ~ 1e-16 / STEP = 1e-11


def _check(forward, inputs, weights, grads):
    """forward(inputs) -> outputs; the scalar is sum over outputs of weights * output."""
    total = lambda: sum(float((weights[k] * v).sum()) for k, v in forward().items() if k in weights)
    for name, g in grads.items():
        x = inputs[name]
        flat, want = x.reshape(-1), g.reshape(-1)
        for i in range(flat.size):
            keep = flat[i]
            flat[i] = keep + STEP
            hi = total()
            flat[i] = keep - STEP
            lo = total()
            flat[i] = keep
            d = (hi - lo) / (2 * STEP)
            assert abs(d - want[i]) <= BAR * max(1.0, abs(d)), (name, i, d, want[i])


@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
def test_groupnorm_gradients(kind):
    r = np.random.default_rng(1)
    i = dict(x=r.normal(size=(2, 5, 6)), gamma=r.normal(size=6), beta=r.normal(size=6))
    gy = r.normal(size=(2, 5, 6))
    f = lambda: M.groupnorm(i["x"], i["gamma"], i["beta"], 3, 1e-5, kind)
    o = M.groupnorm(i["x"], i["gamma"], i["beta"], 3, 1e-5, kind, gy)
    _check(f, i, dict(y=gy), dict(x=o["gx"], gamma=o["ggamma"], beta=o["gbeta"]))


@pytest.mark.parametrize("K,kind", [(2, "silu"), (4, "silu"), (3, "none")])
def test_causal_conv_gradients(K, kind):
    r = np.random.default_rng(2)
    lens = np.array([5, 0, 1, 2])
    i = dict(x=r.normal(size=(4, 5, 3)), w=r.normal(size=(3, K)), bias=r.normal(size=3), state=r.normal(size=(4, K - 1, 3)))
    gy, gs = r.normal(size=(4, 5, 3)), r.normal(size=(4, K - 1, 3))
    f = lambda: M.causal_conv(i["x"], i["w"], i["bias"], kind, i["state"], lens)
    o = M.causal_conv(i["x"], i["w"], i["bias"], kind, i["state"], lens, gy, gs)
    _check(f, i, dict(y=gy, state=gs), dict(x=o["gx"], w=o["gw"], bias=o["gb"], state=o["gstate"]))


@pytest.mark.parametrize("softplus,gate", [(True, True), (False, False)])
def test_scan_gradients(softplus, gate):
    r = np.random.default_rng(3)
    B, L, D, G, N = 3, 4, 4, 2, 3
    lens = np.array([4, 0, 1])
    i = dict(u=r.normal(size=(B, L, D)), dt=r.uniform(0.05, 0.5, size=(B, L, D)), A=-r.uniform(0.5, 2, size=(D, N)),
             Bm=r.normal(size=(B, L, G * N)), Cm=r.normal(size=(B, L, G * N)), D=r.normal(size=D),
             bias=r.normal(size=D) * 0.1, h0=r.normal(size=(B, D, N)))
    if gate:
        i["z"] = r.normal(size=(B, L, D))
    gy, gh = r.normal(size=(B, L, D)), r.normal(size=(B, D, N))
    run = lambda **k: M.scan(i["u"], i["dt"], i["A"], i["Bm"], i["Cm"], G, softplus, i["D"], i.get("z"), i["bias"],
                             i["h0"], lens, **k)
    o = run(gy=gy, ghT=gh)
    g = dict(u=o["gu"], dt=o["gdt"], A=o["gA"], Bm=o["gB"], Cm=o["gC"], D=o["gD"], bias=o["gdt_bias"], h0=o["gstate"])
    if gate:
        g["z"] = o["gz"]
    _check(run, i, dict(y=gy, state=gh), g)


def test_blocks_with_carried_states_are_the_whole():
    """A sequence cut in two, the states handed over, forward and backward, is the uncut one."""
    r = np.random.default_rng(4)
    B, L, D, N, K, cut = 2, 7, 3, 4, 3, 3
    x, w, bias = r.normal(size=(B, L, D)), r.normal(size=(D, K)), r.normal(size=D)
    gy, dt = r.normal(size=(B, L, D)), r.normal(size=(B, L, D))
    Bm, Cm, A = r.normal(size=(B, L, N)), r.normal(size=(B, L, N)), -r.uniform(0.5, 2, size=(D, N))
    whole = M.causal_conv(x, w, bias, "silu", gy=gy)
    left = M.causal_conv(x[:, :cut], w, bias, "silu")
    right = M.causal_conv(x[:, cut:], w, bias, "silu", left["state"], gy=gy[:, cut:])
    left = M.causal_conv(x[:, :cut], w, bias, "silu", gy=gy[:, :cut], gstate_out=right["gstate"])
    assert np.allclose(np.concatenate([left["y"], right["y"]], 1), whole["y"], atol=1e-12)
    assert np.allclose(np.concatenate([left["gx"], right["gx"]], 1), whole["gx"], atol=1e-12)
    assert np.allclose(left["gw"] + right["gw"], whole["gw"], atol=1e-12)
    part = lambda s, **k: M.scan(x[:, s], dt[:, s], A, Bm[:, s], Cm[:, s], 1, gy=gy[:, s], **k)
    a, b = slice(0, cut), slice(cut, L)
    whole = part(slice(0, L))
    right = part(b, h0=part(a)["state"])
    left = part(a, ghT=right["gstate"])
    for k in ("y", "gu", "gdt", "gB", "gC"):
        assert np.allclose(np.concatenate([left[k], right[k]], 1), whole[k], atol=1e-12), k
    assert np.allclose(left["gA"] + right["gA"], whole["gA"], atol=1e-12)
