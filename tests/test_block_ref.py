"""The gradients of the 64-bit formulas in block_ref.py against central differences (no GPU)."""
import numpy as np
import pytest

import block_ref as R

H = 1e-6


def against_differences(f, values, grads, weights):
    """f(**values) -> outputs; the gradients of sum(weights * outputs) along random directions."""
    total = lambda v: sum(float((weights[k] * o).sum()) for k, o in f(**v).items() if k in weights)
    for name, g in grads.items():
        v = np.random.default_rng(1).normal(size=values[name].shape)
        up, down = dict(values, **{name: values[name] + H * v}), dict(values, **{name: values[name] - H * v})
        want = (total(up) - total(down)) / (2 * H)
        got = float((g * v).sum())
        assert abs(got - want) <= 1e-6 * max(1.0, abs(want)), (name, got, want)


@pytest.mark.parametrize("lens", [None, [5, 0, 2]])
def test_layernorm(lens):
    r = np.random.default_rng(0)
    v = dict(x=r.normal(size=(3, 5, 7)), gamma=r.normal(size=7), beta=r.normal(size=7))
    gy = r.normal(size=(3, 5, 7))
    o = R.layernorm(**v, eps=1e-5, lens=lens, gy=gy)
    against_differences(lambda **a: R.layernorm(**a, eps=1e-5, lens=lens), v,
                        dict(x=o["gx"], gamma=o["ggamma"], beta=o["gbeta"]), dict(y=gy))


@pytest.mark.parametrize("lens", [None, [6, 0, 1]])
def test_linear_attn(lens):
    r = np.random.default_rng(0)
    v = dict(q=r.normal(size=(3, 6, 8)), k=r.normal(size=(3, 6, 8)), v=r.normal(size=(3, 6, 10)),
             h0=r.normal(size=(3, 2, 4, 5)))
    w = dict(y=r.normal(size=(3, 6, 10)), state=r.normal(size=(3, 2, 4, 5)))
    kw = dict(H=2, scale=0.7, decay=np.array([-0.2, -1.5]), lens=lens)
    o = R.linear_attn(**v, **kw, gy=w["y"], ghT=w["state"])
    against_differences(lambda **a: R.linear_attn(**a, **kw), v, dict(q=o["gq"], k=o["gk"], v=o["gv"], h0=o["gstate"]), w)


@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
def test_gated_ffn(kind):
    r = np.random.default_rng(0)
    v = dict(x=r.normal(size=(5, 4)), w_in=r.normal(size=(4, 12)), w_out=r.normal(size=(6, 4)))
    gy = r.normal(size=(5, 4))
    o = R.gated_ffn(**v, kind=kind, gy=gy)
    against_differences(lambda **a: R.gated_ffn(**a, kind=kind), v, dict(x=o["gx"], w_in=o["gw_in"], w_out=o["gw_out"]),
                        dict(y=gy))
