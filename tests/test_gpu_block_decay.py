"""Linear attention over long and idle streams, head by head: states that are carried over many rows with a slow decay,
states that fade while nothing is added, heads of every memory beside one another.

A factor lambda that is rounded once near 1 is the same amount off at every row (or chunk, or cell of a sequence), so
that the state of n of them is up to n half steps (2^-24) off; what does not build up are roundings of the sums, which
have random signs: sqrt(n) of them.  Outputs are compared with the largest value of their own head: a head that
remembers thousands of rows holds values tens of times those of one that remembers three.

Tolerances are those of test_gpu_block.py (1e-5 for states) unless a test derives its own."""
import numpy as np
import pytest
import torch

import block_ref as R
from test_gpu_block import attn_inputs, run_attn
from test_gpu_mixer import DT, ROUND, Data, Out, lens_of, near, space

pytestmark = pytest.mark.gpu
SLOW = (-2.4e-4, -1.3e-4, -7e-5, -3e-5, -1e-5, -1e-6, 0.0)


@pytest.fixture(scope="module")
def hc():
    assert torch.cuda.is_available()
    from spatially_sharded_cnn_gb300 import build
    build.build()
    from spatially_sharded_cnn_gb300 import hc as mod
    return mod


def near_heads(name, out, ref, H, bar):
    """near() for each head: states (B, H, Dk, Dv), rows (B, L, H * D)."""
    got = torch.from_numpy(out.numpy()).to(out.t.dtype) if isinstance(out, Out) else out
    for h in range(H):
        one = lambda t: t[:, h] if t.ndim == 4 else t.reshape(*t.shape[:2], H, -1)[:, :, h]
        near(f"{name}, head {h}", one(got), one(ref), bar)


def summed(k, v, a, z0, first=0):
    """z0 lambda^n + sum over rows j of lambda^(n - 1 - j + first) k_j v_j^T, in 64 bits: k (n, H, Dk), v (n, H, Dv)."""
    n = k.shape[0]
    a = a.double()
    w = torch.exp(a * torch.arange(n - 1 + first, first - 1, -1, device="cuda", dtype=torch.float64)[:, None])  # (n, H)
    z = torch.einsum("nhd,nhe->hde", k.double() * w[..., None], v.double())
    return z + torch.exp(a * n)[:, None, None] * z0.double()


# ---------------------------------------------------------------- one token after another

@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_step_slow_decays(hc, dt):
    """8192 single tokens end in the state that the sequence ends in.  Each is rounded twice at most, by up to 2^-24 of
    the state, with random signs: sqrt(2 * 8192) * 2^-24 / sqrt(3) = 4.4e-6 of it."""
    t, n, H, D = DT[dt], 8192, len(SLOW), 16
    s = Data(11, t)
    q, k, v = (s.rows(n, 1, H * D)[0][:, 0] for _ in range(3))
    decay, _ = s.param(H, value=np.array(SLOW))
    h0, _ = s.param(1, H, D, D)
    d = hc.linear_attn_desc(1, 1, H, D, D, t)
    state, y = h0.clone(), Out((1, H * D), t)
    for i in range(n):
        hc.check(hc.hc_linear_attn_step(d, q[i:i + 1], k[i:i + 1], v[i:i + 1], state, y.t, decay))
    ref = summed(k.view(n, H, D), v.view(n, H, D), decay, h0[0])
    near_heads("state", state, ref[None].cpu().numpy(), H, 1e-5)
    last = D ** -0.5 * torch.einsum("hd,hde->he", q[-1].view(H, D).double(), ref)
    near_heads("y", y.t[None], last.reshape(1, 1, H * D).cpu().numpy(), H, 1e-5)


def test_step_idle(hc):
    """Tokens whose k is zero: the state is lambda^n of what it was, whatever lambda is."""
    values = (-0.2, -0.7, -3.0, -9.0, -16.0, -40.0)
    H, D, n = len(values), 8, 2
    s = Data(12, torch.float32)
    q, v = (s.rows(1, 1, H * D)[0][:, 0] for _ in range(2))
    decay, a = s.param(H, value=np.array(values))
    h0, hr = s.param(1, H, D, D)
    d = hc.linear_attn_desc(1, 1, H, D, D, torch.float32)
    state, y = h0.clone(), Out((1, H * D))
    for _ in range(n):
        hc.check(hc.hc_linear_attn_step(d, q, torch.zeros_like(q), v, state, y.t, decay))
    # (a * log2(e) is rounded by up to 2^-24 of it: 40 * 6e-8 = 2.4e-6 of lambda)
    near_heads("state", state, hr * np.exp(n * a)[None, :, None, None], H, 1e-5)


# ---------------------------------------------------------------- sequences

@pytest.mark.parametrize("dt,Dk,Dv,sms", [("bf16", 64, 64, 1), ("bf16", 64, 64, 0), ("bf16", 128, 128, 1),
                                          ("bf16", 128, 72, 0), ("bf16", 40, 128, 1), ("f32", 32, 32, 1),
                                          ("f32", 32, 41, 0), ("f16", 32, 32, 0)])
def test_sequence_slow_decays(hc, dt, Dk, Dv, sms):
    """98341 rows, as one segment (one SM) and cut into segments: states, their gradients, the rows at the far end."""
    t, L, H, tail = DT[dt], 98341, len(SLOW) + 1, 40
    a = attn_inputs(13, t, 1, 1, H, Dk, Dv, 0, None, True, False)  # (its rows are not used)
    s = Data(14, t)
    rows = lambda D: torch.randn(1, L, H * D, generator=torch.Generator("cuda").manual_seed(int(s.r.integers(1 << 30))),
                                 device="cuda").to(t)
    q, k, v, gy = rows(Dk), rows(Dk), rows(Dv), rows(Dv)
    a.update(q=(q,), k=(k,), v=(v,), gy=(gy,), decay=s.param(H, value=np.array(SLOW + (-0.3,))))
    decay, ar = a["decay"]
    d = hc.linear_attn_desc(1, L, H, Dk, Dv, t)
    hc.check(hc.hc_set_sm_count(sms))
    try:
        o = run_attn(hc, d, a, 1, L, H, Dk, Dv, t, 0, None)
    finally:
        hc.check(hc.hc_set_sm_count(0))
    assert hc.hc_sync_check(None) == hc.HC_OK
    heads = lambda x: x[0].view(x.shape[1], H, -1)
    # the state ahead of the last rows, the state's gradient behind the first (lambda G of row `tail`)
    ahead = summed(heads(k)[:-tail], heads(v)[:-tail], decay, a["h0"][0][0])
    back = lambda x: heads(x).flip(0)
    behind = summed(d.scale * back(q)[:-tail].double(), back(gy)[:-tail], decay, a["ghT"][0][0], first=1)
    n = lambda x: x.double().cpu().numpy()
    lo, hi = slice(0, tail), slice(L - tail, L)
    end = R.linear_attn(*(n(x[:, hi]) for x in (q, k, v)), H, d.scale, ar, n(ahead[None]), None, n(gy[:, hi]))
    top = R.linear_attn(*(n(x[:, lo]) for x in (q, k, v)), H, d.scale, ar, a["h0"][1], None, n(gy[:, lo]), n(behind[None]))
    bar = 1e-5 + ROUND[t]
    near_heads("state", o["state"], end["state"], H, 1e-5)
    near_heads("gstate", o["gstate"], top["gstate"], H, 1e-5)
    near_heads("y", o["y"].t[:, hi], end["y"], H, bar)
    near_heads("gq", o["gq"].t[:, hi], end["gq"], H, bar)
    near_heads("gk", o["gk"].t[:, lo], top["gk"], H, bar)
    near_heads("gv", o["gv"].t[:, lo], top["gv"], H, bar)


@pytest.mark.parametrize("decay", [-1.7e-5, -9e-6, -5.3e-6, -3.1e-6, -1.1e-6, -4e-7])
def test_cells_slow_decays(hc, decay):
    """One head of fp32 rows alone, cut into some 400 cells: what a state loses over a cell is not rounded to a factor
    near 1, either.  Sums inside cells are rounded at every row, by up to 2^-24 of the cell's sum (state / sqrt(400)):
    224 rows of 400 cells leave sqrt(224) * 2^-24 / sqrt(3) = 5e-7 of the state, the joins sqrt(400) * 2^-24 / sqrt(3) =
    7e-7; held to 3e-6."""
    t, L, D = torch.float32, 98304, 32
    s = Data(15, t)
    q, k, v = (torch.randn(1, L, D, generator=torch.Generator("cuda").manual_seed(i), device="cuda") for i in range(3))
    a, _ = s.param(1, value=np.array([decay]))
    h0, _ = s.param(1, 1, D, D)
    d = hc.linear_attn_desc(1, L, 1, D, D, t)
    y, hT = torch.empty_like(q), Out((1, 1, D, D))
    hc.check(hc.hc_linear_attn_fwd(d, q, k, v, y, a, h0, hT.t, None, *space(hc, hc.hc_linear_attn_workspace_size(d, 0))))
    ref = summed(k[0][:, None], v[0][:, None], a, h0[0])
    near("state", hT, ref[None].cpu().numpy(), 3e-6)


@pytest.mark.parametrize("dt,D,rows,values", [("f32", 24, 32, (-0.01, -0.1, -0.3, -0.6)), ("f16", 40, 32, (-0.02, -0.2, -0.6)),
                                              ("bf16", 64, 128, (-0.003, -0.02, -0.1, -0.15)),
                                              ("bf16", 128, 128, (-0.003, -0.02, -0.1, -0.15)),
                                              ("bf16", 8, 600, (-0.003, -0.02, -0.04)), ("f32", 8, 600, (-0.003, -0.02, -0.04))])
def test_sequence_fades(hc, dt, D, rows, values):
    """After `rows` rows nothing is added for twice as long (k is zero): the state is lambda^n of what it was, down to
    e^-50, relative to itself (exponents are rounded by 2^-24 of 50: 3e-6)."""
    t, L, H = DT[dt], 3 * rows, len(values)
    a = attn_inputs(16, t, 1, L, H, D, D, 0, None, True, False)
    a["k"][0][:, rows:] = 0
    a["k"][1][:, rows:] = 0
    a["q"][0][:, :2 * rows] = 0  # and backwards: the state's gradient from the last third
    a["q"][1][:, :2 * rows] = 0
    a["decay"] = Data(17, t).param(H, value=np.array(values))
    d = hc.linear_attn_desc(1, L, H, D, D, t)
    o = run_attn(hc, d, a, 1, L, H, D, D, t, 0, None)
    ref = R.linear_attn(a["q"][1], a["k"][1], a["v"][1], H, d.scale, a["decay"][1], a["h0"][1], None, a["gy"][1], a["ghT"][1])
    near_heads("state", o["state"], ref["state"], H, 1e-5)
    near_heads("gstate", o["gstate"], ref["gstate"], H, 1e-5)


HEADS = (-0.01, -0.3, -0.0004, -40.0, -np.inf, 0.0)


@pytest.mark.parametrize("dt,B,L,Dk,Dv,ragged", [("bf16", 2, 300, 64, 64, False), ("bf16", 1, 900, 128, 128, False),
                                                 ("bf16", 5, 200, 40, 128, True), ("bf16", 5, 515, 64, 64, True),
                                                 ("f32", 5, 150, 41, 24, True), ("f16", 1, 400, 64, 32, False)])
def test_heads(hc, dt, B, L, Dk, Dv, ragged):
    """Heads that remember 100 rows, 3, thousands, nothing to speak of, nothing at all and everything, each against itself."""
    t, H = DT[dt], len(HEADS)
    lens, lens_t = lens_of(ragged, B, L)
    a = attn_inputs(18, t, B, L, H, Dk, Dv, 0, lens, True, False)
    a["decay"] = Data(19, t).param(H, value=np.array(HEADS))
    d = hc.linear_attn_desc(B, L, H, Dk, Dv, t)
    o = run_attn(hc, d, a, B, L, H, Dk, Dv, t, 0, lens_t)
    ref = R.linear_attn(a["q"][1], a["k"][1], a["v"][1], H, d.scale, a["decay"][1], a["h0"][1], lens, a["gy"][1], a["ghT"][1])
    for name, out in o.items():
        near_heads(name, out, ref[name], H, 1e-5 + (ROUND[t] if out.t.dtype == t and t != torch.float32 else 0.0))
