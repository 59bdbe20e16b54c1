"""The mixer operators' calls one right after another: each kernel may start while the one before it
in the stream ends, and has to see everything that one wrote.  The same calls with a wait after each
give the same bits."""
import pytest
import torch

from test_gpu_mixer import Data, scan_data, space

pytestmark = pytest.mark.gpu

CALLS = 300


@pytest.fixture(scope="module")
def hc():
    assert torch.cuda.is_available()
    from spatially_sharded_cnn_gb300 import build
    build.build()
    from spatially_sharded_cnn_gb300 import hc as mod
    return mod


def both(run):
    """What run(after) leaves with nothing after each call, and with a wait."""
    got, want = run(lambda: None), run(torch.cuda.synchronize)
    torch.cuda.synchronize()
    assert len(got) == len(want)
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.isfinite(b).all()
        assert torch.equal(a, b), i


@pytest.mark.parametrize("B,D,N", [(1, 8, 4), (64, 256, 16), (64, 2048, 16), (3, 47, 7)])
def test_scan_tokens_on_one_state(hc, B, D, N):
    """A token reads the state that the token before it wrote."""
    x, _ = scan_data(B, 1, D, 1, N, torch.float32, True, True, None, 0, seed=40)
    d = hc.selective_scan_desc(B, 1, D, N, torch.float32)
    row = {k: x[k][:, 0] for k in ("u", "dt", "Bm", "Cm", "z")}

    def run(after):
        state, y = x["h0"].clone(), torch.empty(CALLS, B, D, device="cuda")
        torch.cuda.synchronize()
        for i in range(CALLS):
            hc.check(hc.hc_selective_scan_step(d, row["u"], row["dt"], x["A"], row["Bm"], row["Cm"], state, y[i], D=x["D"],
                                               z=row["z"], dt_bias=x["bias"]))
            after()
        return y, state

    both(run)


@pytest.mark.parametrize("B,D,K", [(1, 8, 4), (64, 256, 4), (64, 2048, 4), (3, 47, 3)])
def test_conv_tokens_on_one_state(hc, B, D, K):
    s = Data(41, torch.float32)
    (x, _), (si, _), (w, _), (bias, _) = s.rows(CALLS, B, D), s.rows(B, K - 1, D), s.param(D, K), s.param(D)
    d = hc.causal_conv_desc(B, 1, D, K, torch.float32, hc.HC_PW_SILU)

    def run(after):
        state, y = si.clone(), torch.empty(CALLS, B, D, device="cuda")
        torch.cuda.synchronize()
        for i in range(CALLS):
            hc.check(hc.hc_causal_conv_step(d, x[i], w, bias, state, y[i]))
            after()
        return y, state

    both(run)


@pytest.mark.parametrize("P,C,G", [(64, 32, 4), (3000, 96, 12), (17000, 1024, 32)])
def test_norm_parameters_written_just_before(hc, P, C, G):
    """Every call's gamma and beta come from the kernel ahead of it, as an optimizer's update does: maps that take a
    cluster, a cooperative grid and three launches, forward and backward."""
    calls = CALLS if P < 10000 else 20
    s = Data(42, torch.float32)
    (gamma0, _), (beta0, _) = s.param(C, shift=1.0), s.param(C)
    g = torch.Generator(device="cuda").manual_seed(42)
    x, gy = (torch.randn(1, P, C, device="cuda", generator=g) for _ in range(2))
    d = hc.groupnorm_desc(1, P, C, G, torch.float32, act=hc.HC_PW_SILU)
    ws, nb = space(hc, hc.hc_groupnorm_workspace_size(d, 1))

    def run(after):
        gamma, beta = gamma0.clone(), beta0.clone()
        mean, rstd = torch.empty(1, G, device="cuda"), torch.empty(1, G, device="cuda")
        y, gx = (torch.empty(1, P, C, device="cuda") for _ in range(2))
        rows, grads, sums = [], torch.empty(calls, P, device="cuda"), torch.empty(calls, 2, C, device="cuda")
        torch.cuda.synchronize()
        for i in range(calls):
            gamma.add_(1.0)
            after()
            beta.sub_(0.25)
            after()
            hc.check(hc.hc_groupnorm_fwd(d, x, gamma, beta, y, mean, rstd, ws, nb))
            after()
            rows.append(y[0, ::7].clone())
            gamma.mul_(0.5)
            after()
            beta.add_(0.125)
            after()
            hc.check(hc.hc_groupnorm_bwd(d, x, gamma, beta, mean, rstd, gy, gx, sums[i, 0], sums[i, 1], ws, nb))
            after()
            grads[i] = gx[0, :, i % C]
        return [sums, grads, y, gx] + rows

    both(run)


@pytest.mark.parametrize("B,L,D", [(2, 40, 24), (8, 300, 264)])
def test_conv_parameters_written_just_before(hc, B, L, D):
    K, s = 4, Data(43, torch.float32)
    (x, _), (gy, _), (w0, _), (bias0, _) = s.rows(B, L, D), s.rows(B, L, D), s.param(D, K), s.param(D)
    d = hc.causal_conv_desc(B, L, D, K, torch.float32, hc.HC_PW_SILU)
    ws, nb = space(hc, hc.hc_causal_conv_workspace_size(d))

    def run(after):
        w, bias = w0.clone(), bias0.clone()
        y, gx, step = torch.empty(B, L, D, device="cuda"), torch.empty(B, L, D, device="cuda"), torch.empty(B, D, device="cuda")
        state = torch.zeros(B, K - 1, D, device="cuda")
        rows, sums = [], torch.empty(CALLS, D * K + D, device="cuda")
        torch.cuda.synchronize()
        for i in range(CALLS):
            for f in (lambda: bias.add_(0.01), lambda: w.mul_(-0.99),
                      lambda: hc.check(hc.hc_causal_conv_fwd(d, x, w, bias, y)), lambda: rows.append(y[0].clone()),
                      lambda: bias.sub_(0.02), lambda: w.add_(0.03),
                      lambda: hc.check(hc.hc_causal_conv_bwd(d, x, w, bias, gy, gx, sums[i, :D * K], sums[i, D * K:],
                                                             ws=ws, ws_bytes=nb)), lambda: rows.append(gx[0].clone()),
                      lambda: bias.add_(0.01), lambda: w.sub_(0.03),
                      lambda: hc.check(hc.hc_causal_conv_step(d, x[:, i % L], w, bias, state, step)),
                      lambda: rows.append(step.clone())):
                f()
                after()
        return [sums, state] + rows

    both(run)


# ---------------------------------------------------------------- the temporal mixer

@pytest.fixture(scope="module")
def mixer(hc):
    from spatially_sharded_cnn_gb300.mixer import TemporalMixer
    T, P = 6, 512
    m = TemporalMixer(C=64, D=128, groups=8, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    x, gy = (torch.randn(T, P, 64, device="cuda", generator=g).to(m.dtype) for _ in range(2))
    return m, x, gy


def mixed(m, x, gy):
    y, kept = m.forward(x, train=True)
    gx, g = m.backward(gy, kept)
    states = m.states(x.shape[1])
    rows = torch.stack([m.step(f, states) for f in x])
    return [y, gx, rows, *states] + [g[k] for k in sorted(g)]


def test_mixer_on_a_side_stream(mixer):
    """Training and single frames on a side stream, many in a row, against the default stream."""
    m, x, gy = mixer
    want = mixed(m, x, gy)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [mixed(m, x, gy) for _ in range(20)]
    side.synchronize()
    for one in got:
        for a, b in zip(one, want):
            assert torch.equal(a, b)


def test_mixer_in_a_graph(mixer):
    """A training step and a frame captured from torch's stream, replayed on new values."""
    m, x, gy = mixer
    x, gy = x.clone(), gy.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            mixed(m, x, gy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = mixed(m, x, gy)
    x.copy_(x.flip(0))
    gy.copy_(gy.flip(1))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, mixed(m, x, gy)):
        assert torch.equal(a, b)
