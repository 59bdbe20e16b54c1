"""Where the mixer operators' rounding shows, against 64 bits: bounds derived from the formats, beside
each test."""
import math

import numpy as np
import pytest
import torch

from test_gpu_mixer import space

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hc():
    assert torch.cuda.is_available()
    from spatially_sharded_cnn_gb300 import build
    build.build()
    from spatially_sharded_cnn_gb300 import hc as mod
    return mod


@pytest.mark.parametrize("P,C,G", [(17000, 1024, 32), (200000, 128, 8), (4096, 32, 4)])
def test_groupnorm_mean_under_a_large_offset(hc, P, C, G):
    """A common offset of 1000 standard deviations, maps that take three launches and one.  Means of chunks are rounded to
    fp32 and so is the mean of all: each by half a unit in the last place of a value below 1024, 2^-15, so 2^-14 in all.
    The sums of offsets, 1e-7 of a value of the size of a standard deviation each, add less than 1e-6."""
    g = torch.Generator(device="cuda").manual_seed(60)
    x = torch.randn(1, P, C, device="cuda", generator=g) + 1000.0
    gamma, beta = torch.ones(C, device="cuda"), torch.zeros(C, device="cuda")
    d = hc.groupnorm_desc(1, P, C, G, torch.float32)
    ws, nb = space(hc, hc.hc_groupnorm_workspace_size(d, 0))
    y, mean, rstd = torch.empty_like(x), torch.empty(1, G, device="cuda"), torch.empty(1, G, device="cuda")
    hc.hc_trace_collect()
    hc.hc_trace_enable(True)
    hc.check(hc.hc_groupnorm_fwd(d, x, gamma, beta, y, mean, rstd, ws, nb))
    hc.hc_trace_enable(False)
    assert ("gn_combine_kernel" in hc.hc_trace_collect()[1]) == (P > 4096)
    ref = x.double().view(P, G, C // G).mean((0, 2)).cpu().numpy()
    assert np.abs(mean[0].double().cpu().numpy() - ref).max() <= 2.0 ** -14 + 1e-6


def test_groupnorm_sums_of_one_channel(hc):
    """The sums of a block whose 256 rows of threads all have the same channel.  Adding m values of spread s in order leaves
    0.29 * m * 2^-24 * s (rms: sum k is off by 0.4 units of its own size sqrt(k) s).  512 values, two a thread, in sixteen
    runs of sixteen rows and then the runs: 16 runs of 0.29 * 16 * sqrt(2) and one of 0.29 * 16 * sqrt(32), 37 in all;
    the values' own rounding 23.  In one run of 256 the sum alone would leave 105.  Held to 75 over 60 inputs."""
    P, off, spread = 512, [], []
    one, zero = torch.ones(4, device="cuda")[:1], torch.zeros(4, device="cuda")[:1]
    d = hc.groupnorm_desc(1, P, 1, 1, torch.float32)
    ws, nb = space(hc, hc.hc_groupnorm_workspace_size(d, 1))
    g = torch.Generator(device="cuda").manual_seed(64)
    for _ in range(60):
        x, gy = (torch.randn(1, P, 1, device="cuda", generator=g) for _ in range(2))
        y, gx = torch.empty_like(x), torch.empty_like(x)
        mean, rstd = torch.empty(1, 1, device="cuda"), torch.empty(1, 1, device="cuda")
        gg, gb = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
        hc.check(hc.hc_groupnorm_fwd(d, x, one, zero, y, mean, rstd, ws, nb))
        hc.check(hc.hc_groupnorm_bwd(d, x, one, zero, mean, rstd, gy, gx, gg, gb, ws, nb))
        t = gy.double() * (x.double() - mean.double()) * rstd.double()
        off.append(float(gg.double() - t.sum()))
        spread.append(float(t.square().mean().sqrt()))
    assert np.sqrt(np.mean(np.square(off))) <= 75 * 2.0 ** -24 * np.mean(spread)


def gelu_of(hc, v):
    """GELU and its slope at v through the norm (gamma 0, beta v: the activation's argument is v), and by the library's
    elementwise calls (the form with erff)."""
    C = v.numel()
    x, z = torch.randn(1, 2, C, device="cuda", generator=torch.Generator(device="cuda").manual_seed(61)), torch.zeros_like(v)
    d = hc.groupnorm_desc(1, 2, C, C // 16, torch.float32, act=hc.HC_PW_GELU)
    ws, nb = space(hc, hc.hc_groupnorm_workspace_size(d, 1))
    y, gx, one = torch.empty_like(x), torch.empty_like(x), torch.ones_like(x)
    mean, rstd = torch.empty(1, C // 16, device="cuda"), torch.empty(1, C // 16, device="cuda")
    gg, gb, ey, es = (torch.empty_like(v) for _ in range(4))
    hc.check(hc.hc_groupnorm_fwd(d, x, z, v, y, mean, rstd, ws, nb))
    hc.check(hc.hc_groupnorm_bwd(d, x, z, v, mean, rstd, one, gx, gg, gb, ws, nb))
    hc.check(hc.hc_gelu_fwd(C, v, ey))
    hc.check(hc.hc_gelu_bwd(C, v, torch.ones_like(v), es))
    torch.cuda.synchronize()
    vd = v.double()
    cdf = torch.special.ndtr(vd)
    return (y[0, 0], gb / 2, ey, es), (vd * cdf, cdf + vd * torch.exp(-0.5 * vd * vd) / math.sqrt(2 * math.pi))


def test_gelu_is_as_accurate_as_the_error_function_form(hc):
    """rms errors over 65536 normal values, a sample's rms being within a few per cent of the distribution's: at most a
    quarter above those of the plain fp32 form."""
    v = torch.randn(1 << 16, device="cuda", generator=torch.Generator(device="cuda").manual_seed(62))
    (y, slope, ey, es), (ref, sref) = gelu_of(hc, v)
    rms = lambda a, b: float((a.double() - b).square().mean().sqrt())
    assert rms(y, ref) <= 1.25 * rms(ey, ref)
    assert rms(slope, sref) <= 1.25 * rms(es, sref)


def test_gelu_far_from_zero(hc):
    """The negative tail to a relative 1e-5: exp(-x^2 / 2)'s argument, up to 18 at -5, is rounded twice (2e-6), the scaled
    function, 0.08 there, is off by a few roundings below 0.5 (1e-6 to 2e-6).  Beyond the format's range: 0 and x."""
    v = torch.cat([torch.linspace(-5, -1, 4080, device="cuda"), torch.linspace(-40, 40, 16, device="cuda")])
    (y, slope, _, _), (ref, sref) = gelu_of(hc, v)
    assert ((y.double() - ref).abs() <= 1e-5 * ref.abs())[:4080].all()
    assert ((y.double() - ref).abs()[4080:] <= 1e-6 * v.abs().double()[4080:]).all()
    assert ((slope.double() - sref).abs() <= 1e-6).all()
    assert torch.isinf(gelu_of(hc, torch.full((16,), float("inf"), device="cuda"))[0][0]).all()


@pytest.mark.parametrize("sms", [1, 0])
def test_slow_states_keep_their_decay(hc, sms):
    """A state that only decays, over 4096 rows with steps of a third to all of 3e-7 ... 1e-2 (times log2 e), uncut and cut
    into segments.  A row's decay is off by 1.2e-8 on average where that is above 3e-7, by 2e-8 below, the same way in every
    row, and by 5e-8 (rms) at random; the state's own rounding adds 3e-8 (rms)."""
    B, L, N, t = 4, 4096, 4, torch.float32
    tops = 10.0 ** np.arange(-6.5, -1.99, 0.25)
    D = tops.size
    r = np.random.default_rng(63)
    dt = torch.from_numpy(tops * r.uniform(1 / 3, 1, size=(B, L, D)) / math.log2(math.e)).float().cuda()
    zero, y, hT = torch.zeros(B, L, D, device="cuda"), torch.empty(B, L, D, device="cuda"), torch.empty(B, D, N, device="cuda")
    Bm = torch.zeros(B, L, N, device="cuda")
    A = -torch.ones(D, N, device="cuda")
    h0 = torch.ones(B, D, N, device="cuda")
    hc.check(hc.hc_set_sm_count(sms))
    try:
        d = hc.selective_scan_desc(B, L, D, N, t, softplus=0)
        ws, nb = space(hc, hc.hc_selective_scan_workspace_size(d, 0))
        hc.check(hc.hc_selective_scan_fwd(d, zero, dt, A, Bm, Bm, y, h0=h0, hT=hT, ws=ws, ws_bytes=nb))
        torch.cuda.synchronize()
    finally:
        hc.check(hc.hc_set_sm_count(0))
    want = torch.exp(-dt.double().sum(1))[..., None]
    off = ((hT.double() - want) / want).abs().amax((0, 2)).cpu().numpy()
    mean = np.where(tops > 6e-7, 1.2e-8, 2e-8)
    assert (off <= mean * L + 5 * math.hypot(5e-8, 3e-8) * math.sqrt(L)).all(), off
