"""Where the mixer operators' rounding shows, against 64 bits: bounds derived from the formats, beside
each test."""
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
