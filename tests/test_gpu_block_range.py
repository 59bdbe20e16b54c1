"""The feed-forward product where h or the gradients of a and u leave the range of fp16: what include/hc_block.h says of it."""
import pytest
import torch

import block_ref as R
from test_gpu_mixer import ROUND, near, space

pytestmark = pytest.mark.gpu
n64 = lambda t: t.double().cpu().numpy()


@pytest.fixture(scope="module")
def hc():
    assert torch.cuda.is_available()
    from spatially_sharded_cnn_gb300 import build
    build.build()
    from spatially_sharded_cnn_gb300 import hc as mod
    return mod


@pytest.mark.parametrize("M", [6, 300, 3000])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_gated_ffn_range(hc, dtype, M):
    """a = u = 300 in one row: h = 90000.  bf16 holds it; in fp16 that row of y alone is not finite (and of the
    gradients that of its x, and those of the weights that it enters)."""
    C, F, bad = 64, 64, M // 2
    g = torch.Generator().manual_seed(31)
    x = torch.randn(M, C, generator=g) * 0.5
    w_in, w_out = torch.zeros(C, 2 * F), torch.randn(F, C, generator=g) * 2.0 ** -8
    for j in range(F):  # column j of a and of u is channel j of x
        w_in[j, j] = w_in[j, F + j] = 1.0
    x[bad, 5] = 300.0
    gy = torch.randn(M, C, generator=g)
    x, w_in, w_out, gy = (t.to(dtype).cuda() for t in (x, w_in, w_out, gy))
    d = hc.gated_ffn_desc(M, C, F, dtype, hc.HC_PW_NONE)
    y, gx = torch.empty_like(x), torch.empty_like(x)
    ws, nb = space(hc, hc.hc_gated_ffn_workspace_size(d, 1))
    hc.check(hc.hc_gated_ffn_fwd(d, x, w_in, w_out, y, ws, nb))
    gwi, gwo = torch.empty_like(w_in), torch.empty_like(w_out)
    hc.check(hc.hc_gated_ffn_bwd(d, x, w_in, w_out, gy, gx, gwi, gwo, ws, nb))
    ref = R.gated_ffn(n64(x), n64(w_in), n64(w_out), "none", n64(gy))
    rest = [i for i in range(M) if i != bad]
    near("y", y[rest], ref["y"][rest], 1e-5 + ROUND[dtype])
    near("gx", gx[rest], ref["gx"][rest], 1e-5 + ROUND[dtype])
    if dtype == torch.bfloat16:
        near("y", y, ref["y"], 1e-5 + ROUND[dtype])
    else:
        assert abs(ref["y"][bad]).max() < 65504 and not torch.isfinite(y[bad]).any()
        finite = torch.isfinite(gwo)
        assert not finite[5].any() and finite[:5].all() and finite[6:].all()
        near("gx", gx, ref["gx"], 1e-5 + ROUND[dtype])  # ga = gh u is in range here
