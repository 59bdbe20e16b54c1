"""The mixer operators' calls one right after another: each kernel may start while the one before it
in the stream ends, and has to see everything that one wrote.  The same calls with a wait after each
give the same bits."""
import pytest
import torch

from test_gpu_mixer import scan_data

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
