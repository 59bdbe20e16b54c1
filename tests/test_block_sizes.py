"""Workspace sizes of the feed-forward product at the ends of its range (no GPU needed)."""
import pytest


@pytest.fixture(scope="module")
def hc():
    from spatially_sharded_cnn_gb300 import build
    build.build()
    from spatially_sharded_cnn_gb300 import hc as mod
    return mod


MOST = 0x7fffffff - 257


@pytest.mark.parametrize("M,C,F", [(MOST, 8, 8), (MOST, 128, 128), (1 << 22, 1 << 16, 1 << 16), (MOST, 8, 128), (1, 1 << 16, 1 << 16)])
def test_gated_ffn_largest_sizes(hc, M, C, F):
    """h, and [ga | gu] beside it, fit, whatever the tiles of the products."""
    hc.check(hc.hc_set_sm_count(152))
    try:
        for p, n in ((0, 1), (1, 3)):
            st, got = hc.hc_gated_ffn_workspace_size(hc.gated_ffn_desc(M, C, F, hc.HC_DTYPE_BF16), p)
            assert st == hc.HC_OK and n * 2 * M * F <= got < n * 2 * M * F + (1 << 30)
    finally:
        hc.check(hc.hc_set_sm_count(0))


@pytest.mark.parametrize("M,C,F", [(MOST, 1 << 16, 1 << 16), (1 << 30, 1 << 16, 1 << 15), (MOST, 8, 1 << 16), (MOST, 1 << 16, 8),
                                   ((1 << 22) + 1, 1 << 16, 8)])
def test_gated_ffn_beyond_its_sizes(hc, M, C, F):
    """More rows times columns than any memory holds: refused (their tiles were counted past 2^31, and the size that came
    back was below that of h)."""
    for p in (0, 1):
        assert hc.hc_gated_ffn_workspace_size(hc.gated_ffn_desc(M, C, F, hc.HC_DTYPE_BF16), p)[0] == hc.HC_ERR_UNSUPPORTED
