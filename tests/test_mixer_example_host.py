"""The host side of the temporal mixer (no GPU): which stream and device its library calls go to, with
the library's calls replaced by ones that take note of it."""
import contextlib
import inspect

import pytest
import torch

CALLS = ("hc_groupnorm_fwd", "hc_groupnorm_bwd", "hc_causal_conv_fwd", "hc_causal_conv_bwd", "hc_causal_conv_step",
         "hc_selective_scan_fwd", "hc_selective_scan_bwd", "hc_selective_scan_step")


@pytest.fixture()
def mod(monkeypatch):
    from spatially_sharded_cnn_gb300 import build
    build.build()
    from spatially_sharded_cnn_gb300 import mixer
    return mixer


def test_library_calls_take_torchs_stream_and_the_mixers_device(mod, monkeypatch):
    seen, asked, current, entered = [], [], object(), []

    @contextlib.contextmanager
    def device(d):
        entered.append(str(d))
        yield
        entered.pop()

    monkeypatch.setattr(torch.cuda, "device", device)

    def note(name, real):
        where = inspect.signature(real)

        def call(*a, **k):
            seen.append((name, where.bind(*a, **k).arguments.get("stream"), list(entered)))
            return 0
        return call

    for name in CALLS:
        monkeypatch.setattr(mod.hc, name, note(name, getattr(mod.hc, name)))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: asked.append(device) or current)
    m = mod.TemporalMixer(C=8, D=12, K=3, N=4, groups=4, dtype=torch.float32, device="cpu")
    x = torch.zeros(5, 6, 8)
    _, kept = m.forward(x, train=True)
    m.backward(x, kept)
    m.forward(x)
    m.step(x[0], m.states(6))
    assert {s[0] for s in seen} == set(CALLS)
    for name, stream, on in seen:
        assert stream is current, f"{name} is not on torch's current stream"
        assert on == ["cpu"], f"{name} is not on the mixer's device"
    assert {str(d) for d in asked} == {"cpu"}  # the mixer's own device
