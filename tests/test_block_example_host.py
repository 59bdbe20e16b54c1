"""The host side of the sequence block (no GPU): which stream and device its library calls go to, with the
library's calls replaced by ones that take note of it."""
import contextlib
import inspect

import pytest
import torch

CALLS = ("hc_layernorm_fwd", "hc_layernorm_bwd", "hc_linear_attn_fwd", "hc_linear_attn_bwd", "hc_linear_attn_step",
         "hc_gated_ffn_fwd", "hc_gated_ffn_bwd")


@pytest.fixture()
def mod():
    from spatially_sharded_cnn_gb300 import build
    build.build()
    from spatially_sharded_cnn_gb300 import block
    return block


def test_library_calls_take_torchs_stream_and_the_blocks_device(mod, monkeypatch):
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
    m = mod.AttentionBlock(C=16, H=2, F=24, device="cpu")
    x = torch.zeros(5, 6, 16, dtype=torch.bfloat16)
    _, kept = m.forward(x, train=True)
    m.backward(x, kept)
    m.forward(x)
    m.step(x[0], m.states(6))
    assert {s[0] for s in seen} == set(CALLS)
    for name, stream, on in seen:
        assert stream is current, f"{name} is not on torch's current stream"
        assert on == ["cpu"], f"{name} is not on the block's device"
    assert {str(d) for d in asked} == {"cpu"}
