"""What the binding of the mixer operators refuses before the library sees it (no GPU): an array of
another type, size or order, or one in host memory, in the place of each argument that is passed to the
library as an address."""
import pytest
import torch

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


class OnGpu(torch.Tensor):
    """A host tensor that says it is on the GPU: enough for checks that come before any launch."""
    is_cuda = True


def gpu(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)


@pytest.fixture()
def hc(monkeypatch):
    from spatially_sharded_cnn_gb300 import build
    build.build()
    from spatially_sharded_cnn_gb300 import hc as mod

    class Lib:
        """The library, its launching calls replaced by ones that only count."""
        reached = 0

        def __getattr__(self, name):
            if name.endswith("_size") or name.endswith("_string"):
                return getattr(real, name)

            def call(*args):
                Lib.reached += 1
                return 0
            return call
    real = mod._lib
    lib = Lib()
    monkeypatch.setattr(mod, "_lib", lib)
    mod.reached = lambda: Lib.reached
    yield mod
    del mod.reached


def groupnorm(hc, back):
    N, P, C, G = 2, 6, 8, 4
    d = hc.groupnorm_desc(N, P, C, G, BF16)
    rows = lambda: gpu(N, P, C, dtype=BF16)
    a = dict(gamma=gpu(C), beta=gpu(C), mean=gpu(N, G), rstd=gpu(N, G), ws=gpu(4096, dtype=torch.uint8))
    if back:
        a.update(x=rows(), gy=rows(), gx=rows(), ggamma=gpu(C), gbeta=gpu(C))
        return a, lambda k: hc.hc_groupnorm_bwd(d, **k, ws_bytes=4096)
    a.update(x=rows(), y=rows())
    return a, lambda k: hc.hc_groupnorm_fwd(d, **k, ws_bytes=4096)


def conv(hc, form):
    B, L, D, K = 3, 6, 8, 4
    d = hc.causal_conv_desc(B, L, D, K, BF16)
    rows = lambda: gpu(B, L, D, dtype=BF16)
    state = lambda: gpu(B, K - 1, D, dtype=BF16)
    a = dict(w=gpu(D, K), bias=gpu(D))
    if form == "step":
        a.update(x=gpu(B, D, dtype=BF16), y=gpu(B, D, dtype=BF16), state=state())
        return a, lambda k: hc.hc_causal_conv_step(d, **k)
    a.update(x=rows(), state_in=state(), lens=gpu(B, dtype=torch.int32))
    if form == "fwd":
        a.update(y=rows(), state_out=state())
        return a, lambda k: hc.hc_causal_conv_fwd(d, **k)
    a.update(gy=rows(), gx=rows(), gw=gpu(D, K), gb=gpu(D), gstate_out=state(), gstate_in=state(),
             ws=gpu(1 << 16, dtype=torch.uint8))
    return a, lambda k: hc.hc_causal_conv_bwd(d, **k, ws_bytes=1 << 16)


def scan(hc, form):
    B, L, D, G, N = 3, 6, 8, 2, 4
    d = hc.selective_scan_desc(B, L, D, N, BF16, G)
    wide = (B,) if form == "step" else (B, L)
    a = {k: gpu(*wide, D, dtype=BF16) for k in ("u", "dt", "z")}
    a.update({k: gpu(*wide, G * N, dtype=BF16) for k in ("Bm", "Cm")}, A=gpu(D, N), D=gpu(D), dt_bias=gpu(D))
    if form == "step":
        a.update(y=gpu(B, D, dtype=BF16), state=gpu(B, D, N))
        return a, lambda k: hc.hc_selective_scan_step(d, **k)
    a.update(h0=gpu(B, D, N), lens=gpu(B, dtype=torch.int32), ws=gpu(1 << 16, dtype=torch.uint8),
             saved=gpu(hc.hc_selective_scan_saved_size(d)[1], dtype=torch.uint8))
    if form == "fwd":
        a.update(y=gpu(B, L, D, dtype=BF16), hT=gpu(B, D, N))
        return a, lambda k: hc.hc_selective_scan_fwd(d, **k, ws_bytes=1 << 16)
    a.update({"g" + k: gpu(B, L, D, dtype=BF16) for k in ("u", "dt", "z", "y")})
    a.update({k: gpu(B, L, G * N, dtype=BF16) for k in ("gB", "gC")}, gA=gpu(D, N), gD=gpu(D), gdt_bias=gpu(D),
             ghT=gpu(B, D, N), gh0=gpu(B, D, N))
    return a, lambda k: hc.hc_selective_scan_bwd(d, **k, ws_bytes=1 << 16)


ROWS = {"x", "y", "gy", "gx", "u", "dt", "z", "Bm", "Cm", "gu", "gdt", "gz", "gB", "gC"}  # the library checks their type
FORMS = [(groupnorm, False), (groupnorm, True), (conv, "fwd"), (conv, "bwd"), (conv, "step"), (scan, "fwd"), (scan, "bwd"),
         (scan, "step")]


@pytest.mark.parametrize("op,form", FORMS)
def test_arrays_of_another_kind_are_refused(hc, op, form):
    args, call = op(hc, form)
    assert call(args) == 0 and hc.reached() == 1

    def refused(why, **bad):
        with pytest.raises(hc.HcError) as e:
            call(dict(args, **bad))
        assert e.value.status == hc.HC_ERR_INVALID_ARG, why
        assert hc.reached() == 1, f"{why}: reached the library"

    for name, t in args.items():
        refused(f"{name} in host memory", **{name: t.as_subclass(torch.Tensor)})
        if name in ("ws", "saved"):
            refused(f"{name} too short", **{name: t[:-1]})
            continue
        if name not in ROWS:
            refused(f"{name} of another type", **{name: t.to(F16)})
        refused(f"{name} too short", **{name: t[:-1]})
        refused(f"{name} too long", **{name: torch.cat([t, t]).as_subclass(OnGpu)})
        if t.dim() > 1 and t.shape[-1] > 1:
            refused(f"{name} in another order", **{name: t.transpose(-1, -2).contiguous().transpose(-1, -2)})
        else:
            refused(f"{name} with gaps", **{name: torch.stack([t, t], -1).as_subclass(OnGpu)[..., 0]})


@pytest.mark.parametrize("op,form", FORMS)
def test_arrays_of_any_shape_and_addresses_are_taken(hc, op, form):
    """A convolution's weights may be (D, 1, K); parameters may be given as addresses."""
    args, call = op(hc, form)
    flat = {k: t.reshape(1, -1) for k, t in args.items() if t.dtype == F32}
    assert call(dict(args, **flat)) == 0
    assert call(dict(args, **{k: t.data_ptr() for k, t in flat.items()})) == 0


@pytest.mark.parametrize("op,form", FORMS)
def test_absent_tensors_reach_the_library(hc, op, form):
    """Which of them may be absent, and when, is the library's to say."""
    args, call = op(hc, form)
    for i, name in enumerate(args):
        assert call(dict(args, **{name: None})) == 0, name
        assert hc.reached() == i + 1
