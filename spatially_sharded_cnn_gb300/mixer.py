"""A temporal mixer over a camera stream's feature maps, built from the channels-last operators.

The maps are frames (T, P, C): T frames of P pixels.  Each frame is normalised over its pixels
(group norm + SiLU), projected to a branch and a gate, and every pixel's sequence of frames runs
through a short causal convolution and a selective scan; the gated result is projected back and
added to the input.  The pixels are the scan's batch: their sequences are read in place as strided
rows of the maps, (P, T, D) views of (T, P, D) tensors.

``forward`` / ``backward`` train on T frames at once, ``step`` takes one new frame and the carried
states (a K - 1 row window and a D x N state a pixel) and gives the row that ``forward`` would.
The operators are the library's kernels; torch holds the memory and multiplies by the projections.
Both run on torch's current stream, which may be a side stream or one that a CUDA graph captures.

    python -m spatially_sharded_cnn_gb300.mixer      # a training step and a stream, timed
"""
from __future__ import annotations

import functools
import math
import time

import torch

from . import hc


def _on_device(method):
    """Runs a method with the mixer's device as the current one: the library launches on the current device."""
    @functools.wraps(method)
    def run(self, *args, **kwargs):
        with torch.cuda.device(self.device):
            return method(self, *args, **kwargs)
    return run


class TemporalMixer:
    def __init__(self, C=256, D=512, K=4, N=16, groups=32, dtype=torch.bfloat16, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.C, self.D, self.K, self.N, self.groups, self.dtype, self.device = C, D, K, N, groups, dtype, device
        self.R = max(1, D // 16)

        def normal(*shape, scale, shift=0.0, to=torch.float32):
            return (torch.randn(*shape, generator=g) * scale + shift).to(device=device, dtype=to)

        step = torch.exp(torch.rand(D, generator=g) * math.log(100.0) + math.log(1e-3))
        self.p = dict(
            gamma=normal(C, scale=0.0, shift=1.0), beta=normal(C, scale=0.0),
            w_in=normal(C, 2 * D, scale=C ** -0.5, to=dtype), conv=normal(D, K, scale=K ** -0.5),
            conv_bias=normal(D, scale=0.0), w_x=normal(D, self.R + 2 * N, scale=D ** -0.5, to=dtype),
            w_dt=normal(self.R, D, scale=self.R ** -0.5, to=dtype),
            dt_bias=(step + torch.log(-torch.expm1(-step))).to(device),
            A=-torch.arange(1, N + 1, dtype=torch.float32, device=device).repeat(D, 1).contiguous(),
            D=torch.ones(D, device=device), w_out=normal(D, C, scale=D ** -0.5, to=dtype))

    def _space(self, got):
        hc.check(got[0], "size")
        return torch.empty(max(got[1], 16), dtype=torch.uint8, device=self.device), got[1]

    def _empty(self, *shape, dtype=None):
        return torch.empty(*shape, dtype=dtype or self.dtype, device=self.device)

    def _stream(self):
        """The stream of the library's calls: the one that torch's products before and after them are on."""
        return torch.cuda.current_stream(self.device)

    def _norm(self, x, keep):
        T, P, C = x.shape
        d = hc.groupnorm_desc(T, P, C, self.groups, self.dtype, act=hc.HC_PW_SILU)
        ws, nb = self._space(hc.hc_groupnorm_workspace_size(d, int(keep)))
        y = torch.empty_like(x)
        mean, rstd = (self._empty(T, self.groups, dtype=torch.float32) for _ in range(2)) if keep else (None, None)
        hc.check(hc.hc_groupnorm_fwd(d, x, self.p["gamma"], self.p["beta"], y, mean, rstd, ws, nb, self._stream()),
                 "norm")
        return y, (d, mean, rstd, ws, nb)

    def _project(self, c):
        proj = c @ self.p["w_x"]
        R, N = self.R, self.N
        return proj, proj[..., :R] @ self.p["w_dt"], proj[..., R:R + N], proj[..., R + N:]

    @_on_device
    def forward(self, x, train=False):
        """x (T, P, C) -> (T, P, C); with `train`, also what `backward` needs."""
        T, P, _ = x.shape
        D, p = self.D, self.p
        n, norm = self._norm(x, train)
        xz = n @ p["w_in"]
        seq = lambda t: t.transpose(0, 1)  # (T, P, .) -> (P, T, .), in place
        dc = hc.causal_conv_desc(P, T, D, self.K, self.dtype, hc.HC_PW_SILU)
        c = self._empty(T, P, D)
        hc.check(hc.hc_causal_conv_fwd(dc, seq(xz)[..., :D], p["conv"], p["conv_bias"], seq(c), stream=self._stream()), "conv")
        proj, dt, Bm, Cm = self._project(c)
        ds = hc.selective_scan_desc(P, T, D, self.N, self.dtype)
        ws, nb = self._space(hc.hc_selective_scan_workspace_size(ds, int(train)))
        saved = self._space(hc.hc_selective_scan_saved_size(ds))[0] if train else None
        s = self._empty(T, P, D)
        hc.check(hc.hc_selective_scan_fwd(ds, seq(c), seq(dt), p["A"], seq(Bm), seq(Cm), seq(s), D=p["D"],
                                          z=seq(xz)[..., D:], dt_bias=p["dt_bias"], saved=saved, ws=ws, ws_bytes=nb,
                                          stream=self._stream()), "scan")
        y = x + s @ p["w_out"]
        return (y, (x, n, norm, xz, dc, c, proj, dt, Bm, Cm, ds, ws, nb, saved, s)) if train else y

    @_on_device
    def backward(self, gy, kept):
        """The gradients of every parameter, and of x, from the gradient of forward's result."""
        x, n, (dn, mean, rstd, nws, nnb), xz, dc, c, proj, dt, Bm, Cm, ds, ws, nb, saved, s = kept
        T, P, _ = x.shape
        D, N, R, p = self.D, self.N, self.R, self.p
        seq = lambda t: t.transpose(0, 1)
        flat = lambda t: t.reshape(T * P, -1)
        f32 = lambda *shape: self._empty(*shape, dtype=torch.float32)
        g = dict(w_out=flat(s).T @ flat(gy))
        gs = gy @ p["w_out"].T
        gxz, gproj = torch.empty_like(xz), torch.empty_like(proj)
        gc, gdt = self._empty(T, P, D), self._empty(T, P, D)
        g["A"], g["D"], g["dt_bias"] = f32(D, N), f32(D), f32(D)
        hc.check(hc.hc_selective_scan_bwd(ds, seq(c), seq(dt), p["A"], seq(Bm), seq(Cm), seq(gs), saved, seq(gc), seq(gdt),
                                          g["A"], seq(gproj)[..., R:R + N], seq(gproj)[..., R + N:], D=p["D"],
                                          z=seq(xz)[..., D:], dt_bias=p["dt_bias"], gD=g["D"], gz=seq(gxz)[..., D:],
                                          gdt_bias=g["dt_bias"], ws=ws, ws_bytes=nb, stream=self._stream()), "scan backward")
        g["w_dt"] = flat(proj[..., :R]).T @ flat(gdt)
        gproj[..., :R] = gdt @ p["w_dt"].T
        g["w_x"] = flat(c).T @ flat(gproj)
        gc += gproj @ p["w_x"].T
        g["conv"], g["conv_bias"] = f32(D, self.K), f32(D)
        cws, cnb = self._space(hc.hc_causal_conv_workspace_size(dc))
        hc.check(hc.hc_causal_conv_bwd(dc, seq(xz)[..., :D], p["conv"], p["conv_bias"], seq(gc), seq(gxz)[..., :D],
                                       g["conv"], g["conv_bias"], ws=cws, ws_bytes=cnb, stream=self._stream()),
                 "conv backward")
        g["w_in"] = flat(n).T @ flat(gxz)
        gn, gx = gxz @ p["w_in"].T, torch.empty_like(x)
        g["gamma"], g["beta"] = f32(self.C), f32(self.C)
        hc.check(hc.hc_groupnorm_bwd(dn, x, p["gamma"], p["beta"], mean, rstd, gn, gx, g["gamma"], g["beta"], nws, nnb,
                                     self._stream()), "norm backward")
        return gx + gy, g

    def states(self, P):
        """A new stream's carried states: zeros."""
        return (torch.zeros(P, self.K - 1, self.D, dtype=self.dtype, device=self.device),
                torch.zeros(P, self.D, self.N, device=self.device))

    @_on_device
    def step(self, x, states):
        """One frame x (P, C) -> (P, C); the states move on in place."""
        P, D, p = x.shape[0], self.D, self.p
        n, _ = self._norm(x[None], False)
        xz = n[0] @ p["w_in"]
        dc, ds = (hc.causal_conv_desc(P, 1, D, self.K, self.dtype, hc.HC_PW_SILU),
                  hc.selective_scan_desc(P, 1, D, self.N, self.dtype))
        c, s = self._empty(P, D), self._empty(P, D)
        st = self._stream()
        hc.check(hc.hc_causal_conv_step(dc, xz[:, :D], p["conv"], p["conv_bias"], states[0], c, st), "conv step")
        _, dt, Bm, Cm = self._project(c)
        hc.check(hc.hc_selective_scan_step(ds, c, dt, p["A"], Bm, Cm, states[1], s, D=p["D"], z=xz[:, D:],
                                           dt_bias=p["dt_bias"], stream=st), "scan step")
        return x + s @ p["w_out"]


def main() -> None:
    T, P, C = 16, 32 * 64, 256
    m = TemporalMixer(C=C)
    x = torch.randn(T, P, C, device="cuda").to(m.dtype)
    gy = torch.randn(T, P, C, device="cuda").to(m.dtype)

    def timed(f, reps=20):
        f()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(reps):
            f()
        torch.cuda.synchronize()
        return (time.perf_counter() - t) / reps * 1e3

    def train():
        y, kept = m.forward(x, train=True)
        m.backward(gy, kept)

    states = m.states(P)
    print(f"{T} frames of {P} pixels, {C} channels: forward {timed(lambda: m.forward(x)):.3f} ms, "
          f"training step {timed(train):.3f} ms, one frame of a stream {timed(lambda: m.step(x[0], states)):.3f} ms")
    states, y = m.states(P), m.forward(x).float()
    rows = torch.stack([m.step(x[t], states) for t in range(T)]).float()
    print(f"stream against the frames at once: largest difference {float((rows - y).abs().max()):.3g} "
          f"of values up to {float(y.abs().max()):.3g}")


if __name__ == "__main__":
    main()
