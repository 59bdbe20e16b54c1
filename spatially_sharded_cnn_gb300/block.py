"""A sequence block over a camera stream's feature maps: layer norm, linear attention, layer norm and a gated
feed-forward product, each half added to its input.

The maps are frames (T, P, C): T frames of P pixels.  Every pixel's sequence of frames runs through linear attention
with a decay for each head (the pixels are its batch: their sequences are read in place as strided rows of the maps,
(P, T, C) views of (T, P, C) tensors); norm and feed-forward product take each pixel of each frame alone.

``forward`` / ``backward`` train on T frames at once, ``step`` takes one new frame and the carried states (a matrix a
head and pixel) and gives the row that ``forward`` would.  The operators are the library's kernels; torch holds the
memory and multiplies by the projections of q, k, v and of the attention's rows.  Both run on torch's current stream,
which may be a side stream or one that a CUDA graph captures.

    python -m spatially_sharded_cnn_gb300.block      # a training step and a stream, timed
"""
from __future__ import annotations

import time

import torch

from . import hc
from .mixer import _on_device


class AttentionBlock:
    def __init__(self, C=256, H=4, F=704, dtype=torch.bfloat16, act=hc.HC_PW_SILU, seed=0, device="cuda"):
        """C channels in H heads, F hidden values; dtype bfloat16 or float16."""
        g = torch.Generator().manual_seed(seed)
        self.C, self.H, self.F, self.dtype, self.act, self.device = C, H, F, dtype, act, device
        self.D = C // H

        def normal(*shape, to=torch.float32):
            return (torch.randn(*shape, generator=g) * shape[0] ** -0.5).to(device=device, dtype=to)

        one = lambda v: torch.full((C,), v, device=device)
        self.p = dict(gamma1=one(1.0), beta1=one(0.0), w_qkv=normal(C, 3 * C, to=dtype),
                      # heads that remember from 8 frames to about 1000
                      log_decay=torch.log1p(-torch.exp2(-3.0 - 7.0 * torch.arange(H) / max(H - 1, 1))).to(device),
                      w_o=normal(C, C, to=dtype), gamma2=one(1.0), beta2=one(0.0), w_in=normal(C, 2 * F, to=dtype),
                      w_out=normal(F, C, to=dtype))

    def _space(self, got):
        hc.check(got[0], "size")
        return torch.empty(max(got[1], 16), dtype=torch.uint8, device=self.device), got[1]

    def _empty(self, *shape, dtype=None):
        return torch.empty(*shape, dtype=dtype or self.dtype, device=self.device)

    def _stream(self):
        return torch.cuda.current_stream(self.device)

    def _norm(self, x, which, keep):
        T, P, C = x.shape
        d = hc.layernorm_desc(T, P, C, self.dtype)
        y = torch.empty_like(x)
        mean, rstd = (self._empty(T, P, dtype=torch.float32) for _ in range(2)) if keep else (None, None)
        hc.check(hc.hc_layernorm_fwd(d, x, self.p["gamma" + which], self.p["beta" + which], y, mean, rstd,
                                     stream=self._stream()), "norm")
        return y, (d, x, mean, rstd)

    def _norm_back(self, kept, which, gy, g):
        d, x, mean, rstd = kept
        gx = torch.empty_like(x)
        g["gamma" + which], g["beta" + which] = (self._empty(self.C, dtype=torch.float32) for _ in range(2))
        ws, nb = self._space(hc.hc_layernorm_workspace_size(d))
        hc.check(hc.hc_layernorm_bwd(d, x, self.p["gamma" + which], mean, rstd, gy, gx, g["gamma" + which],
                                     g["beta" + which], ws=ws, ws_bytes=nb, stream=self._stream()), "norm backward")
        return gx

    def _qkv(self, rows):
        C = self.C
        return rows[..., :C], rows[..., C:2 * C], rows[..., 2 * C:]

    def _ffn(self, x, train):
        d = hc.gated_ffn_desc(x.shape[0], self.C, self.F, self.dtype, self.act)
        ws, nb = self._space(hc.hc_gated_ffn_workspace_size(d, int(train)))
        y = torch.empty_like(x)
        hc.check(hc.hc_gated_ffn_fwd(d, x, self.p["w_in"], self.p["w_out"], y, ws, nb, self._stream()), "feed-forward")
        return y, (d, ws, nb)

    @_on_device
    def forward(self, x, train=False):
        """x (T, P, C) -> (T, P, C); with `train`, also what `backward` needs."""
        T, P, C = x.shape
        seq = lambda t: t.transpose(0, 1)  # (T, P, .) -> (P, T, .), in place
        n1, norm1 = self._norm(x, "1", train)
        qkv = n1 @ self.p["w_qkv"]
        d = hc.linear_attn_desc(P, T, self.H, self.D, self.D, self.dtype)
        ws, nb = self._space(hc.hc_linear_attn_workspace_size(d, int(train)))
        s = self._empty(T, P, C)
        hc.check(hc.hc_linear_attn_fwd(d, *self._qkv(seq(qkv)), seq(s), self.p["log_decay"], ws=ws, ws_bytes=nb,
                                       stream=self._stream()), "attention")
        y1 = x + s @ self.p["w_o"]
        n2, norm2 = self._norm(y1, "2", train)
        f, ffn = self._ffn(n2.reshape(T * P, C), train)
        y = y1 + f.view(T, P, C)
        return (y, (norm1, n1, qkv, d, ws, nb, s, norm2, n2, ffn)) if train else y

    @_on_device
    def backward(self, gy, kept):
        """The gradients of x and of every parameter but the decays, from the gradient of forward's result."""
        norm1, n1, qkv, d, ws, nb, s, norm2, n2, (df, wf, nf) = kept
        T, P, C = n1.shape
        p, g = self.p, {}
        seq = lambda t: t.transpose(0, 1)
        flat = lambda t: t.reshape(T * P, -1)
        g["w_in"], g["w_out"], gn = torch.empty_like(p["w_in"]), torch.empty_like(p["w_out"]), self._empty(T * P, C)
        hc.check(hc.hc_gated_ffn_bwd(df, flat(n2), p["w_in"], p["w_out"], flat(gy), gn, g["w_in"], g["w_out"], wf, nf,
                                     self._stream()), "feed-forward backward")
        gy = gy + self._norm_back(norm2, "2", gn.view(T, P, C), g)
        g["w_o"] = flat(s).T @ flat(gy)
        gs, gqkv = gy @ p["w_o"].T, torch.empty_like(qkv)
        hc.check(hc.hc_linear_attn_bwd(d, *self._qkv(seq(qkv)), seq(gs), *self._qkv(seq(gqkv)), p["log_decay"], ws=ws,
                                       ws_bytes=nb, stream=self._stream()), "attention backward")
        g["w_qkv"] = flat(n1).T @ flat(gqkv)
        return gy + self._norm_back(norm1, "1", gqkv @ p["w_qkv"].T, g), g

    def states(self, P):
        """A new stream's carried states: zeros."""
        return torch.zeros(P, self.H, self.D, self.D, device=self.device)

    @_on_device
    def step(self, x, states):
        """One frame x (P, C) -> (P, C); the states move on in place."""
        P, C = x.shape
        n1, _ = self._norm(x[None], "1", False)
        qkv = n1[0] @ self.p["w_qkv"]
        s = self._empty(P, C)
        d = hc.linear_attn_desc(P, 1, self.H, self.D, self.D, self.dtype)
        hc.check(hc.hc_linear_attn_step(d, *self._qkv(qkv), states, s, self.p["log_decay"], stream=self._stream()),
                 "attention step")
        y1 = x + s @ self.p["w_o"]
        n2, _ = self._norm(y1[None], "2", False)
        return y1 + self._ffn(n2[0], False)[0]


def main() -> None:
    T, P, C = 16, 32 * 64, 256
    m = AttentionBlock(C=C)
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
        _, kept = m.forward(x, train=True)
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
