"""The operators of a channels-last sequence block in 64 bits on the host: numpy, one row after
another, written from the formulas of include/hc_block.h.  Rows past a sequence's length are left out
by construction, whatever they hold."""
from __future__ import annotations

import numpy as np

from mixer_ref import act, slope


def layernorm(x, gamma, beta, eps, lens=None, gy=None):
    """x (B, L, C) float64 -> dict of y, mean, rstd and, with gy, gx, ggamma, gbeta."""
    B, L, C = x.shape
    out = dict(y=np.zeros_like(x), mean=np.zeros((B, L)), rstd=np.zeros((B, L)))
    if gy is not None:
        out.update(gx=np.zeros_like(x), ggamma=np.zeros(C), gbeta=np.zeros(C))
    for b in range(B):
        for t in range(L if lens is None else int(lens[b])):
            v = x[b, t]
            m = v.mean()
            r = 1 / np.sqrt(((v - m) ** 2).mean() + eps)
            xh = (v - m) * r
            out["mean"][b, t], out["rstd"][b, t] = m, r
            out["y"][b, t] = gamma * xh + beta
            if gy is not None:
                g = gy[b, t]
                q = gamma * g
                out["ggamma"] += g * xh
                out["gbeta"] += g
                out["gx"][b, t] = r * (q - q.mean() - xh * (q * xh).mean())
    return out


def linear_attn(q, k, v, H, scale, decay=None, h0=None, lens=None, gy=None, ghT=None):
    """q, k (B, L, H * Dk), v (B, L, H * Dv); decay (H,) log decays; h0, ghT (B, H, Dk, Dv)."""
    B, L, _ = q.shape
    Dk, Dv = q.shape[2] // H, v.shape[2] // H
    lam = np.ones(H) if decay is None else np.exp(decay)
    out = dict(y=np.zeros_like(v), state=np.zeros((B, H, Dk, Dv)))
    if gy is not None:
        out.update(gq=np.zeros_like(q), gk=np.zeros_like(k), gv=np.zeros_like(v), gstate=np.zeros((B, H, Dk, Dv)))
    for b in range(B):
        n = L if lens is None else int(lens[b])
        for h in range(H):
            K, V = slice(h * Dk, (h + 1) * Dk), slice(h * Dv, (h + 1) * Dv)
            S = np.zeros((Dk, Dv)) if h0 is None else h0[b, h].copy()
            for t in range(n):
                S = lam[h] * S + np.outer(k[b, t, K], v[b, t, V])
                out["y"][b, t, V] = scale * q[b, t, K] @ S
                if gy is not None:
                    out["gq"][b, t, K] = scale * S @ gy[b, t, V]
            out["state"][b, h] = S
            if gy is None:
                continue
            G = np.zeros((Dk, Dv)) if ghT is None else ghT[b, h].copy()
            for t in reversed(range(n)):
                G = G + scale * np.outer(q[b, t, K], gy[b, t, V])
                out["gk"][b, t, K] = G @ v[b, t, V]
                out["gv"][b, t, V] = k[b, t, K] @ G
                G = lam[h] * G
            out["gstate"][b, h] = G
    return out


def gated_ffn(x, w_in, w_out, kind, gy=None):
    """x (M, C), w_in (C, 2 F), w_out (F, C)."""
    F = w_out.shape[0]
    a, u = x @ w_in[:, :F], x @ w_in[:, F:]
    h = act(a, kind) * u
    out = dict(y=h @ w_out)
    if gy is not None:
        gh = gy @ w_out.T
        g = np.concatenate([gh * u * slope(a, kind), gh * act(a, kind)], 1)
        out.update(gx=g @ w_in.T, gw_in=x.T @ g, gw_out=h.T @ gy)
    return out
