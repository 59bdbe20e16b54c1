"""The channels-last mixer operators in 64 bits on the host: numpy, one row after another,
written from the formulas of include/hc_mixer.h.  Rows past a sequence's length are left out
by construction (the loops end there), whatever they hold."""
from __future__ import annotations

import numpy as np
from scipy.special import erf, expit


def act(x, kind):
    if kind == "silu":
        return x * expit(x)
    if kind == "gelu":
        return 0.5 * x * (1 + erf(x / np.sqrt(2)))
    return x


def slope(x, kind):
    if kind == "silu":
        s = expit(x)
        return s * (1 + x * (1 - s))
    if kind == "gelu":
        return 0.5 * (1 + erf(x / np.sqrt(2))) + x * np.exp(-0.5 * x * x) / np.sqrt(2 * np.pi)
    return np.ones_like(x)


def groupnorm(x, gamma, beta, groups, eps, kind, gy=None):
    """x (N, P, C) float64 -> dict of y, mean, rstd and, with gy, gx, ggamma, gbeta."""
    N, P, C = x.shape
    v = x.reshape(N, P, groups, C // groups)
    mean = v.mean((1, 3))
    rstd = 1 / np.sqrt(((v - mean[:, None, :, None]) ** 2).mean((1, 3)) + eps)
    xh = ((v - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(N, P, C)
    pre = xh * gamma + beta
    out = dict(y=act(pre, kind), mean=mean, rstd=rstd)
    if gy is not None:
        g = gy * slope(pre, kind)
        out["ggamma"], out["gbeta"] = (g * xh).sum((0, 1)), g.sum((0, 1))
        q = (g * gamma).reshape(v.shape)
        xv = xh.reshape(v.shape)
        m1, m2 = q.mean((1, 3), keepdims=True), (q * xv).mean((1, 3), keepdims=True)
        out["gx"] = (rstd[:, None, :, None] * (q - m1 - xv * m2)).reshape(N, P, C)
    return out


def causal_conv(x, w, bias, kind, state=None, lens=None, gy=None, gstate_out=None):
    """x (B, L, D), w (D, K), state (B, K - 1, D)."""
    B, L, D = x.shape
    K = w.shape[1]
    state = np.zeros((B, K - 1, D)) if state is None else state
    bias = np.zeros(D) if bias is None else bias
    out = dict(y=np.zeros((B, L, D)), state=np.zeros((B, K - 1, D)))
    if gy is not None:
        out.update(gx=np.zeros((B, L, D)), gw=np.zeros((D, K)), gb=np.zeros(D), gstate=np.zeros((B, K - 1, D)))
    for b in range(B):
        n = L if lens is None else int(lens[b])
        rows = np.concatenate([state[b], x[b, :n]])  # row t of the sequence is rows[t + K - 1]
        out["state"][b] = rows[n:n + K - 1]
        grows = np.zeros_like(rows)
        for t in range(n):
            win = rows[t:t + K]
            pre = bias + (win * w.T).sum(0)
            out["y"][b, t] = act(pre, kind)
            if gy is not None:
                g = gy[b, t] * slope(pre, kind)
                out["gb"] += g
                out["gw"] += (g * win).T
                grows[t:t + K] += g * w.T
        if gy is not None:
            if gstate_out is not None:
                grows[n:n + K - 1] += gstate_out[b]
            out["gstate"][b], out["gx"][b, :n] = grows[:K - 1], grows[K - 1:]
    return out


def scan(u, dt, A, Bm, Cm, groups, softplus=True, D=None, z=None, bias=None, h0=None, lens=None, gy=None, ghT=None):
    """u, dt, z (B, L, D); A (D, N); Bm, Cm (B, L, groups * N); h0 (B, D, N)."""
    B, L, Dm = u.shape
    N, per = A.shape[1], Dm // groups
    D = np.zeros(Dm) if D is None else D
    bias = np.zeros(Dm) if bias is None else bias
    wide = lambda r: np.repeat(r.reshape(groups, N), per, axis=0)  # (D, N)
    out = dict(y=np.zeros((B, L, Dm)), state=np.zeros((B, Dm, N)))
    if gy is not None:
        out.update(gu=np.zeros((B, L, Dm)), gdt=np.zeros((B, L, Dm)), gz=np.zeros((B, L, Dm)),
                   gB=np.zeros((B, L, groups * N)), gC=np.zeros((B, L, groups * N)), gA=np.zeros((Dm, N)),
                   gD=np.zeros(Dm), gdt_bias=np.zeros(Dm), gstate=np.zeros((B, Dm, N)))
    for b in range(B):
        n = L if lens is None else int(lens[b])
        h = np.zeros((Dm, N)) if h0 is None else h0[b].copy()
        hs, ys = [h], []
        raw = dt[b, :n] + bias
        delta = np.logaddexp(0, raw) if softplus else raw
        gate = np.ones((n, Dm)) if z is None else act(z[b, :n], "silu")
        for t in range(n):
            h = np.exp(delta[t][:, None] * A) * h + (delta[t] * u[b, t])[:, None] * wide(Bm[b, t])
            hs.append(h)
            ys.append((h * wide(Cm[b, t])).sum(1) + D * u[b, t])
            out["y"][b, t] = ys[t] * gate[t]
        out["state"][b] = h
        if gy is None:
            continue
        G = np.zeros((Dm, N)) if ghT is None else ghT[b].copy()
        for t in reversed(range(n)):
            q = gy[b, t] * gate[t]
            if z is not None:
                out["gz"][b, t] = gy[b, t] * ys[t] * slope(z[b, t], "silu")
            G = G + q[:, None] * wide(Cm[b, t])
            a = np.exp(delta[t][:, None] * A)
            E = G * a * hs[t]
            GB = (G * wide(Bm[b, t])).sum(1)
            out["gu"][b, t] = GB * delta[t] + D * q
            gd = (GB * u[b, t] + (E * A).sum(1)) * (expit(raw[t]) if softplus else 1.0)
            out["gdt"][b, t] = gd
            out["gdt_bias"] += gd
            out["gD"] += q * u[b, t]
            out["gA"] += E * delta[t][:, None]
            fold = lambda m: m.reshape(groups, per, N).sum(1).reshape(-1)
            out["gB"][b, t] = fold(G * (delta[t] * u[b, t])[:, None])
            out["gC"][b, t] = fold(q[:, None] * hs[t + 1])
            G = G * a
        out["gstate"][b] = G
    return out
