"""Float64 definitions of the short causal convolution, the selective state
space scan and the slot copies (numpy, token by token).

TEST INFRASTRUCTURE ONLY, as the rest of this package: it shares no code with
the GPU library.
"""
from __future__ import annotations

import numpy as np


def _f64(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def silu(x):
    return x / (1.0 + np.exp(-x))


def softplus(x):
    return np.logaddexp(x, 0.0)


def short_conv(x, w, bias=None, s0=None, lens=None, act="silu"):
    """x [B,H,T,d], w [H,d,W] (the last tap meets the current token), bias
    [H,d], s0 [B,H,W-1,d], lens [B].  Returns (y, sT); rows of y behind a
    sequence's length are NaN."""
    x, w, bias, s0 = _f64(x), _f64(w), _f64(bias), _f64(s0)
    B, H, T, d = x.shape
    W = w.shape[-1]
    y = np.full((B, H, T, d), np.nan)
    sT = np.zeros((B, H, W - 1, d))
    for b in range(B):
        n = T if lens is None else min(max(int(lens[b]), 0), T)
        win = np.zeros((H, W, d))  # the last W inputs, oldest first
        if s0 is not None:
            win[:, 1:] = s0[b]
        for t in range(n):
            win = np.concatenate([win[:, 1:], x[b, :, t][:, None]], axis=1)
            v = np.einsum("hwd,hdw->hd", win, w) + (0.0 if bias is None else bias)
            y[b, :, t] = silu(v) if act == "silu" else v
        sT[b] = win[:, 1:]
    return y, sT


def selective_scan(u, delta, A, Bm, Cm, D=None, z=None, delta_bias=None, h0=None, lens=None,
                   use_softplus=True):
    """u, delta, z [B,T,D], A [D,N], Bm, Cm [B,T,G,N], h0 [B,D,N].  Returns
    (y, hT); rows of y behind a sequence's length are NaN."""
    u, delta, A, Bm, Cm = map(_f64, (u, delta, A, Bm, Cm))
    D, z, delta_bias, h0 = map(_f64, (D, z, delta_bias, h0))
    nB, T, nD = u.shape
    group = np.arange(nD) // (nD // Bm.shape[2])
    y = np.full((nB, T, nD), np.nan)
    hT = np.zeros((nB,) + A.shape) if h0 is None else h0.copy()
    for b in range(nB):
        n = T if lens is None else min(max(int(lens[b]), 0), T)
        h = hT[b]
        for t in range(n):
            dt = delta[b, t] + (0.0 if delta_bias is None else delta_bias)
            if use_softplus:
                dt = softplus(dt)
            h = np.exp(dt[:, None] * A) * h + (dt * u[b, t])[:, None] * Bm[b, t, group]
            v = (Cm[b, t, group] * h).sum(-1)
            if D is not None:
                v = v + D * u[b, t]
            y[b, t] = v if z is None else v * silu(z[b, t])
        hT[b] = h
    return y, hT


def state_copy(pool, src, dst):
    """pool [layers, slots, ...]: the copies one after the other, in order."""
    pool = np.array(pool)
    for i, j in zip(src, dst):
        pool[:, j] = pool[:, i]
    return pool
