"""Inputs and derived error bounds for the tests of the short convolution and
the selective scan.

The bounds follow the float32 arithmetic step by step in float64: E = 2^-24 is
half a step of float32, every product, sum or approximate function adds its
own relative error, and the state's error is carried through the recurrence as
the state is.  The output's own rounding (half a step of its type) comes last.
"""
import numpy as np
import torch

import workloads as W
from oracle import state_space as O

E = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}  # torch.finfo(t).eps / 2
TINY = 1e-30  # below: products under float32's range are flushed


def store(a, dtype):
    a = np.asarray(a, dtype=np.float32)
    return W.round_bf16(a) if dtype == "bf16" else a


def silu_err(v, dv):
    """Error of silu at v known to dv: slope at most 1.1; the exponential is
    off by (|v| + 4) E relative (its argument's rounding, then itself), the
    sum, the reciprocal (2 steps of 2^-23) and the product by 8 E more."""
    return 1.1 * dv + np.abs(O.silu(v)) * (np.abs(v) + 12.0) * E


def conv_bound(x, w, bias, s0, lens, act, dtype, y):
    """Elementwise bound on |y_gpu - y| for oracle values y (NaN behind a length)."""
    W_ = w.shape[-1]
    mag, _ = O.short_conv(np.abs(x), np.abs(w), None if bias is None else np.abs(bias),
                          None if s0 is None else np.abs(s0), lens, "none")
    dv = (W_ + 1) * E * mag
    if act == "silu":
        v, _ = O.short_conv(x, w, bias, s0, lens, "none")
        dv = silu_err(v, dv)
    return 1.01 * (dv + HALF[dtype] * np.abs(y)) + TINY


def scan_bound(u, delta, A, Bm, Cm, D, z, delta_bias, h0, lens, use_softplus, dtype):
    """(bound on y, bound on hT), elementwise, and the oracle's (y, hT)."""
    f = lambda a: None if a is None else np.asarray(a, dtype=np.float64)  # noqa: E731
    u, delta, A, Bm, Cm, D, z, delta_bias, h0 = map(f, (u, delta, A, Bm, Cm, D, z, delta_bias, h0))
    nB, T, nD = u.shape
    N = A.shape[1]
    group = np.arange(nD) // (nD // Bm.shape[2])
    y, yb = np.full((nB, T, nD), np.nan), np.full((nB, T, nD), np.nan)
    hT = np.zeros((nB, nD, N)) if h0 is None else h0.copy()
    hb = np.zeros((nB, nD, N))
    for b in range(nB):
        n = T if lens is None else min(max(int(lens[b]), 0), T)
        h, e = hT[b], hb[b]
        for t in range(n):
            raw = delta[b, t] + (0.0 if delta_bias is None else delta_bias)
            dt, ddt = raw, E * np.abs(raw)
            if use_softplus:
                # slope = sigmoid(raw) <= min(1, dt); 8 E for exp, log1p and the sum
                dt = O.softplus(raw)
                ddt = E * np.abs(raw) * np.minimum(1.0, dt) + 8 * E * dt
            x = dt * u[b, t]
            dx = np.abs(u[b, t]) * ddt + E * np.abs(x)
            # a = 2^(dt (A log2 e)): argument off by ddt and three roundings, and, where a
            # sequence is split, by a sum of step sizes (T / 32 + 8 additions); the
            # exponential itself by 4 E (2^-22), one E for its own rounding
            arg = np.abs(dt[:, None] * A)
            rel = ddt[:, None] * np.abs(A) + arg * (3 + T / 32 + 8) * E + 5 * E
            a = np.exp(dt[:, None] * A)
            xb = x[:, None] * Bm[b, t, group]
            e = a * e * (1 + rel) + np.abs(a * h) * (rel + 2 * E) \
                + np.abs(Bm[b, t, group]) * (dx + E * np.abs(x))[:, None]
            h = a * h + xb
            e = e + 2 * E * np.abs(h) + TINY
            C = Cm[b, t, group]
            v, dv = (C * h).sum(-1), (np.abs(C) * e).sum(-1) + (N + 2) * E * np.abs(C * h).sum(-1)
            if D is not None:
                v = v + D * u[b, t]
                dv = dv + 2 * E * np.abs(D * u[b, t]) + E * np.abs(v)
            if z is not None:
                zt = z[b, t]
                s = O.silu(zt)
                dv = np.abs(s) * dv + np.abs(v) * (silu_err(zt, 0.0) + E * np.abs(s))
                v = v * s
            y[b, t] = v
            yb[b, t] = 1.01 * (dv + HALF[dtype] * np.abs(v)) + TINY
        hT[b], hb[b] = h, 1.01 * e
    return yb, hb, y, hT


def conv_case(seed, B, H, T, d, W_, dtype, bias=False, state=False, lens=None):
    r = np.random.default_rng(seed)
    return dict(x=store(r.standard_normal((B, H, T, d)), dtype),
                w=(0.5 * r.standard_normal((H, d, W_))).astype(np.float32),
                bias=(0.2 * r.standard_normal((H, d))).astype(np.float32) if bias else None,
                s0=store(r.standard_normal((B, H, W_ - 1, d)), dtype) if state else None,
                lens=None if lens is None else np.asarray(lens, np.int32))


def scan_case(seed, B, T, D, G, N, dtype, gate=True, state=False, bias=True, skip=True, lens=None,
              use_softplus=True):
    r = np.random.default_rng(seed)
    n = r.standard_normal
    step = np.exp(r.uniform(np.log(1e-3), np.log(0.1), D))
    if use_softplus:
        delta = 0.5 * n((B, T, D))
        db = step + np.log(-np.expm1(-step))
        if not bias:
            delta = delta + db
    else:
        delta, db = step * np.exp(0.3 * n((B, T, D))), 0.1 * step
    return dict(u=store(n((B, T, D)), dtype), delta=store(delta, dtype),
                A=(-np.arange(1, N + 1) * np.exp(0.1 * n((D, N)))).astype(np.float32),
                Bm=store(n((B, T, G, N)), dtype), Cm=store(n((B, T, G, N)), dtype),
                D=(1 + 0.1 * n(D)).astype(np.float32) if skip else None,
                z=store(n((B, T, D)), dtype) if gate else None,
                delta_bias=db.astype(np.float32) if bias else None,
                h0=(0.5 * n((B, D, N))).astype(np.float32) if state else None,
                lens=None if lens is None else np.asarray(lens, np.int32))


def dev(a, dtype=None):
    """Array to the device: floats in `dtype` ("f32"/"bf16"/None = as they are)."""
    if a is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def host(t):
    return t.detach().double().cpu().numpy()


def within(got, ref, bound, what=""):
    """got (NaN nowhere) within bound of ref where ref is not NaN."""
    live = ~np.isnan(ref)
    assert np.isfinite(got[live]).all(), what
    off = np.abs(got[live] - ref[live]) - bound[live]
    assert off.size == 0 or off.max() <= 0.0, \
        f"{what}: {off.max():.3e} over the bound at a bound of {bound[live].flat[off.argmax()]:.3e}"
