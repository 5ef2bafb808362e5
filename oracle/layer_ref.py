"""Float64 reference of the state space layer's operators, token by token.

Each function also returns the sums of magnitudes that bound its rounding errors (``*_abs``): what
the result would be if every term were positive.  Arrays are numpy float64; a batch is one sequence
here, and the tests loop over sequences.
"""
from __future__ import annotations

import numpy as np


def sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1 / (1 + e), e / (1 + e))


def softplus(x):
    return np.maximum(x, 0) + np.log1p(np.exp(-np.abs(x)))


def short_conv(x, w, bias, state, silu):
    """x [T, C], w [C, K], bias [C], state [K-1, C] -> y, y_abs [T, C] (before the SiLU), new state."""
    T, C = x.shape
    K = w.shape[1]
    whole = np.concatenate([state, x], 0)
    y, y_abs = np.empty((T, C)), np.empty((T, C))
    for t in range(T):
        window = whole[t:t + K].T * w
        y[t] = bias + window.sum(1)
        y_abs[t] = np.abs(bias) + np.abs(window).sum(1)
    return (y * sigmoid(y) if silu else y), y_abs, whole[T:]


def ssm_scan(x, dt, A, B, C, h, D=None, z=None, dt_bias=None, softplus_on=True):
    """x [T, H, P], dt [T, H], B, C [T, G, N], h [H, P, N] -> y, y_abs [T, H, P], h, h_abs.

    y_abs: sum of magnitudes, times |silu(z)|."""
    T, H, P = x.shape
    G, N = B.shape[1:]
    h, h_abs = h.copy(), np.abs(h)
    y, y_abs = np.empty_like(x), np.empty_like(x)
    s = dt + (0 if dt_bias is None else dt_bias)
    s = softplus(s) if softplus_on else s
    for t in range(T):
        dec = np.exp(A * s[t])[:, None, None]
        b, c = np.repeat(B[t], H // G, 0), np.repeat(C[t], H // G, 0)
        new = (s[t][:, None] * x[t])[:, :, None] * b[:, None, :]
        h = dec * h + new
        h_abs = dec * h_abs + np.abs(new)
        y[t] = (h * c[:, None, :]).sum(-1)
        y_abs[t] = (h_abs * np.abs(c)[:, None, :]).sum(-1)
        if D is not None:
            y[t] += D[:, None] * x[t]
            y_abs[t] += np.abs(D[:, None] * x[t])
    if z is not None:
        gate = z * sigmoid(z)
        y, y_abs = y * gate, y_abs * np.abs(gate)
    return y, y_abs, h, h_abs


def rms_norm(x, w, residual, eps):
    """x, residual [M, D] -> v, r."""
    r = x + residual
    return r / np.sqrt((r * r).mean(1, keepdims=True) + eps) * w, r


def scales(v, top, group):
    """Scales [M, groups] of rows (group 0: one) for codes up to `top`."""
    M, D = v.shape
    width = group or D
    parts = [np.abs(v[:, i:i + width]).max(1) for i in range(0, D, width)]
    s = np.stack(parts, 1) / top
    return np.where(s < 2.0 ** -126, 1.0, s)
