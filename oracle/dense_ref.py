"""Float64 references of the products with an epilogue and the layer norm, and of their gradients.

Test infrastructure.  Every function also returns the sums of magnitudes that a bound on a float32
computation of the same formula needs.
"""
import numpy as np
from scipy.special import erfc


def act(v, kind):
    """none, v sigmoid(v), v Phi(v)."""
    if kind == "silu":
        return v / (1 + np.exp(-v))
    if kind == "gelu":
        return v * erfc(-v / np.sqrt(2)) / 2
    return v


def slope(v, kind):
    """The activation's derivative, and the sum of its terms' magnitudes."""
    if kind == "silu":
        s = 1 / (1 + np.exp(-v))
        return s + v * s * (1 - s), s + np.abs(v) * s * (1 - s)
    if kind == "gelu":
        cdf, density = erfc(-v / np.sqrt(2)) / 2, np.exp(-v * v / 2) / np.sqrt(2 * np.pi)
        return cdf + v * density, cdf + np.abs(v) * density
    return np.ones_like(v), np.ones_like(v)


def linear(x, w, bias=None, residual=None, kind="none", x_scale=None, w_scale=None):
    """y = act(v) + residual, v = (x x_scale) (w w_scale)^T + bias; returns y, v and the sum of v's magnitudes."""
    if x_scale is not None:
        x = x * x_scale[:, None]
    if w_scale is not None:
        w = w * w_scale[:, None]
    v, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias is not None:
        v, mag = v + bias, mag + np.abs(bias)
    y = act(v, kind)
    return (y if residual is None else y + residual), v, mag


def linear_backward(dy, x, w, pre=None, kind="none"):
    """dx, dw, db and the sums of their terms' magnitudes."""
    s, m = slope(pre, kind) if kind != "none" else (1.0, 1.0)
    g, mag = dy * s, np.abs(dy) * m
    return (g @ w, g.T @ x, g.sum(0)), (mag @ np.abs(w), mag.T @ np.abs(x), mag.sum(0))


def layer_norm(x, w, b=None, residual=None, eps=1e-5):
    """y, r, mean, rstd."""
    r = x if residual is None else x + residual
    mean = r.mean(1)
    rstd = 1 / np.sqrt(((r - mean[:, None]) ** 2).mean(1) + eps)
    y = (r - mean[:, None]) * rstd[:, None] * w
    return (y if b is None else y + b), r, mean, rstd


def layer_norm_backward(dy, x, w, mean, rstd, dresidual=None):
    """dx, dw, db and the sums of their terms' magnitudes."""
    h, a = (x - mean[:, None]) * rstd[:, None], dy * w
    along, along_mag = (a * h).mean(1, keepdims=True), np.abs(a * h).mean(1, keepdims=True)
    dx = rstd[:, None] * (a - a.mean(1, keepdims=True) - h * along)
    mag = rstd[:, None] * (np.abs(a) + np.abs(a).mean(1, keepdims=True) + np.abs(h) * along_mag)
    if dresidual is not None:
        dx, mag = dx + dresidual, mag + np.abs(dresidual)
    return (dx, (dy * h).sum(0), dy.sum(0)), (mag, np.abs(dy * h).sum(0), np.abs(dy).sum(0))
