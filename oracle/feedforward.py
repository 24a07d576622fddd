"""fp64 oracle of the feed-forward operators: RMS norm with the residual's
addition, rows in e4m3 with a scale, the linear layer with its epilogue, and
their gradients.  Everything is evaluated in fp64 and nothing is rounded but
the e4m3 codes (e4m3_rne), which follow the format's definition: 4 exponent
bits with bias 7, 3 fraction bits, largest finite value 448, subnormals in
steps of 2^-9, round to nearest, ties to even."""

from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
AMAX_FLOOR = 1e-30
GELU_C = np.sqrt(2.0 / np.pi)


def sigmoid(t):
    t = np.asarray(t, np.float64)
    e = np.exp(-np.abs(t))
    return np.where(t >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def act(u, kind):
    u = np.asarray(u, np.float64)
    if kind == "relu":
        return np.where(u < 0, 0.0, u)
    if kind == "gelu":
        return 0.5 * u * (1.0 + np.tanh(GELU_C * (u + 0.044715 * u ** 3)))
    if kind == "silu":
        return u * sigmoid(u)
    return u


def act_grad(u, kind):
    u = np.asarray(u, np.float64)
    if kind == "relu":
        return (u > 0).astype(np.float64)
    if kind == "gelu":
        t = np.tanh(GELU_C * (u + 0.044715 * u ** 3))
        return 0.5 * (1.0 + t) + 0.5 * u * (1.0 - t * t) * GELU_C * (1.0 + 3 * 0.044715 * u ** 2)
    if kind == "silu":
        s = sigmoid(u)
        return s + u * s * (1.0 - s)
    return np.ones_like(u)


def e4m3_rne(v):
    """The e4m3 value nearest to v (saturating at +-448; NaN stays NaN)."""
    v = np.asarray(v, np.float64)
    a = np.minimum(np.abs(v), E4M3_MAX)
    e = np.floor(np.log2(np.where(a > 0, a, 1.0)))
    step = np.exp2(np.maximum(e, -6.0) - 3.0)
    q = np.minimum(np.rint(a / step) * step, E4M3_MAX)
    return np.where(np.isnan(v), np.nan, np.copysign(q, v))


def row_scale(y):
    return np.maximum(np.max(np.abs(y), axis=-1), AMAX_FLOOR) / E4M3_MAX


def rmsnorm(x, gamma, eps, residual=None):
    """(h, y, rstd)."""
    h = np.asarray(x, np.float64) + (0.0 if residual is None else np.asarray(residual, np.float64))
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=-1) + eps)
    return h, h * rstd[..., None] * np.asarray(gamma, np.float64), rstd


def rmsnorm_backward(dy, h, gamma, rstd, dh=None):
    """(dx, dgamma) at h with the given rstd."""
    dy, h, gamma = (np.asarray(t, np.float64) for t in (dy, h, gamma))
    rstd = np.asarray(rstd, np.float64)[:, None]
    n, g = h * rstd, dy * gamma
    dx = rstd * (g - n * np.mean(g * n, axis=-1, keepdims=True))
    if dh is not None:
        dx = dx + np.asarray(dh, np.float64)
    return dx, np.sum(dy * n, axis=0)


def linear(x, w, bias=None, kind="none", residual=None, x_scale=None, w_scale=None):
    """(y, z)."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    if x_scale is not None:
        x = x * np.asarray(x_scale, np.float64)[:, None]
        w = w * np.asarray(w_scale, np.float64)[:, None]
    z = x @ w.T
    if bias is not None:
        z = z + np.asarray(bias, np.float64)
    y = act(z, kind)
    if residual is not None:
        y = y + np.asarray(residual, np.float64)
    return y, z


def linear_backward(dz, x, w, z_prev=None, kind_prev="none"):
    """(dx, dw, dbias)."""
    dz, x, w = (np.asarray(t, np.float64) for t in (dz, x, w))
    dx = dz @ w
    if z_prev is not None:
        dx = dx * act_grad(z_prev, kind_prev)
    return dx, dz.T @ x, dz.sum(axis=0)
