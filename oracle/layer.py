"""Plain float64 forms of what an MoE layer computes around its FP8 products:
expert products over ragged row runs, the dense product with an epilogue,
layer norm and the combine step, each with its gradients.  Loops and textbook
formulas; no code shared with the HIP path.
"""
import math

import numpy as np


def _f64(*arrays):
    return [np.asarray(a, np.float64) for a in arrays]


# ------------------------------------------------- products over ragged runs
def grouped(x, w, offsets):
    """(y, S): y[r] = x[r] w[e]^T for the rows of expert e's run, zeros for the
    rows of no run; S the same sums of absolute values."""
    x, w = _f64(x, w)
    y = np.zeros((x.shape[0], w.shape[1]))
    s = np.zeros_like(y)
    for e in range(w.shape[0]):
        a, b = offsets[e], offsets[e + 1]
        y[a:b] = x[a:b] @ w[e].T
        s[a:b] = np.abs(x[a:b]) @ np.abs(w[e]).T
    return y, s


def grouped_dgrad(dy, w, offsets):
    return grouped(dy, np.swapaxes(np.asarray(w, np.float64), 1, 2), offsets)


def grouped_wgrad(dy, x, offsets):
    dy, x = _f64(dy, x)
    shape = (len(offsets) - 1, dy.shape[1], x.shape[1])
    dw, s = np.zeros(shape), np.zeros(shape)
    for e in range(shape[0]):
        a, b = offsets[e], offsets[e + 1]
        dw[e] = dy[a:b].T @ x[a:b]
        s[e] = np.abs(dy[a:b]).T @ np.abs(x[a:b])
    return dw, s


# ----------------------------------------------------- product with epilogue
_erf = np.vectorize(math.erf, otypes=[np.float64])


def activation(name, z):
    z = np.asarray(z, np.float64)
    if name == "relu":
        return np.maximum(z, 0)
    if name == "silu":
        return z / (1 + np.exp(-z))
    if name == "gelu":
        return z * (1 + _erf(z / math.sqrt(2))) / 2
    return z


def slope(name, z):
    z = np.asarray(z, np.float64)
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "silu":
        p = 1 / (1 + np.exp(-z))
        return p + z * p * (1 - p)
    if name == "gelu":
        return (1 + _erf(z / math.sqrt(2))) / 2 + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return np.ones_like(z)


def dense(x, w, bias=None):
    """(z, S) of x w^T + bias."""
    x, w = _f64(x, w)
    z, s = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias is not None:
        z, s = z + bias, s + np.abs(bias)
    return z, s


# --------------------------------------------------------------- layer norm
def layer_norm(x, weight, bias, eps):
    x, weight = _f64(x, weight)
    mean = x.mean(-1, keepdims=True)
    rstd = 1 / np.sqrt(((x - mean) ** 2).mean(-1, keepdims=True) + eps)
    y = (x - mean) * rstd * weight + (0 if bias is None else np.asarray(bias, np.float64))
    return y, mean[..., 0], rstd[..., 0]


def layer_norm_backward(dy, x, weight, mean, rstd):
    dy, x, weight, mean, rstd = _f64(dy, x, weight, mean, rstd)
    h = (x - mean[:, None]) * rstd[:, None]
    g = dy * weight
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True) - h * (g * h).mean(1, keepdims=True))
    return dx, (dy * h).sum(0), dy.sum(0)


# ------------------------------------------------------------------ combine
def combine(y, token_row, weights, residual=None):
    y, weights = _f64(y, weights)
    out = np.zeros((token_row.shape[0], y.shape[1]))
    for t in range(token_row.shape[0]):
        for j in range(token_row.shape[1]):
            r = token_row[t, j]
            if 0 <= r < y.shape[0]:
                out[t] += weights[t, j] * y[r]
    return out if residual is None else out + residual


def combine_backward(dout, y, token_row, weights):
    dout, y, weights = _f64(dout, y, weights)
    dy, dp = np.zeros_like(y), np.zeros_like(weights)
    for t in range(token_row.shape[0]):
        for j in range(token_row.shape[1]):
            r = token_row[t, j]
            if 0 <= r < y.shape[0]:
                dy[r] = weights[t, j] * dout[t]
                dp[t, j] = dout[t] @ y[r]
    return dy, dp
