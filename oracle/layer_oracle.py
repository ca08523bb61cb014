"""fp64 CPU definitions of the layer operators (numpy): residual add + RMS norm
with e4m3 output, the projection with its epilogue, and the gated linear
recurrence with its gradients. Test infrastructure only, like the rest of this
package."""

from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0


def add_rmsnorm(x, residual, weight, eps):
    """(y, r) of r = x + residual, y = r / sqrt(mean(r^2) + eps) * weight by rows."""
    r = x if residual is None else x + residual
    return r / np.sqrt(np.mean(r * r, axis=-1, keepdims=True) + eps) * weight, r


def row_scale(y):
    """Largest magnitude of each row over 448; 1 for rows of zeros."""
    m = np.max(np.abs(y), axis=-1)
    return np.where(m > 0, np.maximum(m / E4M3_MAX, 2.0 ** -126), 1.0)


def activate(v, kind):
    if kind == "silu":
        return v / (1 + np.exp(-v))
    if kind == "gelu":
        return 0.5 * v * (1 + np.vectorize(math.erf, otypes=[np.float64])(v / math.sqrt(2)))
    if kind == "sigmoid":
        return 1 / (1 + np.exp(-v))
    if kind == "relu":
        return np.maximum(v, 0)
    if kind != "none":
        raise ValueError(kind)
    return v


def linear(x, w, *, x_scale=None, w_scale=None, bias=None, activation="none", residual=None):
    v = x @ w.T
    if x_scale is not None:
        v = v * x_scale[:, None] * w_scale[None, :]
    if bias is not None:
        v = v + bias
    v = activate(v, activation)
    return v if residual is None else v + residual


def scan_decay(gate, gate_mode):
    return np.exp(gate) if gate_mode == "log" else 1 / (1 + np.exp(-gate))


def scan(x, gate, *, gate_mode, complement, h0=None):
    """One sequence: x, gate [T, D]. Returns (y [T, D], hT [D], states before each token [T, D])."""
    a = scan_decay(gate, gate_mode)
    h = np.zeros(x.shape[1]) if h0 is None else np.array(h0, np.float64)
    y, before = np.zeros_like(x), np.zeros_like(x)
    for t in range(x.shape[0]):
        before[t] = h
        h = a[t] * h + ((1 - a[t]) * x[t] if complement else x[t])
        y[t] = h
    return y, h, before


def scan_grad(x, gate, dy, *, gate_mode, complement, h0=None, dhT=None):
    """(dx, dgate, dh0) of sum(dy * y) + sum(dhT * hT) for one sequence."""
    a = scan_decay(gate, gate_mode)
    _, _, before = scan(x, gate, gate_mode=gate_mode, complement=complement, h0=h0)
    d = np.zeros(x.shape[1]) if dhT is None else np.array(dhT, np.float64)
    dx, dgate = np.zeros_like(x), np.zeros_like(x)
    for t in range(x.shape[0] - 1, -1, -1):
        d = d + dy[t]
        dx[t] = (1 - a[t]) * d if complement else d
        da = d * (before[t] - x[t]) if complement else d * before[t]
        dgate[t] = da * a[t] * (1 if gate_mode == "log" else 1 - a[t])
        d = a[t] * d
    return dx, dgate, d
