"""Error bounds of the gated recurrence and its gradients that follow the formulas'
own weights, so that they shrink where the values do: inputs under 1 - a, gradients
under a (1 - a). Two of each: by element, from the roundings along a state's path,
and by channel (the norm over its tokens), as roundings of different tokens add up
when they are independent, which is what finds a factor that is a per cent off.

In half steps of fp32 (E24): a decay is off by at most 8 of itself (exponential 4,
sum, reciprocal 2, product), with bf16 logits by 1.3 (1 - a) |f| more (the rounded
argument of its exponential); 1 - a by 12, with bf16 logits by 1.3 |f| more; its
products by one each. The chunked order adds one rounding of A per token, and one of
the state."""

from __future__ import annotations

import numpy as np
import torch

from oracle import layer_oracle as lo

E24 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def np64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def sequences(B, T, cu):
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    return [(0, int(cu[i]), int(cu[i + 1])) for i in range(len(cu) - 1)]


def weights(gate, mode):
    """a and 1 - a in 64 bits, neither as a difference."""
    if mode == "log":
        return np.exp(gate), -np.expm1(gate)
    e = np.exp(-np.abs(gate))
    return np.where(gate < 0, e, 1) / (1 + e), np.where(gate < 0, 1, e) / (1 + e)


def by_element(name, got, ref, dtype, err):
    bound = err + half_step(dtype) * (np.abs(ref) + err) + 1e-37
    off = np.abs(got - ref) / bound
    assert np.all(off <= 1), f"{name}: {(~(off <= 1)).sum()} of {off.size} off, worst {np.nanmax(off):.2f} times the bound"


def by_channel(name, got, ref, size, dtype, steps):
    """The norm of each channel's errors over its tokens: `steps` roundings of a state, of
    different signs, and 16 of the values that it is a sum of."""
    rel = half_step(dtype) + steps * E24
    off = np.linalg.norm(got - ref, axis=0)
    bound = rel * np.linalg.norm(ref, axis=0) + 16 * E24 * np.linalg.norm(size, axis=0) + 1e-37
    assert np.all(off <= bound), f"{name}: {(~(off <= bound)).sum()} channels off, worst {np.nanmax(off / bound):.2f} times the bound"


class Run:
    """One sequence: values, the sums of magnitudes behind them, and errors, forward and backward."""

    def __init__(self, x, gate, mode, comp, h0, gate_dtype):
        T, D = x.shape
        self.x, self.comp, self.mode = x, comp, mode
        self.a, self.b = weights(gate, mode)
        rounded = 1.3 * np.abs(gate) if mode == "logits" and gate_dtype == torch.bfloat16 else np.zeros_like(gate)
        self.ca, self.cb = 8 + rounded * self.b, 12 + rounded
        u = self.b * x if comp else x
        cu = self.cb + 1 if comp else np.zeros_like(x)
        h = np.zeros(D) if h0 is None else h0
        s, e = np.abs(h), np.zeros(D)
        self.h, self.before, self.size, self.size_before, self.err, self.err_before = (np.zeros((T, D)) for _ in range(6))
        for t in range(T):
            self.before[t], self.size_before[t], self.err_before[t] = h, s, e
            e = self.a[t] * e + E24 * ((self.ca[t] + 2) * self.a[t] * s + cu[t] * np.abs(u[t]))
            h = self.a[t] * h + u[t]
            s = self.a[t] * s + np.abs(u[t])
            e = e + 2 * E24 * s
            self.h[t], self.size[t], self.err[t] = h, s, e
        self.last, self.last_size, self.last_err = h, s, e

    def gradients(self, dy, dhT):
        T, D = dy.shape
        d = np.zeros(D) if dhT is None else dhT
        s, e = np.abs(d), np.zeros(D)
        ds, ss, es = (np.zeros((T, D)) for _ in range(3))
        for t in range(T - 1, -1, -1):
            d, s = d + dy[t], s + np.abs(dy[t])
            e = e + 2 * E24 * s
            ds[t], ss[t], es[t] = d, s, e
            e = self.a[t] * e + E24 * (self.ca[t] + 2) * self.a[t] * s
            d, s = self.a[t] * d, self.a[t] * s
        w = self.b if self.comp else np.ones_like(self.a)
        k = self.a * self.b if self.mode == "logits" else self.a
        ck = self.ca + 4 + (self.cb if self.mode == "logits" else 0)
        of = self.before - (self.x if self.comp else 0)
        of_size = self.size_before + (np.abs(self.x) if self.comp else 0)
        self.dx, self.dx_size, self.dx_err = w * ds, w * ss, w * (es + (E24 * (self.cb + 1) * ss if self.comp else 0))
        self.dgate, self.dgate_size = k * ds * of, k * ss * of_size
        self.dgate_err = k * (es * of_size + ss * self.err_before) + E24 * ck * self.dgate_size
        self.dh0, self.dh0_err = d, e + 2 * E24 * s
        return self


def check_scan(got, x, gate, mode, comp, h0=None, dy=None, dhT=None, cu=None):
    """got: a dict of some of y, hT, dx, dgate, dh0, as numpy or torch values, against
    the recurrence over x, gate (torch, as stored)."""
    B, T, D = x.shape
    val = lambda k: np64(got[k]) if isinstance(got[k], torch.Tensor) else np.asarray(got[k], np.float64)  # noqa: E731
    out = {k: val(k) for k in got if got[k] is not None}
    xs, gs = np64(x), np64(gate)
    n64 = lambda t, n: None if t is None else np64(t[n])  # noqa: E731
    for n, (b, s, e) in enumerate(sequences(B, T, cu)):
        run = Run(xs[b, s:e], gs[b, s:e], mode, comp, n64(h0, n), gate.dtype)
        steps = 14 * np.sqrt(max(e - s, 1))
        ref, _, _ = lo.scan(xs[b, s:e], gs[b, s:e], gate_mode=mode, complement=comp, h0=n64(h0, n))
        assert np.allclose(ref, run.h, rtol=1e-6, atol=1e-9)  # (the oracle forms 1 - a as a difference)
        if "y" in out and e > s:
            by_element("y", out["y"][b, s:e], run.h, x.dtype, run.err)
            by_channel("y", out["y"][b, s:e], run.h, run.size, x.dtype, steps)
        if "hT" in out:
            by_element("hT", out["hT"][n], run.last, torch.float32, run.last_err)
        if dy is None:
            continue
        run.gradients(np64(dy)[b, s:e], n64(dhT, n))
        if "dx" in out and e > s:
            by_element("dx", out["dx"][b, s:e], run.dx, x.dtype, run.dx_err)
            by_channel("dx", out["dx"][b, s:e], run.dx, run.dx_size, x.dtype, steps)
        if "dgate" in out and e > s:
            by_element("dgate", out["dgate"][b, s:e], run.dgate, gate.dtype, run.dgate_err)
            by_channel("dgate", out["dgate"][b, s:e], run.dgate, run.dgate_size, gate.dtype, 2 * steps)
        if "dh0" in out:
            by_element("dh0", out["dh0"][n], run.dh0, torch.float32, run.dh0_err)
