"""The recurrence's error bounds let a plain fp32 loop pass and find planted mistakes
in it (on the CPU; the GPU's outputs meet the same bounds in test_gpu_layer_bounds.py)."""

import numpy as np
import pytest
import torch

import layer_bounds as lb

MODES = [("log", False), ("logits", True), ("log", True), ("logits", False)]
F32, BF = torch.float32, torch.bfloat16


def inputs(T, D, mode, dtype, gate_dtype, seed=0):
    """Channels from two tokens' memory to thousands'."""
    gen = torch.Generator().manual_seed(seed)
    f = torch.randn(1, T, D, generator=gen) + torch.linspace(0, 12, D)
    gate = (f if mode == "logits" else torch.nn.functional.logsigmoid(f)).to(gate_dtype)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return r(1, T, D).to(dtype), gate, r(1, D), r(1, T, D).to(dtype), r(1, D)


def plain(x, gate, mode, comp, h0, dy, dhT, difference=False):
    """The recurrence and its gradients in fp32, token by token; difference: 1 - a from the rounded a."""
    f, xs, ds = gate.float()[0], x.float()[0], dy.float()[0]
    a = torch.exp(f) if mode == "log" else torch.sigmoid(f)
    b = 1 - a if difference else -torch.expm1(f) if mode == "log" else torch.sigmoid(-f)
    h, d = h0[0].clone(), dhT[0].clone()
    y, before, dx, dg = (torch.zeros_like(xs) for _ in range(4))
    for t in range(len(xs)):
        before[t] = h
        h = a[t] * h + (b[t] * xs[t] if comp else xs[t])
        y[t] = h
    for t in range(len(xs) - 1, -1, -1):
        d = d + ds[t]
        dx[t] = b[t] * d if comp else d
        dg[t] = (b[t] if mode == "logits" else 1) * (a[t] * d * (before[t] - xs[t] if comp else before[t]))
        d = a[t] * d
    return dict(y=y[None].to(x.dtype), hT=h[None], dx=dx[None].to(x.dtype), dgate=dg[None].to(gate.dtype), dh0=d[None])


def check(got, ins, mode, comp):
    x, gate, h0, dy, dhT = ins
    lb.check_scan(got, x, gate, mode, comp, h0, dy, dhT)


@pytest.mark.parametrize("mode,comp", MODES)
@pytest.mark.parametrize("dtype,gate_dtype", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("T,D", [(1, 40), (17, 33), (300, 72), (2000, 30)])
def test_a_plain_loop_passes(mode, comp, dtype, gate_dtype, T, D):
    ins = inputs(T, D, mode, dtype, gate_dtype)
    check(plain(ins[0], ins[1], mode, comp, *ins[2:]), ins, mode, comp)


@pytest.mark.parametrize("mode,comp", MODES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("what", ["y", "hT", "dx", "dgate", "dh0"])
def test_a_per_cent_is_found(mode, comp, dtype, what):
    """1 % in any sixth of the channels, the slowest or fastest among them, and a sixth of zeros."""
    ins = inputs(300, 72, mode, dtype, dtype)
    for at in range(0, 72, 12):
        for factor in (1.01, 0.0):
            got = plain(ins[0], ins[1], mode, comp, *ins[2:])
            part = got[what].to(torch.float64)
            part[..., at:at + 12] *= factor
            got[what] = part
            with pytest.raises(AssertionError):
                check(got, ins, mode, comp)


@pytest.mark.parametrize("mode,comp", [("logits", True), ("log", True), ("logits", False)])
def test_a_difference_for_1_minus_a_is_found(mode, comp):
    ins = inputs(300, 72, mode, F32, F32)
    got = plain(ins[0], ins[1], mode, comp, *ins[2:], difference=True)
    with pytest.raises(AssertionError):
        check(got, ins, mode, comp)


@pytest.mark.parametrize("mode", ["log", "logits"])
def test_a_forgotten_weight_is_found(mode):
    ins = inputs(300, 72, mode, BF, BF)
    for made, asked in ((False, True), (True, False)):
        with pytest.raises(AssertionError):
            check(plain(ins[0], ins[1], mode, made, *ins[2:]), ins, mode, asked)
