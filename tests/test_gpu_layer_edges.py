"""The layer operators where their arithmetic or their sizes end: infinite inputs
and states, rows outside the range of a sum of squares, gates far from zero, sizes
next to 2^31. Against the fp64 oracle; E24 is half a step of fp32, relative."""

import math

import numpy as np
import pytest
import torch

import kimi_delta_attention_04_gb300 as kda
from oracle import layer_oracle as lo

from kda_cases import np64
from test_gpu_layer import BF, E4, E24, F32, check_norm, randn, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kimi_delta_attention_04_gb300 import build
    build.build()
    kda.load()


def same_or_within(got, ref, err):
    """Infinities and NaN in the same places, the rest within err and fp32's rounding."""
    got, odd = np64(got), ~np.isfinite(ref)
    assert np.array_equal(got[odd], ref[odd], equal_nan=True), f"{(got[odd] != ref[odd]).sum()} of {odd.sum()} differ"
    within(got[~odd], ref[~odd], F32, np.broadcast_to(err, ref.shape)[~odd])


# --- sizes next to 2^31 ---

@pytest.mark.parametrize("dtype", [BF, E4])
def test_linear_k_next_to_2_31(dtype):
    """One row of 2^31 - 1 values against another: the last block of K is not whole."""
    K = 2 ** 31 - 1
    x, w = (torch.zeros(1, K, dtype=dtype, device="cuda") for _ in range(2))
    at = torch.tensor([0, 5, 2 ** 30, K - 129, K - 64, K - 2, K - 1], device="cuda")
    x[0, at] = torch.arange(1.0, 8.0, device="cuda").to(dtype)
    w[0, at] = torch.tensor([1.0, -1.0, 2.0, 0.5, -2.0, 1.0, 4.0], device="cuda").to(dtype)
    one = None if dtype == BF else torch.ones(1, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = kda.kda_linear(x, w, x_scale=one, w_scale=one, out_dtype=F32, err=err)
    assert err.item() == 0
    assert y.item() == 1 - 2 + 6 + 2 - 10 + 6 + 28  # (every product and sum is exact)


@pytest.mark.parametrize("D", [2 ** 31 - 1, 2 ** 31 - 4])
def test_scan_step_channels_next_to_2_31(D):
    x = torch.zeros(1, D, dtype=BF, device="cuda")
    gate = torch.zeros(1, D, dtype=BF, device="cuda")  # a = 1
    x[0, 0], x[0, D - 1] = 2, 3
    pool = torch.zeros(1, D, device="cuda")
    pool[0, D - 1] = 5
    y = kda.kda_scan_step(x, gate, pool, torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert y[0, 0] == 2 and y[0, D - 1] == 8 and pool[0, 0] == 2 and pool[0, D - 1] == 8
    assert torch.count_nonzero(y) == 2


# --- infinite inputs ---

def infinite_inputs(mode):
    gen = torch.Generator().manual_seed(21)
    T, D = 12, 70
    x, f = randn(gen, 1, T, D), randn(gen, 1, T, D)
    gate = f if mode == "logits" else torch.nn.functional.logsigmoid(f)
    x[0, 3, 5], x[0, 7, 6], x[0, 0, 66], x[0, 11, 69] = float("inf"), float("-inf"), float("-inf"), float("inf")
    return x, gate, randn(gen, 1, D), randn(gen, 1, T, D), randn(gen, 1, D)


@pytest.mark.parametrize("mode", ["log", "logits"])
def test_scan_infinite_inputs(mode):
    """An infinite x under the weight 1 - a: the states are infinite from there on, its channel alone."""
    x, gate, h0, dy, dhT = infinite_inputs(mode)
    T, D = x.shape[1:]
    how = dict(gate_mode=mode, complement=True)
    states = torch.empty(kda.chunk_count(1, T), D, device="cuda")
    y, hT = kda.kda_scan_fwd(x.cuda(), gate.cuda(), h0=h0.cuda(), h_chunks=states, **how)
    ref, last, _ = lo.scan(np64(x[0]), np64(gate[0]), h0=np64(h0[0]), **how)
    assert np.isinf(ref[3:, 5]).all() and np.isfinite(ref[:3, 5]).all() and np.isinf(last).sum() == 4
    # 12 tokens of weights <= 1 on values below 6: at most 12 roundings of 12 steps each
    same_or_within(y[0], ref, 12 * 12 * E24 * 6)
    same_or_within(hT[0], last, 12 * 12 * E24 * 6)
    dx, dg, dh0 = kda.kda_scan_bwd(x.cuda(), gate.cuda(), dy.cuda(), states, dhT=dhT.cuda(), **how)
    rx, rg, r0 = lo.scan_grad(np64(x[0]), np64(gate[0]), np64(dy[0]), h0=np64(h0[0]), dhT=np64(dhT[0]), **how)
    same_or_within(dx[0], rx, 12 * 12 * E24 * 6)
    same_or_within(dh0[0], r0, 12 * 12 * E24 * 6)
    same_or_within(dg[0], rg, 2 * 12 * 12 * E24 * 36)


@pytest.mark.parametrize("mode", ["log", "logits"])
def test_scan_step_infinite_inputs(mode):
    x, gate, h0, _, _ = infinite_inputs(mode)
    pool = h0.cuda()
    idx = torch.zeros(1, dtype=torch.int32, device="cuda")
    for D in (70, 68):  # one channel an access, and four
        pool = h0[:, :D].contiguous().cuda()
        y = kda.kda_scan_step(x[0, 3:4, :D].contiguous().cuda(), gate[0, 3:4, :D].contiguous().cuda(), pool, idx,
                              gate_mode=mode, complement=True)
        ref, _, _ = lo.scan(np64(x[0, 3:4, :D]), np64(gate[0, 3:4, :D]), gate_mode=mode, complement=True, h0=np64(h0[0, :D]))
        assert np.isinf(ref).sum() == 1
        same_or_within(y, ref, 12 * E24 * 6)
        same_or_within(pool, ref, 12 * E24 * 6)


# --- infinite states over products of decays that leave fp32's range ---

@pytest.mark.parametrize("comp", [False, True])
@pytest.mark.parametrize("T", [40, 64, 200, 1500])
def test_scan_infinite_states_stay(T, comp):
    """h0 (and dhT) infinite, decays of e^-5 to e^-8 a token: 0 < a, so the state stays infinite,
    although the product of 32 of them is below the smallest fp32."""
    gen = torch.Generator().manual_seed(T)
    D = 70
    x, dy = randn(gen, 1, T, D), randn(gen, 1, T, D)
    gate = -5 - 3 * torch.rand(1, T, D, generator=gen)
    h0, dhT = randn(gen, 1, D), randn(gen, 1, D)
    h0[0, 7], h0[0, 40], dhT[0, 9], dhT[0, 69] = float("inf"), float("-inf"), float("-inf"), float("inf")
    x[0, T // 2, 60] = float("inf")
    h0[0, 11] = 3e38   # a finite one decays away
    how = dict(gate_mode="log", complement=comp)
    states = torch.empty(kda.chunk_count(1, T), D, device="cuda")
    y, hT = kda.kda_scan_fwd(x.cuda(), gate.cuda(), h0=h0.cuda(), h_chunks=states, **how)
    ref, last, before = lo.scan(np64(x[0]), np64(gate[0]), h0=np64(h0[0]), **how)
    assert np.isinf(ref[:, [7, 40]]).all() and np.isinf(ref[T // 2:, 60]).all()
    # decays below 1/100: a state is off by some roundings of itself and its last input; a product that
    # ends at the smallest fp32 (2^-149) is off by up to that
    err = 16 * E24 * (np.abs(np.where(np.isfinite(ref), ref, 0)) + 6) + 2.0 ** -149 * 3e38
    same_or_within(y[0], ref, err)
    same_or_within(hT[0], last, err[-1])
    dx, dg, dh0 = kda.kda_scan_bwd(x.cuda(), gate.cuda(), dy.cuda(), states, dhT=dhT.cuda(), **how)
    rx, rg, r0 = lo.scan_grad(np64(x[0]), np64(gate[0]), np64(dy[0]), h0=np64(h0[0]), dhT=np64(dhT[0]), **how)
    assert np.isinf(rx[:, [9, 69]]).all() and np.isinf(r0[[9, 69]]).all()
    fin = lambda v: np.abs(np.where(np.isfinite(v), v, 0))  # noqa: E731
    same_or_within(dx[0], rx, 16 * E24 * (fin(rx) + 6))
    same_or_within(dh0[0], r0, 16 * E24 * (fin(r0) + 6))
    same_or_within(dg[0], rg, 48 * E24 * (fin(rg) + 6 * (fin(before) + 6)))


@pytest.mark.parametrize("D", [70, 71, 72])
def test_scan_infinite_states_beside_nan(D):
    """An infinite channel next to one of NaN, in the same thread's pair and in the next."""
    T = 200
    h0 = torch.ones(1, D)
    h0[0, [7, 12, 20, 21]] = float("inf")
    h0[0, [6, 13, 39, 44, 52, 53]] = float("nan")  # (a thread holds 2 l and 2 l + 1, or l and l + 32)
    x, gate = torch.zeros(1, T, D), torch.full((1, T, D), -6.0)
    y, hT = kda.kda_scan_fwd(x.cuda(), gate.cuda(), h0=h0.cuda())
    states = torch.zeros(kda.chunk_count(1, T), D, device="cuda")
    _, _, dh0 = kda.kda_scan_bwd(x.cuda(), gate.cuda(), x.cuda(), states, dhT=h0.cuda())
    for v in (y[0, -1].cpu(), hT[0].cpu(), dh0[0].cpu()):
        assert torch.equal(torch.isinf(v), torch.isinf(h0[0])) and torch.equal(torch.isnan(v), torch.isnan(h0[0]))


def test_scan_resets_stay_exact():
    """A decay of exactly 0 lets nothing finite through, wherever it stands in its chunk, next to
    decays whose product alone leaves fp32's range."""
    gen = torch.Generator().manual_seed(2)
    T, D = 700, 66
    x = randn(gen, 1, T, D)
    gate = torch.full((1, T, D), -6.0)
    reset = torch.rand(T, D, generator=gen) < 0.05
    gate[0][reset] = float("-inf")
    x[0, ::3] = 0
    h0 = torch.full((1, D), 3e38)
    y, _ = kda.kda_scan_fwd(x.cuda(), gate.cuda(), h0=h0.cuda())
    y = y[0].cpu()
    assert torch.equal(y[reset], x[0][reset])


# --- norm: rows outside the range of a sum of squares ---

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("out_dtype", [BF, F32, E4])
@pytest.mark.parametrize("D", [96, 101, 600, 4096, 9001])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6])
def test_add_rmsnorm_large_and_small_rows(dtype, out_dtype, D, eps):
    """Finite rows whose squares leave fp32's range on either side."""
    gen = torch.Generator().manual_seed(D)
    size = torch.tensor([1e20, 6e37, 1.0, 1e-18, 1e-21, 1e-30, 1e-36, 3e18])
    x = (randn(gen, len(size), D).clamp(-4, 4) * size[:, None]).to(dtype)
    res = (randn(gen, len(size), D).clamp(-1, 1) * size[:, None] / 4).to(dtype)
    w = 1 + 0.2 * randn(gen, D)
    y, s, r = kda.kda_add_rmsnorm(x.cuda(), w.cuda(), eps=eps, residual=res.cuda(), out_dtype=out_dtype)
    check_norm(y, s, r, x, res, w, eps, out_dtype)


def test_add_rmsnorm_smallest_rows():
    """Rows of fp32's smallest values, and a single one among zeros."""
    x = torch.zeros(3, 200)
    x[0], x[1, 17], x[2, :2] = 2.0 ** -149, 2.0 ** -149, torch.tensor([2.0 ** -127, 3e38])
    w = torch.ones(200)
    y, _, _ = kda.kda_add_rmsnorm(x.cuda(), w.cuda(), eps=0.0)
    ref, _ = lo.add_rmsnorm(np64(x), None, np64(w), 0.0)
    within(y, ref, F32, np.abs(ref) * E24 * 40)


# --- gates far from zero ---

FAR = torch.linspace(-30, 30, 241)


def one_token(f, x, h0, mode, comp, dy):
    """(y, h, dx, dgate, dh0) of one token on every path that takes one."""
    D = f.numel()
    t = lambda v: v.reshape(1, 1, D).cuda()  # noqa: E731
    how = dict(gate_mode=mode, complement=comp)
    states = torch.empty(1, D, device="cuda")
    y, hT = kda.kda_scan_fwd(t(x), t(f), h0=t(h0)[0], h_chunks=states, **how)
    g = kda.kda_scan_bwd(t(x), t(f), t(dy), states, **how)
    pool = t(h0)[0].clone()
    ys = kda.kda_scan_step(t(x)[0], t(f)[0], pool, torch.zeros(1, dtype=torch.int32, device="cuda"), **how)
    # the same token as the last of 101: zero inputs and logits that keep the state before it
    T = 101
    xl, fl = torch.zeros(1, T, D), torch.full((1, T, D), 200.0 if mode == "logits" else 0.0)
    dl = torch.zeros(1, T, D)
    xl[0, -1], fl[0, -1], dl[0, -1] = x, f, dy
    states = torch.empty(kda.chunk_count(1, T), D, device="cuda")
    yl, hl = kda.kda_scan_fwd(xl.cuda(), fl.cuda(), h0=t(h0)[0], h_chunks=states, **how)
    gl = kda.kda_scan_bwd(xl.cuda(), fl.cuda(), dl.cuda(), states, **how)
    return [(y[0], hT, g[0][0], g[1][0], g[2]), (ys, pool, None, None, None), (yl[0, -1:], hl, gl[0][0, -1:], gl[1][0, -1:], gl[2])]


def test_scan_decays_far_from_zero():
    """a = sigmoid(f) to fp32, relative: exponential 4 half steps, sum 1, reciprocal 2, products 1 each."""
    f = FAR
    x, h0 = torch.zeros_like(f), 1 + torch.rand(f.numel(), generator=torch.Generator().manual_seed(1))
    ref, _, _ = lo.scan(np64(x)[None], np64(f)[None], gate_mode="logits", complement=False, h0=np64(h0))
    for y, h, _, _, dh0 in one_token(f, x, h0, "logits", False, torch.ones_like(f)):
        within(y, ref, F32, 9 * E24 * ref)
        within(h, ref, F32, 9 * E24 * ref)
        if dh0 is not None:
            within(dh0, 1 / (1 + np.exp(-np64(f)))[None], F32, 9 * E24)
            assert np.all(np.abs(np64(dh0)[0] * (1 + np.exp(-np64(f))) - 1) <= 10 * E24)


def test_scan_decays_of_bf16_gates_far_from_zero():
    """Their exponential's argument is rounded once: 1.3 |f| half steps more (the states are fp32)."""
    f = FAR.to(BF)
    h0 = 1 + torch.rand(1, f.numel(), generator=torch.Generator().manual_seed(1))
    a = 1 / (1 + np.exp(-np64(f)))
    x = torch.zeros(1, 1, f.numel(), dtype=BF, device="cuda")
    states = torch.empty(1, f.numel(), device="cuda")
    _, hT = kda.kda_scan_fwd(x, f.view(1, 1, -1).cuda(), gate_mode="logits", h0=h0.cuda(), h_chunks=states)
    _, _, dh0 = kda.kda_scan_bwd(x, f.view(1, 1, -1).cuda(), x + 1, states, gate_mode="logits")
    err = (10 + 1.3 * np.abs(np64(f))) * E24 * a
    assert np.all(np.abs(np64(hT)[0] - a * np64(h0)[0]) <= err * np64(h0)[0]) and np.all(np.abs(np64(dh0)[0] - a) <= err)


# --- 1 - a ---

@pytest.mark.parametrize("mode", ["log", "logits"])
@pytest.mark.parametrize("comp", [False, True])
def test_scan_complement_far_from_zero(mode, comp):
    """1 - a to fp32, relative: as an input's weight, in dx and in a logit's gradient."""
    f = FAR if mode == "logits" else -torch.logspace(-8, 2, 241)
    gen = torch.Generator().manual_seed(4)
    n = f.numel()
    x, h0, dy = 1 + torch.rand(n, generator=gen), torch.zeros(n), 1 + torch.rand(n, generator=gen)
    how = dict(gate_mode=mode, complement=comp)
    for grad_only in (False, True):
        if grad_only:  # a state beside the input, so that the decay's gradient is of one product
            h0 = 4 + torch.rand(n, generator=gen)
        ref, _, _ = lo.scan(np64(x)[None], np64(f)[None], h0=np64(h0), **how)
        b = -np.expm1(np64(f)) if mode == "log" else 1 / (1 + np.exp(np64(f)))
        a = np.exp(np64(f)) if mode == "log" else 1 / (1 + np.exp(-np64(f)))
        want = (b if comp else 1) * np64(x)
        rx = (b if comp else 1) * np64(dy)
        rg = a * np64(dy) * (np64(h0) - np64(x) if comp else np64(h0)) * (b if mode == "logits" else 1)
        for y, h, dx, dg, _ in one_token(f, x, h0, mode, comp, dy):
            if not grad_only:
                within(y, want[None], F32, 12 * E24 * want)
                within(h, want[None], F32, 12 * E24 * want)
            if dx is not None:
                within(dx, rx[None], F32, 12 * E24 * rx)
                within(dg, rg[None], F32, 24 * E24 * np.abs(rg))


# --- activations ---

VALUES = torch.cat([torch.linspace(-12, 12, 449), torch.logspace(-6, 0, 25), -torch.logspace(-6, 0, 25), torch.tensor([0.0, 60.0, -60.0, 80.0, -80.0])]).to(BF)


def activated(act, v):
    """act of v and the steps that half a step of v itself costs, both in 64 bits without cancellation."""
    if act == "gelu":
        return 0.5 * v * np.array([math.erfc(-u / math.sqrt(2)) for u in v]), v * v
    s = np.where(v < 0, np.exp(-np.abs(v)), 1) / (1 + np.exp(-np.abs(v)))
    return s if act == "sigmoid" else v * s, np.abs(v)


@pytest.mark.parametrize("act", ["silu", "gelu", "sigmoid"])
@pytest.mark.parametrize("rows", [3, 100, 300])
def test_linear_activations_alone(act, rows):
    """Every value as an output of its own (K = 1, ones against the values): 20 half steps of the
    result, and 1.5 times what half a step of the argument comes to, its square or product being rounded."""
    x = torch.ones(rows, 1, dtype=BF, device="cuda")
    ref, slope = activated(act, np64(VALUES))
    for out_dtype in (F32, BF):
        for n in (VALUES.numel(), VALUES.numel() // 16 * 16, VALUES.numel() // 16 * 16 - 8):  # any rows, 32 and 16 bytes
            y = kda.kda_linear(x, VALUES[:n, None].contiguous().cuda(), activation=act, out_dtype=out_dtype)
            assert torch.equal(y, y[:1].expand_as(y))
            within(y[0], ref[:n], out_dtype, (20 + 1.5 * slope[:n]) * E24 * np.abs(ref[:n]))
