"""GPU parity of the layer operators (add + RMS norm, projection, gated
recurrence) against the fp64 oracle through the public calls.

Tolerances. A stored value is off by at most half a step of its type, eps/2 of
its size (2^-4 for e4m3, and 2^-10 below its normal range), plus the fp32
rounding of what precedes it, which each helper counts: E24 = 2^-24 is fp32's."""

import numpy as np
import pytest
import torch

import kimi_delta_attention_04_gb300 as kda
from kimi_delta_attention_04_gb300 import _lib
from oracle import layer_oracle as lo

from kda_cases import Canary, np64

pytestmark = pytest.mark.gpu
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
E24 = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kimi_delta_attention_04_gb300 import build
    build.build()
    kda.load()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def within(got, ref, dtype, err):
    """|got - ref| <= err (of the fp32 computation) and the rounding of ref + err."""
    got = np64(got) if isinstance(got, torch.Tensor) else got
    bound = err + half_step(dtype) * (np.abs(ref) + err) + 1e-37
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.max(np.abs(got - ref) / bound):.2f} times the bound"


def randn(gen, *shape, dtype=F32):
    return torch.randn(*shape, generator=gen).to(dtype)


def strided(t, pad=3):
    """The same values as rows of a wider buffer whose gaps hold NaN."""
    wide = torch.full((*t.shape[:-1], t.shape[-1] + pad), float("nan"), device="cuda").to(t.dtype)
    wide[..., :t.shape[-1]] = t.cuda()
    return wide[..., :t.shape[-1]]


# --- norm ---

def norm_error(ref, D):
    # sum of squares: at most D/32 + 16 dependent fp32 additions of one sign, halved by the root;
    # then root, quotient and three products
    return np.abs(ref) * E24 * (D / 64 + 32)


def check_norm(y, scale, ro, x, res, w, eps, out_dtype):
    D = x.shape[-1]
    ref, r = lo.add_rmsnorm(np64(x), None if res is None else np64(res), np64(w), eps)
    if ro is not None:
        within(ro, r, x.dtype, np.abs(r) * E24)
    if out_dtype != E4:
        within(y, ref, out_dtype, norm_error(ref, D))
        return
    s = lo.row_scale(ref)
    assert np.all(np.abs(np64(scale) - s) <= s * E24 * (D / 64 + 40))
    q = ref / s[..., None]
    # below 2^-6 an e4m3 step is 2^-9, half of it 2^-10
    err = norm_error(q, D) * 3
    assert np.all(np.abs(np64(y.float()) - q) <= err + np.maximum(2.0 ** -4 * (np.abs(q) + err), 2.0 ** -10))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("out_dtype", [BF, F32, E4])
@pytest.mark.parametrize("R,D", [(1, 1), (3, 7), (5, 64), (2, 129), (37, 1000), (9, 4096), (4, 8200), (2, 20001)])
def test_add_rmsnorm(dtype, out_dtype, R, D):
    gen = torch.Generator().manual_seed(R * 100003 + D)
    x = randn(gen, R, D, dtype=dtype)
    res = (randn(gen, R, D) * torch.logspace(-2, 2, R)[:, None]).to(dtype)
    w = randn(gen, D)
    cn = Canary()
    y, ro = cn.empty((R, D), out_dtype, name="y"), cn.empty((R, D), dtype, name="residual")
    scale = cn.empty((R,), F32, name="scale") if out_dtype == E4 else None
    kda.kda_add_rmsnorm(x.cuda(), w.cuda(), eps=1e-6, residual=res.cuda(), residual_out=ro, out=y, out_scale=scale)
    cn.check()
    check_norm(y, scale, ro, x, res, w, 1e-6, out_dtype)
    y, scale, ro = kda.kda_add_rmsnorm(x.cuda(), w.cuda(), eps=1e-6, out_dtype=out_dtype)
    assert ro is None
    check_norm(y, scale, None, x, None, w, 1e-6, out_dtype)


@pytest.mark.parametrize("D", [96, 101])
def test_add_rmsnorm_strides_and_in_place(D):
    gen = torch.Generator().manual_seed(D)
    x, res, w = randn(gen, 3, 5, D, dtype=BF), randn(gen, 3, 5, D, dtype=BF), randn(gen, D)
    xs, rs = strided(x), strided(res, 8)
    y, s, ro = kda.kda_add_rmsnorm(xs, w.cuda(), eps=1e-5, residual=rs, residual_out=rs, out_dtype=E4)
    assert ro is rs and s.shape == (3, 5)
    check_norm(y, s, rs, x, res, w, 1e-5, E4)
    kda.kda_add_rmsnorm(xs, w.cuda(), eps=1e-5, out=xs)
    check_norm(xs, None, None, x, None, w, 1e-5, BF)


def test_add_rmsnorm_rows_of_zero_nan_inf():
    D = 200
    x = torch.ones(5, D)
    x[0], x[1, 3], x[2, 150] = 0, float("nan"), float("inf")
    x[3] = 1e-30
    for out_dtype in (BF, E4):
        y, s, _ = kda.kda_add_rmsnorm(x.cuda(), torch.ones(D).cuda(), eps=0.0 if out_dtype == E4 else 1e-6,
                                      out_dtype=out_dtype)
        y = y.float().cpu()
        assert torch.isnan(y[1]).all() and torch.isnan(y[2, 150])
        if out_dtype == BF:  # with eps a row of zeros stays zero, a tiny one goes to x / sqrt(eps)
            assert (y[0] == 0).all() and (y[4] == 1).all()
        else:  # eps 0: the zero row is 0 / 0
            assert s[4].item() == pytest.approx(1 / 448, rel=1e-6) and (y[4] == 448).all()
    y, s, _ = kda.kda_add_rmsnorm(x.cuda(), torch.ones(D).cuda(), eps=1e-6, out_dtype=E4)
    assert (y[0].float() == 0).all() and s[0] == 1 and s[1] == 1


# --- projection ---

def linear_inputs(gen, M, N, K, dtype):
    x, w = randn(gen, M, K), randn(gen, N, K) / K ** 0.5
    if dtype == BF:
        return x.to(BF), w.to(BF), None, None
    xs, ws = torch.rand(M, generator=gen) + 0.01, torch.rand(N, generator=gen) + 0.01
    return (20 * x).to(E4), (100 * w).to(E4), xs, ws


def check_linear(y, x, w, xs, ws, bias=None, act="none", res=None):
    f = lambda t: None if t is None else np64(t.float())  # noqa: E731
    ref = lo.linear(f(x), f(w), x_scale=f(xs), w_scale=f(ws), bias=f(bias), activation=act, residual=f(res))
    size = np.abs(f(x)) @ np.abs(f(w)).T
    if xs is not None:
        size = size * f(xs)[:, None] * f(ws)
    # products of two bf16 or e4m3 values are exact; K sums in fp32 (each off by a step, 2 E24, at most),
    # scales, bias; the activations' slopes stay below 1.2 and their own error below 16 E24 of their argument
    v = size + (0 if bias is None else np.abs(f(bias)))
    err = 1.2 * v * E24 * (2 * x.shape[-1] + 24) + (0 if res is None else np.abs(f(res)) * E24)
    within(y, ref, y.dtype, err)


SHAPES = [(1, 1, 1), (1, 128, 64), (2, 130, 40), (7, 64, 1000), (16, 512, 256), (33, 100, 24), (64, 256, 512), (65, 129, 136),
          (128, 384, 1024), (129, 127, 72), (257, 300, 520), (300, 1111, 1001), (512, 640, 2048)]


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear_plain(dtype, M, N, K):
    gen = torch.Generator().manual_seed(M * 7919 + N * 31 + K)
    x, w, xs, ws = linear_inputs(gen, M, N, K, dtype)
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    for out_dtype in (BF, F32):
        cn = Canary()
        y = cn.empty((M, N), out_dtype, name="y")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        kda.kda_linear(x.cuda(), w.cuda(), x_scale=cuda(xs), w_scale=cuda(ws), out=y, err=err)
        cn.check()
        assert err.item() == 0
        check_linear(y, x, w, xs, ws)


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "sigmoid", "relu"])
@pytest.mark.parametrize("M,N,K", [(5, 200, 96), (140, 260, 160)])
def test_linear_epilogue(act, M, N, K):
    gen = torch.Generator().manual_seed(M + N)
    for dtype, out_dtype in ((BF, BF), (E4, BF), (BF, F32)):
        x, w, xs, ws = linear_inputs(gen, M, N, K, dtype)
        bias, res = 3 * randn(gen, N), randn(gen, M, N, dtype=out_dtype)
        cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
        y = kda.kda_linear(x.cuda(), w.cuda(), bias=bias.cuda(), activation=act, residual=res.cuda(), x_scale=cuda(xs),
                           w_scale=cuda(ws), out_dtype=out_dtype)
        check_linear(y, x, w, xs, ws, bias, act, res)


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("pad", [1, 16])
@pytest.mark.parametrize("M", [3, 150])
def test_linear_strided_rows(dtype, pad, M):
    """Rows of wider buffers whose gaps hold NaN (16 elements: aligned rows; 1: not),
    a leading axis of heads, and an output that is the residual."""
    N, K = 144, 208
    gen = torch.Generator().manual_seed(pad)
    x, w, xs, ws = linear_inputs(gen, 2 * M, N, K, dtype)
    res = randn(gen, 2, M, N, dtype=BF)
    cuda = lambda t, s: None if t is None else t.reshape(s).cuda()  # noqa: E731
    out = strided(res, 5)
    y = kda.kda_linear(strided(x.reshape(2, M, K), pad), strided(w, pad), x_scale=cuda(xs, (2, M)), w_scale=cuda(ws, (N,)),
                       residual=out, out=out)
    assert y is out
    check_linear(out.reshape(2 * M, N), x, w, xs, ws, res=res.reshape(2 * M, N))


def test_linear_start_off_alignment():
    gen = torch.Generator().manual_seed(5)
    base = randn(gen, 70, 136, dtype=BF).cuda()
    w = randn(gen, 90, 128, dtype=BF)
    y = kda.kda_linear(base[:, 3:131], w.cuda())
    check_linear(y, base[:, 3:131].cpu(), w, None, None)


def test_linear_workspace_of_the_caller():
    gen = torch.Generator().manual_seed(15)
    x, w = randn(gen, 40, 51, dtype=BF), randn(gen, 30, 51, dtype=BF)
    cn = Canary()
    need = 2 * (40 * 112 // 256 + 1) * 256
    ws = cn.empty((need,), torch.uint8, name="workspace")
    y = kda.kda_linear(x.cuda(), w.cuda(), workspace=ws)
    cn.check()
    check_linear(y, x, w, None, None)
    with pytest.raises(ValueError, match="workspace"):
        kda.kda_linear(x.cuda(), w.cuda(), workspace=ws[:256])


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("start", [0, 1, 2, 3, 5])
@pytest.mark.parametrize("M,N,K", [(3, 5, 1), (9, 140, 2), (20, 130, 3), (70, 129, 61), (16, 300, 259), (130, 200, 1030)])
def test_linear_rows_at_any_byte(dtype, start, M, N, K):
    """Contiguous rows of any pitch from an operand that starts at any element."""
    gen = torch.Generator().manual_seed(M * K + start)
    x, w, xs, ws = linear_inputs(gen, M, N, K, dtype)

    def moved(t):
        buf = torch.full((t.numel() + start + 8,), float("nan"), device="cuda").to(t.dtype)
        buf[start:start + t.numel()] = t.cuda().flatten()
        return buf[start:start + t.numel()].view(t.shape)

    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    cn = Canary()
    y = cn.empty((M, N), BF, name="y")
    kda.kda_linear(moved(x), moved(w), x_scale=cuda(xs), w_scale=cuda(ws), out=y)
    cn.check()
    check_linear(y, x, w, xs, ws)


@pytest.mark.parametrize("M,N,K", [(9, 140, 515), (300, 260, 129)])
def test_linear_calls_in_turn_share_a_workspace(M, N, K):
    """Copies of one call's operands after the products of the call before, eager and captured."""
    gen = torch.Generator().manual_seed(M)
    ops = [tuple(t.cuda() for t in (randn(gen, M, K, dtype=BF), randn(gen, N, K, dtype=BF))) for _ in range(4)]
    alone = [kda.kda_linear(x, w) for x, w in ops]
    scratch = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    for _ in range(5):
        got = [kda.kda_linear(x, w, workspace=scratch) for x, w in ops]
        assert all(torch.equal(a, b) for a, b in zip(alone, got))
    out = [torch.empty_like(y) for y in alone]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for (x, w), y in zip(ops, out):
            kda.kda_linear(x, w, workspace=scratch, out=y)
    for _ in range(20):
        graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(alone, out))


def test_linear_nan_and_inf_stay_in_their_rows():
    gen = torch.Generator().manual_seed(6)
    for M in (20, 300):
        x, w = randn(gen, M, 200, dtype=BF), randn(gen, 150, 200, dtype=BF)
        good = kda.kda_linear(x.cuda(), w.cuda())
        x[3, 7], w[11, 9] = float("nan"), float("inf")
        y = kda.kda_linear(x.cuda(), w.cuda()).cpu()
        assert torch.isnan(y[3]).all() and not torch.isfinite(y[:, 11]).any()
        keep = torch.ones(M, 150, dtype=torch.bool)
        keep[3], keep[:, 11] = False, False
        assert torch.equal(y[keep], good.cpu()[keep])


def test_linear_repeats_bit_for_bit():
    gen = torch.Generator().manual_seed(8)
    for M, N, K in ((16, 512, 4096), (700, 500, 1000)):
        x, w = randn(gen, M, K, dtype=BF).cuda(), randn(gen, N, K, dtype=BF).cuda()
        first = kda.kda_linear(x, w)
        for _ in range(5):
            assert torch.equal(kda.kda_linear(x, w), first)


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("M,N,K", [(100, 1024, 512), (128, 30000, 80), (3000, 5008, 64), (2500, 4999, 144), (200, 12288, 48),
                                   (70, 20000, 33), (1300, 2100, 65), (130, 200, 6000), (70, 300, 8005)])
def test_linear_many_tiles(dtype, M, N, K):
    """Several tiles for each SM (both accumulators in turn), widths that divide nothing,
    and few tiles with a long K, split over clusters."""
    gen = torch.Generator().manual_seed(M + N + K)
    x, w, xs, ws = linear_inputs(gen, M, N, K, dtype)
    res = randn(gen, M, N, dtype=BF)
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    cn = Canary()
    y = cn.empty((M, N), BF, name="y")
    kda.kda_linear(x.cuda(), w.cuda(), x_scale=cuda(xs), w_scale=cuda(ws), residual=res.cuda(), out=y)
    cn.check()
    check_linear(y, x, w, xs, ws, res=res)


# --- recurrence ---

def scan_inputs(gen, B, T, D, dtype, gate_dtype, mode):
    f = randn(gen, B, T, D) + 6 * torch.rand(D, generator=gen)
    gate = (f if mode == "logits" else torch.nn.functional.logsigmoid(f)).to(gate_dtype)
    return randn(gen, B, T, D, dtype=dtype), gate


def sequences(B, T, cu):
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    return [(0, int(cu[i]), int(cu[i + 1])) for i in range(len(cu) - 1)]


# fp32 steps a token: decay (exponential, quotient, 1 - a: 8), its product with the state, the sum; the
# chunked order of the products adds one more rounding of the decay per token
PER_TOKEN = 12


def check_scan(y, hT, x, gate, mode, comp, h0, cu=None):
    B, T, D = x.shape
    xs, gs = np64(x), np64(gate)
    for n, (b, s, e) in enumerate(sequences(B, T, cu)):
        h = None if h0 is None else np64(h0[n])
        ref, last, _ = lo.scan(xs[b, s:e], gs[b, s:e], gate_mode=mode, complement=comp, h0=h)
        size, _, _ = lo.scan(np.abs(xs[b, s:e]), gs[b, s:e], gate_mode=mode, complement=False,
                             h0=None if h is None else np.abs(h))
        err, elast, _ = lo.scan(PER_TOKEN * E24 * size, gs[b, s:e], gate_mode=mode, complement=False)
        if e > s:
            within(y[b, s:e], ref, y.dtype, err)
        if hT is not None:
            within(hT[n], last, F32, elast)


def check_scan_grad(dx, dgate, dh0, x, gate, dy, mode, comp, h0, dhT, cu=None):
    B, T, D = x.shape
    xs, gs, ds = np64(x), np64(gate), np64(dy)
    for n, (b, s, e) in enumerate(sequences(B, T, cu)):
        xx, gg, dd = xs[b, s:e], gs[b, s:e], ds[b, s:e]
        a = lo.scan_decay(gg, mode)
        h = np.zeros(D) if h0 is None else np64(h0[n])
        dT = np.zeros(D) if dhT is None else np64(dhT[n])
        rx, rg, r0 = lo.scan_grad(xx, gg, dd, gate_mode=mode, complement=comp, h0=h, dhT=dT)
        # sizes and errors of the states before each token and of the d's, as sums of magnitudes
        _, _, hsize = lo.scan(np.abs(xx), gg, gate_mode=mode, complement=False, h0=np.abs(h))
        size, _, _ = lo.scan(np.abs(xx), gg, gate_mode=mode, complement=False, h0=np.abs(h))
        _, _, herr = lo.scan(PER_TOKEN * E24 * size, gg, gate_mode=mode, complement=False)
        dsize, derr = np.zeros_like(xx), np.zeros_like(xx)
        ca, ce = np.abs(dT), np.zeros(D)
        for t in range(e - s - 1, -1, -1):
            dsize[t] = ca + np.abs(dd[t])
            derr[t] = ce + PER_TOKEN * E24 * dsize[t]
            ca, ce = a[t] * dsize[t], a[t] * derr[t]
        w = (1 - a) if comp else np.ones_like(a)
        if e > s:
            within(dx[b, s:e], rx, dx.dtype, w * derr + 8 * E24 * dsize)
            k = a if mode == "log" else a * (1 - a)
            both = hsize + (np.abs(xx) if comp else 0)
            within(dgate[b, s:e], rg, dgate.dtype, k * (derr * both + dsize * herr) + 16 * E24 * a * dsize * both)
        if dh0 is not None:
            within(dh0[n], r0, F32, ce + 8 * E24 * ca)


TYPES = [(BF, BF), (BF, F32), (F32, F32)]


@pytest.mark.parametrize("dtype,gate_dtype", TYPES)
@pytest.mark.parametrize("mode,comp", [("log", False), ("logits", True), ("log", True), ("logits", False)])
@pytest.mark.parametrize("B,T,D", [(1, 1, 1), (2, 15, 33), (1, 16, 64), (3, 17, 130), (1, 300, 200), (2, 1100, 72), (1, 2500, 37)])
def test_scan_and_gradient(dtype, gate_dtype, mode, comp, B, T, D):
    gen = torch.Generator().manual_seed(B * 1000 + T + D)
    x, gate = scan_inputs(gen, B, T, D, dtype, gate_dtype, mode)
    h0, dhT, dy = randn(gen, B, D), randn(gen, B, D), randn(gen, B, T, D, dtype=dtype)
    how = dict(gate_mode=mode, complement=comp)
    cn = Canary()
    y, hT = cn.empty((B, T, D), dtype, name="y"), cn.empty((B, D), F32, name="hT")
    states = cn.empty((kda.chunk_count(B, T), D), F32, name="states")
    xc, gc = x.cuda(), gate.cuda()
    kda.kda_scan_fwd(xc, gc, h0=h0.cuda(), y=y, hT=hT, h_chunks=states, **how)
    dx, dg, dh0 = cn.empty((B, T, D), dtype, name="dx"), cn.empty((B, T, D), gate_dtype, name="dgate"), cn.empty((B, D), F32, name="dh0")
    kda.kda_scan_bwd(xc, gc, dy.cuda(), states, dhT=dhT.cuda(), dx=dx, dgate=dg, dh0=dh0, **how)
    cn.check()
    check_scan(y, hT, x, gate, mode, comp, h0)
    check_scan_grad(dx, dg, dh0, x, gate, dy, mode, comp, h0, dhT)
    # without the optional inputs and outputs
    y2, none = kda.kda_scan_fwd(xc, gc, output_final_state=False, h_chunks=states, **how)
    assert none is None
    check_scan(y2, None, x, gate, mode, comp, None)
    dx, dg, none = kda.kda_scan_bwd(xc, gc, dy.cuda(), states, output_dh0=False, **how)
    assert none is None
    check_scan_grad(dx, dg, None, x, gate, dy, mode, comp, None, None)


@pytest.mark.parametrize("D", [40, 128])
@pytest.mark.parametrize("lens", [[5], [0, 3, 0, 0, 129, 16, 1, 0], [700, 31, 1, 256, 2000], [1] * 70, [0, 0]])
def test_scan_packed(lens, D):
    gen = torch.Generator().manual_seed(sum(lens) + D)
    T, N = sum(lens), len(lens)
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
    x, gate = scan_inputs(gen, 1, T, D, BF, BF, "logits")
    h0, dhT, dy = randn(gen, N, D), randn(gen, N, D), randn(gen, 1, T, D, dtype=BF)
    how = dict(gate_mode="logits", complement=True, cu_seqlens=cu.cuda())
    cn = Canary()
    states = cn.empty((kda.chunk_count(1, T, cu), D), F32, name="states")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, hT = kda.kda_scan_fwd(x.cuda(), gate.cuda(), h0=h0.cuda(), h_chunks=states, err=err, **how)
    dx, dg, dh0 = kda.kda_scan_bwd(x.cuda(), gate.cuda(), dy.cuda(), states, dhT=dhT.cuda(), err=err, **how)
    cn.check()
    assert err.item() == 0
    check_scan(y, hT, x, gate, "logits", True, h0, cu)
    check_scan_grad(dx, dg, dh0, x, gate, dy, "logits", True, h0, dhT, cu)


@pytest.mark.parametrize("N,D", [(256, 24), (257, 70), (3000, 8)])
def test_scan_many_sequences(N, D):
    """More packed sequences than the CTAs that take them."""
    gen = torch.Generator().manual_seed(N)
    lens = [int(v) for v in torch.randint(0, 40, (N,), generator=gen)]
    lens[N // 2] = 600
    T = sum(lens)
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
    x, gate = scan_inputs(gen, 1, T, D, BF, BF, "logits")
    h0, dhT, dy = randn(gen, N, D), randn(gen, N, D), randn(gen, 1, T, D, dtype=BF)
    how = dict(gate_mode="logits", cu_seqlens=cu.cuda())
    states = torch.empty(kda.chunk_count(1, T, cu), D, device="cuda")
    y, hT = kda.kda_scan_fwd(x.cuda(), gate.cuda(), h0=h0.cuda(), h_chunks=states, **how)
    dx, dg, dh0 = kda.kda_scan_bwd(x.cuda(), gate.cuda(), dy.cuda(), states, dhT=dhT.cuda(), **how)
    check_scan(y, hT, x, gate, "logits", False, h0, cu)
    check_scan_grad(dx, dg, dh0, x, gate, dy, "logits", False, h0, dhT, cu)


@pytest.mark.parametrize("dtype,gate_dtype", TYPES)
@pytest.mark.parametrize("D", [33, 66, 72])
@pytest.mark.parametrize("T", [1, 16, 17, 31, 33, 48, 63, 64, 65, 128, 129])
def test_scan_short_sequences(T, D, dtype, gate_dtype):
    """Lengths around those at which the number of warps and the kernel change."""
    gen = torch.Generator().manual_seed(T * D)
    N = 5
    x, gate = scan_inputs(gen, N, T, D, dtype, gate_dtype, "logits")
    h0, dhT, dy = randn(gen, N, D), randn(gen, N, D), randn(gen, N, T, D, dtype=dtype)
    how = dict(gate_mode="logits", complement=True)
    cn = Canary()
    states = cn.empty((N * -(-T // 16), D), F32, name="states")
    y, dx = cn.empty((N, T, D), dtype, name="y"), cn.empty((N, T, D), dtype, name="dx")
    dg = cn.empty((N, T, D), gate_dtype, name="dgate")
    _, hT = kda.kda_scan_fwd(x.cuda(), gate.cuda(), h0=h0.cuda(), h_chunks=states, y=y, **how)
    _, _, dh0 = kda.kda_scan_bwd(x.cuda(), gate.cuda(), dy.cuda(), states, dhT=dhT.cuda(), dx=dx, dgate=dg, **how)
    cn.check()
    check_scan(y, hT, x, gate, "logits", True, h0)
    check_scan_grad(dx, dg, dh0, x, gate, dy, "logits", True, h0, dhT)


def test_scan_many_rows():
    """More sequences of a batch, and more single tokens, than a grid's second axis."""
    N, D = 65535 + 300, 4
    x = torch.randn(N, 2, D, device="cuda")
    gate = torch.full((N, 2, D), -0.5, device="cuda")
    y, hT = kda.kda_scan_fwd(x, gate)
    a = float(np.exp(-0.5))
    # two tokens: one product, one sum
    assert torch.allclose(hT, a * x[:, 0] + x[:, 1], rtol=0, atol=1e-5) and torch.equal(y[:, 1], hT) and torch.equal(y[:, 0], x[:, 0])
    pool = torch.randn(N, D, device="cuda")
    idx = torch.arange(N - 1, -1, -1, dtype=torch.int32, device="cuda")
    out = torch.empty_like(pool)
    y = kda.kda_scan_step(x[:, 0].contiguous(), gate[:, 0].contiguous(), pool, idx, state_out=out)
    assert torch.allclose(y, a * pool.flip(0) + x[:, 0], rtol=0, atol=1e-5) and torch.equal(out.flip(0), y)


def test_scan_empty_batch_of_tokens():
    h0 = torch.randn(2, 24, device="cuda")
    x = torch.empty(2, 0, 24, dtype=BF, device="cuda")
    y, hT = kda.kda_scan_fwd(x, x, h0=h0)
    assert y.shape == x.shape and torch.equal(hT, h0)
    _, hT = kda.kda_scan_fwd(x, x)
    assert (hT == 0).all()
    dx, dg, dh0 = kda.kda_scan_bwd(x, x, x, torch.empty(0, 24, device="cuda"), dhT=h0)
    assert torch.equal(dh0, h0)


@pytest.mark.parametrize("cu", [[0, 5, 3, 10], [1, 5, 7, 10], [0, 5, 7, 9], [0, 5, 11, 10], [0, -1, 5, 10]])
def test_scan_bad_cu_seqlens(cu):
    x = torch.ones(1, 10, 48, dtype=BF, device="cuda")
    y, hT = torch.full_like(x, 7), torch.full((3, 48), 7.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    states = torch.zeros(8, 48, device="cuda")
    cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    kda.kda_scan_fwd(x, x, cu_seqlens=cu, y=y, hT=hT, err=err)
    assert err.item() == _lib.KDA_ERR_INVALID_ARG and (y == 7).all() and (hT == 7).all()
    err.zero_()
    kda.kda_scan_bwd(x, x, x, states, cu_seqlens=cu, dx=y, dgate=y.clone(), dh0=hT, err=err)
    assert err.item() == _lib.KDA_ERR_INVALID_ARG and (y == 7).all() and (hT == 7).all()


def test_scan_too_few_states():
    """Three sequences of 1 token need 3 states; room for the 1 that 3 tokens in a row would need."""
    x = torch.ones(1, 3, 8, dtype=BF, device="cuda")
    cu = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cn = Canary()
    states = cn.empty((1, 8), F32, name="states")
    kda.kda_scan_fwd(x, x, cu_seqlens=cu, h_chunks=states, err=err)
    cn.check()
    assert err.item() == _lib.KDA_ERR_INVALID_ARG


@pytest.mark.parametrize("D,pad", [(64, 64), (64, 1), (33, 33)])
def test_scan_views_of_one_projection(D, pad):
    """x and gate as halves of one packed row, gradients in place."""
    gen = torch.Generator().manual_seed(D + pad)
    B, T = 2, 150
    x, gate = scan_inputs(gen, B, T, D, BF, BF, "log")
    packed = torch.full((B, T, 2 * D + pad), float("nan"), dtype=BF, device="cuda")
    packed[..., :D], packed[..., D:2 * D] = x.cuda(), gate.cuda()
    xv, gv = packed[..., :D], packed[..., D:2 * D]
    states = torch.empty(kda.chunk_count(B, T), D, device="cuda")
    y, hT = kda.kda_scan_fwd(xv, gv, h_chunks=states)
    check_scan(y, hT, x, gate, "log", False, None)
    dy = randn(gen, B, T, D, dtype=BF)
    _, _, dh0 = kda.kda_scan_bwd(xv, gv, dy.cuda(), states, dx=xv, dgate=gv)
    check_scan_grad(packed[..., :D], packed[..., D:2 * D], dh0, x, gate, dy, "log", False, None, None)
    assert torch.isnan(packed[..., 2 * D:]).all()


def test_scan_extreme_gates():
    """Decays of exactly 0 and 1, logits far outside the exponential's range, and
    a NaN that stays in its channel and after its token."""
    T, D = 100, 70
    gen = torch.Generator().manual_seed(9)
    x = randn(gen, 1, T, D)
    gate = torch.zeros(1, T, D)
    gate[0, ::7, :30] = float("-inf")          # reset
    y, hT = kda.kda_scan_fwd(x.cuda(), gate.cuda())
    check_scan(y, hT, x, gate, "log", False, None)
    gate = torch.where(torch.rand(1, T, D, generator=gen) < 0.5, 300.0, -300.0)
    y, hT = kda.kda_scan_fwd(x.cuda(), gate.cuda(), gate_mode="logits", complement=True)
    with np.errstate(over="ignore"):
        check_scan(y, hT, x, gate, "logits", True, None)
    x[0, 40, 5] = float("nan")
    y, _ = kda.kda_scan_fwd(x.cuda(), torch.full_like(x, -0.1).cuda())
    nan = torch.isnan(y[0]).cpu()
    assert nan[40:, 5].all() and not nan[:40].any() and not nan[:, :5].any() and not nan[:, 6:].any()


@pytest.mark.parametrize("dtype,gate_dtype", TYPES)
@pytest.mark.parametrize("B,D", [(1, 1), (3, 50), (40, 257), (9, 1024)])
def test_scan_step(dtype, gate_dtype, B, D):
    gen = torch.Generator().manual_seed(B * D)
    slots = B + 5
    for mode, comp in (("log", False), ("logits", True)):
        x, gate = scan_inputs(gen, 1, B, D, dtype, gate_dtype, mode)
        x, gate = x[0], gate[0]
        pool = randn(gen, slots, D)
        idx = torch.randperm(slots, generator=gen)[:B].to(torch.int32)
        idx[::4] = -1
        if B > 2:
            idx[1] = slots + 3  # out of range: reported, treated as padding
        cn = Canary()
        y, other = cn.empty((B, D), dtype, name="y"), cn.clone(torch.full((slots, D), 5.0, device="cuda"), name="pool")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        how = dict(gate_mode=mode, complement=comp)
        kda.kda_scan_step(strided(x), strided(gate), pool.cuda(), idx.cuda(), state_out=other, y=y, err=err, **how)
        cn.check()
        assert err.item() == (_lib.KDA_ERR_INVALID_ARG if B > 2 else 0)
        inplace = pool.cuda()
        y2 = kda.kda_scan_step(x.cuda(), gate.cuda(), inplace, idx.cuda(), **how)
        assert torch.equal(y2, y)
        seen = set()
        for b in range(B):
            s = int(idx[b])
            if not 0 <= s < slots:
                assert (y[b] == 0).all()
                continue
            seen.add(s)
            check_scan(y[b].view(1, 1, D), other[s].view(1, D), x[b].view(1, 1, D), gate[b].view(1, 1, D), mode, comp,
                       pool[s].view(1, D))
            assert torch.equal(inplace[s], other[s])
        for s in set(range(slots)) - seen:
            assert (other[s] == 5).all() and torch.equal(inplace[s].cpu(), pool[s])


def test_scan_step_reports_repeated_slots():
    x = torch.ones(3, 8, dtype=BF, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    idx = torch.tensor([2, 1, 1], dtype=torch.int32, device="cuda")
    kda.kda_scan_step(x, x, torch.zeros(4, 8, device="cuda"), idx, err=err, check_indices=True)
    assert err.item() == _lib.KDA_ERR_INVALID_ARG


def test_scan_step_continues_a_prefill():
    """A prefill's hT in a slot, then single tokens: the same as one longer scan."""
    gen = torch.Generator().manual_seed(12)
    x, gate = scan_inputs(gen, 1, 60, 90, F32, F32, "logits")
    how = dict(gate_mode="logits", complement=True)
    _, hT = kda.kda_scan_fwd(x[:, :50].contiguous().cuda(), gate[:, :50].contiguous().cuda(), **how)
    pool = torch.zeros(2, 90, device="cuda")
    pool[1] = hT[0]
    idx = torch.tensor([1], dtype=torch.int32, device="cuda")
    ys = [kda.kda_scan_step(x[:, t].cuda(), gate[:, t].cuda(), pool, idx, **how) for t in range(50, 60)]
    ref, last, _ = lo.scan(np64(x[0]), np64(gate[0]), gate_mode="logits", complement=True)
    assert np.allclose(np64(torch.cat(ys)), ref[50:], atol=1e-5) and np.allclose(np64(pool[1]), last, atol=1e-5)


# --- streams and graphs ---

def test_layer_calls_on_a_side_stream_and_in_a_graph():
    gen = torch.Generator().manual_seed(3)
    M, D = 48, 96
    x, w, nw = randn(gen, 1, M, D, dtype=BF).cuda(), randn(gen, 2 * D, D, dtype=BF).cuda(), randn(gen, D).cuda()

    def layer(stream=None):
        y, _, _ = kda.kda_add_rmsnorm(x, nw, eps=1e-6, residual=x, stream=stream)
        p = kda.kda_linear(y, w, activation="silu", stream=stream)
        states = torch.empty(kda.chunk_count(1, M), D, device="cuda")
        h, _ = kda.kda_scan_fwd(p[..., :D], p[..., D:], gate_mode="logits", complement=True, h_chunks=states, stream=stream)
        return (h, *kda.kda_scan_bwd(p[..., :D], p[..., D:], h, states, gate_mode="logits", complement=True, stream=stream))

    want = layer()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = layer(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer()
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# --- sizes past 32 bits ---

def test_layer_offsets_past_32_bits():
    """More than 2^31 elements in each tensor: the last rows against the same rows alone."""
    T, D, tail = 2 ** 19 + 1000, 4104, 64
    x = torch.ones(1, T, D, dtype=BF, device="cuda")
    gate = torch.zeros(1, T, D, dtype=BF, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(17)
    x[:, -tail:] = torch.randn(1, tail, D, generator=gen, device="cuda")
    gate[:, -tail:] = torch.randn(1, tail, D, generator=gen, device="cuda")
    how = dict(gate_mode="logits", complement=True)  # a = 1/2 of ones before the tail: the state there is 1
    states = torch.empty(kda.chunk_count(1, T), D, device="cuda")
    y, hT = kda.kda_scan_fwd(x, gate, h_chunks=states, **how)
    one = torch.ones(1, D, device="cuda")
    xt, gt = x[:, -tail:].contiguous(), gate[:, -tail:].contiguous()
    states_t = torch.empty(kda.chunk_count(1, tail), D, device="cuda")
    yt, hTt = kda.kda_scan_fwd(xt, gt, h0=one, h_chunks=states_t, **how)
    # 64 tokens of decays <= 1 from the same state, composed in other groups
    assert torch.allclose(hT, hTt, rtol=0, atol=64 * PER_TOKEN * E24 * 8)
    assert torch.allclose(y[:, -tail:].float(), yt.float(), rtol=2 * half_step(BF), atol=1e-4)
    dx, dg, _ = kda.kda_scan_bwd(x, gate, y, states, **how)
    dxt, dgt, _ = kda.kda_scan_bwd(xt, gt, y[:, -tail:].contiguous(), states_t, **how)
    assert torch.allclose(dx[:, -tail:].float(), dxt.float(), rtol=2 * half_step(BF), atol=1e-4)
    assert torch.allclose(dg[:, -tail:].float(), dgt.float(), rtol=2 * half_step(BF), atol=1e-4)
    del y, dx, dg, states
    w = torch.ones(D, device="cuda")
    for a, b in zip(kda.kda_add_rmsnorm(x, w, eps=1e-6, residual=gate, out_dtype=E4),
                    kda.kda_add_rmsnorm(xt, w, eps=1e-6, residual=gt, out_dtype=E4)):
        assert torch.equal(a[:, -tail:].contiguous().view(torch.uint8), b.view(torch.uint8))
    wide = torch.randn(24, D, generator=gen, device="cuda").to(BF)
    check_linear(kda.kda_linear(x, wide)[0, -200:], x[0, -200:].cpu(), wide.cpu(), None, None)
