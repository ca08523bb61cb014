"""The projection's epilogue on every way it reads and writes rows, with the sum of one
SM, of a pair and of a cluster that splits K; and the packed q|k|v row that a
projection makes, taken on by the decode step and the chunk forward."""

import numpy as np
import pytest
import torch

import kimi_delta_attention_04_gb300 as kda
from kimi_delta_attention_04_gb300 import workloads as W
from oracle import kda_oracle as ko
from oracle import layer_oracle as lo

from kda_cases import Canary, assert_close, np64
from test_gpu_layer import BF, E24, E4, F32, check_linear, linear_inputs, randn, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kimi_delta_attention_04_gb300 import build
    build.build()
    kda.load()


# (rows of 32-byte, 16-byte and any alignment: N a multiple of 16, of 8, of neither)
SHAPES = [(7, 272, 96),                                             # few tokens
          (100, 272, 96), (100, 264, 96), (100, 261, 96),           # one SM a tile
          (300, 272, 96), (300, 264, 96), (300, 261, 96), (129, 5008, 72),  # pairs
          (16, 384, 4096), (128, 512, 4096), (100, 200, 8005)]      # K split over a cluster


def check(y, x, w, xs, ws, bias, act, res):
    """K exact products summed in fp32 (each sum off by a step, 2 E24, at most), scales, bias,
    carried over with slopes up to 1.2; the activation's own error as kda.h has it: 20 half steps
    of its result (which for a sigmoid is 1/2 where its argument is 0) and 1.5 times what half a
    step of the argument comes to; the residual's sum."""
    f = lambda t: None if t is None else np64(t.float())  # noqa: E731
    v = lo.linear(f(x), f(w), x_scale=f(xs), w_scale=f(ws), bias=f(bias))
    size = np.abs(f(x)) @ np.abs(f(w)).T
    if xs is not None:
        size = size * f(xs)[:, None] * f(ws)
    err = 1.2 * (size + (0 if bias is None else np.abs(f(bias)))) * E24 * (2 * x.shape[-1] + 24)
    a = lo.activate(v if act in ("none", "relu") else np.clip(v, -700, None), act)
    slope = {"gelu": v * v, "silu": np.abs(v), "sigmoid": np.abs(v)}.get(act)
    if slope is not None:
        err = err + E24 * (20 + 1.5 * slope) * np.abs(a)
    ref = a if res is None else a + f(res)
    within(y, ref, y.dtype, err + (0 if res is None else np.abs(f(res)) * E24))


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "sigmoid", "relu"])
@pytest.mark.parametrize("dtype,out_dtype", [(BF, BF), (BF, F32), (E4, BF), (E4, F32)])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_epilogue(act, dtype, out_dtype, M, N, K):
    gen = torch.Generator().manual_seed(M + N + K)
    x, w, xs, ws = linear_inputs(gen, M, N, K, dtype)
    if dtype == E4:  # arguments of a few units, so that the activations are neither flat nor straight
        xs, ws = xs / 20, ws / 100
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    for bias, res in ((True, True), (True, False), (False, True)):
        b = 3 * randn(gen, N) if bias else None
        r = randn(gen, M, N, dtype=out_dtype) if res else None
        cn = Canary()
        y = cn.empty((M, N), out_dtype, name="y")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        kda.kda_linear(x.cuda(), w.cuda(), bias=cuda(b), activation=act, residual=cuda(r), x_scale=cuda(xs), w_scale=cuda(ws),
                       out=y, err=err)
        cn.check()
        assert err.item() == 0
        check(y, x, w, xs, ws, b, act, r)
        if res:  # and in the residual's place
            z = cn.clone(r.cuda(), name="residual")
            kda.kda_linear(x.cuda(), w.cuda(), bias=cuda(b), activation=act, residual=z, x_scale=cuda(xs), w_scale=cuda(ws), out=z)
            cn.check()
            assert torch.equal(z, y)


@pytest.mark.parametrize("dtype", [BF, E4])
def test_projected_row_into_the_decode_step(dtype):
    """norm -> q|k|v projection -> decode, each against its own definition on what it was given."""
    gen = torch.Generator().manual_seed(1)
    d = W.decode_workload(seed=8, B=40, H=2, HV=2, num_slots=64)
    D, C = 512, d["packed_qkv"].shape[1]
    x, res, nw = randn(gen, 40, D, dtype=BF), randn(gen, 40, D, dtype=BF), 1 + 0.1 * randn(gen, D)
    n, scale, _ = kda.kda_add_rmsnorm(x.cuda(), nw.cuda(), eps=1e-6, residual=res.cuda(), out_dtype=dtype)
    w, ws = randn(gen, C, D) / D ** 0.5, None
    if dtype == E4:
        ws = w.abs().amax(1) / 448
        w = w / ws[:, None]
    w = w.to(dtype)
    packed = kda.kda_linear(n, w.cuda(), x_scale=scale, w_scale=None if ws is None else ws.cuda())
    check_linear(packed, n.cpu(), w, None if scale is None else scale.cpu(), ws)
    dev = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in d.items()}
    o = kda.kda_decode_step(packed, dev["a"], dev["b"], dev["A_log"], dev["dt_bias"], dev["state_pool"], dev["indices"],
                            H=2, HV=2, K=128, V=128, scale=d["scale"])
    ref, pool = ko.kda_decode(np64(packed), np64(d["a"]), np64(d["b"]), np64(d["A_log"]), np64(d["dt_bias"]), np64(d["state_pool"]),
                              d["indices"].numpy(), H=2, HV=2, K=128, V=128, scale=d["scale"])
    assert_close("o", np64(o), ref, BF)
    assert_close("states", np64(dev["state_pool"]), pool, F32)


def test_projected_rows_into_the_chunk_forward():
    gen = torch.Generator().manual_seed(2)
    wl = W.prefill(T=100, H=2, seed=9)
    T, H, D = 100, 2, 384
    x, w = randn(gen, 1, T, D, dtype=BF), (randn(gen, 3 * H * 128, D) / D ** 0.5).to(BF)
    packed = kda.kda_linear(x.cuda(), w.cuda())
    check_linear(packed[0], x[0], w, None, None)
    q, k, v = (t.reshape(1, T, H, 128).contiguous() for t in packed.chunk(3, -1))
    dev = {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in wl.items()}
    o, hT = kda.kda_chunk_fwd(q, k, v, scale=wl["scale"], a=dev["a"], dt_bias=dev["dt_bias"], A_log=dev["A_log"], b=dev["b"],
                              h0=dev["h0"], l2norm_qk=True)
    ref, last = ko.kda_forward(np64(q), np64(k), np64(v), scale=wl["scale"], a=np64(wl["a"]), dt_bias=np64(wl["dt_bias"]),
                               A_log=np64(wl["A_log"]), b=np64(wl["b"]), h0=np64(wl["h0"]), l2norm_qk=True)
    assert_close("o", np64(o), ref, BF)
    assert_close("hT", np64(hT), last, BF)
    assert np.isfinite(ref).all()
