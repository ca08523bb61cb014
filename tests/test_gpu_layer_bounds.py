"""The recurrence, its gradients and its step within the bounds of layer_bounds, which
follow the formulas' weights: channels with memories from two tokens to thousands, equal
and packed sequences, every pair of types, rows of any alignment."""

import numpy as np
import pytest
import torch

import kimi_delta_attention_04_gb300 as kda
import layer_bounds as lb
from test_layer_bounds_cpu import MODES, inputs

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TYPES = [(BF, BF), (BF, F32), (F32, F32)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kimi_delta_attention_04_gb300 import build
    build.build()
    kda.load()


def run_and_check(x, gate, h0, dy, dhT, mode, comp, cu=None):
    how = dict(gate_mode=mode, complement=comp, cu_seqlens=None if cu is None else cu.cuda())
    states = torch.empty(kda.chunk_count(x.shape[0], x.shape[1], cu), x.shape[2], device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    xc, gc = x.cuda(), gate.cuda()
    y, hT = kda.kda_scan_fwd(xc, gc, h0=h0.cuda(), h_chunks=states, err=err, **how)
    dx, dg, dh0 = kda.kda_scan_bwd(xc, gc, dy.cuda(), states, dhT=dhT.cuda(), err=err, **how)
    assert err.item() == 0
    lb.check_scan(dict(y=y, hT=hT, dx=dx, dgate=dg, dh0=dh0), x, gate, mode, comp, h0, dy, dhT, cu)


@pytest.mark.parametrize("mode,comp", MODES)
@pytest.mark.parametrize("dtype,gate_dtype", TYPES)
@pytest.mark.parametrize("T,D", [(1, 40), (16, 64), (17, 33), (63, 72), (300, 72), (1100, 130), (2500, 37)])
def test_one_sequence(mode, comp, dtype, gate_dtype, T, D):
    run_and_check(*inputs(T, D, mode, dtype, gate_dtype, seed=T), mode, comp)


@pytest.mark.parametrize("mode,comp", MODES)
@pytest.mark.parametrize("dtype,gate_dtype", TYPES)
@pytest.mark.parametrize("D", [33, 66, 72])
@pytest.mark.parametrize("lens", [[0, 3, 0, 129, 16, 1, 0], [700, 31, 1, 256], [7] * 300])
def test_packed(mode, comp, dtype, gate_dtype, D, lens):
    T, N = sum(lens), len(lens)
    x, gate, _, dy, _ = inputs(T, D, mode, dtype, gate_dtype, seed=D)
    gen = torch.Generator().manual_seed(N)
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
    run_and_check(x, gate, torch.randn(N, D, generator=gen), dy, torch.randn(N, D, generator=gen), mode, comp, cu)


@pytest.mark.parametrize("mode,comp", MODES)
@pytest.mark.parametrize("dtype,gate_dtype", TYPES)
@pytest.mark.parametrize("D", [66, 129, 1024])
def test_step(mode, comp, dtype, gate_dtype, D):
    B = 6
    x, gate, _, _, _ = inputs(B, D, mode, dtype, gate_dtype, seed=D)
    pool = torch.randn(B, D, generator=torch.Generator().manual_seed(D))
    state = pool.cuda()
    y = kda.kda_scan_step(x[0].cuda(), gate[0].cuda(), state, torch.arange(B, dtype=torch.int32, device="cuda"),
                          gate_mode=mode, complement=comp)
    rows = lambda t: t.view(B, 1, D)  # noqa: E731
    lb.check_scan(dict(y=rows(y), hT=state), rows(x[0]), rows(gate[0]), mode, comp, pool)
