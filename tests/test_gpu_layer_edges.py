"""The layer operators where their arithmetic or their sizes end: infinite inputs
and states, rows outside the range of a sum of squares, gates far from zero, sizes
next to 2^31. Against the fp64 oracle; E24 is half a step of fp32, relative."""

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
