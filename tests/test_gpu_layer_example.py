"""The gated recurrent layer of examples/ against a plain fp64 one."""

import importlib.util
from pathlib import Path

import numpy as np
import pytest
import torch

import kimi_delta_attention_04_gb300 as kda
from oracle import layer_oracle as lo

from kda_cases import np64, rel_f

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    from kimi_delta_attention_04_gb300 import build
    build.build()
    kda.load()
    spec = importlib.util.spec_from_file_location(
        "gated_recurrent_layer", Path(__file__).resolve().parents[1] / "examples" / "gated_recurrent_layer.py")
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_prefill_against_plain_layer(example):
    D, C, T = 200, 96, 150
    layer = example.GatedRecurrentLayer(D, C, seed=3)
    gen = torch.Generator().manual_seed(4)
    x, res = (torch.randn(1, T, D, generator=gen).to(torch.bfloat16) for _ in range(2))
    out, hT = layer.prefill(x.cuda(), res.cuda())
    y, r = lo.add_rmsnorm(np64(x[0]), np64(res[0]), np64(layer.norm), 1e-6)
    w_in = np64(layer.w_in.float()) * np64(layer.w_in_scale)[:, None]
    p = y @ w_in.T + np64(layer.b_in)
    h, last, _ = lo.scan(p[:, :C], p[:, C:], gate_mode="logits", complement=True)
    ref = h @ np64(layer.w_out).T + r
    # the norm's output in e4m3: each value off by up to 2^-4, uniformly, 2^-4 / sqrt(3) in the mean
    # square; as independent errors of a projection's terms they carry over as such, through slopes <= 1;
    # the bf16 roundings (2^-8 and less) are small beside it
    assert rel_f(np64(hT[0]), last) <= 2.0 ** -4
    assert rel_f(np64(out[0]), ref) <= 2.0 ** -4


def test_steps_continue_the_prefill(example):
    """Single tokens run other tile shapes than a prefill: sums in another order,
    rounded to bf16 (2^-8) at each of three stages, states in fp32."""
    off, state_off = example.main()
    assert off <= 3 * 2.0 ** -8 and state_off <= 2 * 2.0 ** -8
