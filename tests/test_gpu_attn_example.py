"""The softmax attention layer of examples/: the calls in a row, as a server would make them."""

import importlib.util
from pathlib import Path

import numpy as np
import pytest
import torch

import kimi_delta_attention_04_gb300 as kda
from oracle import attn_oracle as ao
from oracle import layer_oracle as lo

from kda_cases import np64, rel_f

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    from kimi_delta_attention_04_gb300 import build
    build.build()
    kda.load()
    spec = importlib.util.spec_from_file_location(
        "attention_layer", Path(__file__).resolve().parents[1] / "examples" / "attention_layer.py")
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_prompts_against_plain_layer(example):
    """One prompt through the layer against the definitions in 64 bits, each on the layer's own weights."""
    D, HQ, HKV, head, T = 192, 4, 2, 64, 50
    layer = example.AttentionLayer(D, HQ, HKV, head, positions=100, seed=3)
    cache = example.PagedCache(8, HKV, 16, head)
    pages = []
    cache.grow(pages, T)
    gen = torch.Generator().manual_seed(4)
    x, res = (torch.randn(T, D, generator=gen).to(torch.bfloat16) for _ in range(2))
    out = layer.prompts(x.cuda(), res.cuda(), cache, example.ints(cache.slots(pages, 0, T)), example.ints(range(7, 7 + T)), example.ints([0, T]))
    n, r = lo.add_rmsnorm(np64(x), np64(res), np64(layer.norm), 1e-6)
    p = (n @ np64(layer.w_qkv).T).reshape(T, HQ + 2 * HKV, head)
    turn = lambda y: ao.rotate(y, np.arange(7, 7 + T), np64(layer.cos_sin))  # noqa: E731
    q, k, v = turn(p[:, :HQ]), turn(p[:, HQ:HQ + HKV]), p[:, HQ + HKV:]
    h, _, _, _ = ao.attend(q, k, v, head ** -0.5, ao.seen_keys(T, T, True))
    ref = h.reshape(T, -1) @ np64(layer.w_out).T + r
    # bf16 roundings one after another: the norm, the projection, the turned heads (scores carry
    # theirs as |q||k| scale 2^-8, here below 2), the weights, the heads, the output
    assert rel_f(np64(out), ref) <= 8 * 2.0 ** -8
    # what the cache holds is what the layer projected
    got = ao.tokens_of(np64(cache.v), pages, T)
    assert rel_f(got, v) <= 3 * 2.0 ** -8


@pytest.mark.parametrize("dtype,steps", [(torch.bfloat16, 1), (torch.float8_e4m3fn, 16)])
def test_shared_beginning_extension_and_steps(example, dtype, steps):
    """The same tokens as one prompt, and in parts: other tiles and orders of sums, rounded to bf16
    (2^-8) at four stages; from an 8-bit cache the heads are off by up to half an e4m3 step, 2^-4."""
    assert example.main(dtype) <= 4 * 2.0 ** -8 * steps
