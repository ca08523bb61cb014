"""Softmax attention on values far apart: cached heads of zeros beside others."""

import numpy as np
import pytest
import torch

import kimi_delta_attention_04_gb300 as kda
from oracle import attn_oracle as ao

from attn_cases import BF, E4, F32, Cache, check, randn
from kda_cases import np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kimi_delta_attention_04_gb300 import build
    build.build()
    kda.load()


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


# Rows and tables that take each of the step's layouts: the row's tokens in one CTA or a
# cluster, in many small CTAs, in several clusters whose results a launch joins, and that
# beside a prefix. (rows, tokens of the table's row or 0: as many as there are, prefix or not)
LAYOUTS = {"few": (1, 0, False), "many": (640, 0, False), "clusters": (1, 20000, False), "prefix": (3, 0, True), "prefix_many": (640, 0, True)}


def steps(cache, n, q, scale, layout, prefix=None):
    """The step of rows q [1, HQ, D] on the cache's sequence 0 of n tokens, in a layout: the
    results of its first and last row. With a prefix the first tokens (whole pages of them)
    are the prefix, unless prefix says that it is the cache's sequence 1."""
    rows, room, shared = LAYOUTS[layout]
    P = cache.P
    table, lens, kw = cache.table[0].cpu(), n, {}
    if shared and prefix is None:
        cut = (n // 2) // P
        kw = dict(prefix_table=table[:cut].cuda().contiguous(), prefix_len=cut * P) if cut else {}
        table, lens = table[cut:], n - cut * P
    elif prefix:
        kw = dict(prefix_table=cache.table[1, :-(-prefix // P)].contiguous(), prefix_len=prefix)
    width = max(-(-lens // P), room // P, 1)
    wide = torch.full((rows, width), 2 ** 30, dtype=torch.int32)
    wide[:, :-(-lens // P)] = table[:-(-lens // P)]
    lse = torch.zeros(rows, q.shape[1], device="cuda")
    o = kda.kda_attn_step(q.expand(rows, -1, -1).contiguous().cuda(), cache.k, cache.v, wide.cuda(), i32([lens] * rows), scale=scale,
                          k_scale=cache.k_scale, v_scale=cache.v_scale, lse=lse, **kw)
    assert torch.equal(o[:1].expand_as(o).isnan(), o.isnan()) and torch.equal(torch.nan_to_num(o[:1].expand_as(o)), torch.nan_to_num(o))
    return o[[0, -1]], lse[[0, -1]]


# --- 8-bit caches: heads of zeros have the factor 1, far above that of ordinary heads ---

@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("HQ,HKV,D,P", [(4, 1, 128, 16), (10, 1, 128, 64), (4, 2, 64, 16)])
@pytest.mark.parametrize("n,spread,nats", [
    (32, 1e-6, 0), (1000, 0.1, 10), (2100, 0.02, 12), (2100, 1.0, 12), (700, 0.02, 25), (700, 1e-6, 40), (40, 1e-24, 3), (700, 3e30, 30)])
def test_step_zero_heads_beside_others(layout, HQ, HKV, D, P, n, spread, nats):
    """A head of zeros with a large score takes most of the weight and adds nothing: what the
    others give comes out as exactly as without it."""
    gen = torch.Generator().manual_seed(n + nats)
    scale = 0.125
    q, k, v = randn(gen, 1, HQ, D), randn(gen, n, HKV, D), (randn(gen, n, HKV, D, dtype=F32) * spread).to(BF)
    q[..., 0], k[..., 0] = 8.0, 0.0
    for at in {n // 3, n - 1}:  # (the second one in a place of its own: another warp or part)
        k[at], v[at] = 0.0, 0.0
        k[at, :, 0] = nats
    cache = Cache(gen, [k], [v], P, E4)
    refs = ao.attend(np64(q), *cache.tokens(0), scale, [n])
    cache.cuda()
    o, lse = steps(cache, n, q, scale, layout)
    for r in range(2):
        check(o[r:r + 1], lse[r:r + 1], refs, n, D)
