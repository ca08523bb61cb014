"""Softmax attention on values far apart: cached heads of zeros beside others, scores and
values of infinity, values near the ends of bf16's range; long rows; and every row of
prompts that pairs of CTAs work on."""

import numpy as np
import pytest
import torch

import kimi_delta_attention_04_gb300 as kda
from oracle import attn_oracle as ao

from attn_cases import BF, E4, F32, NAN, Cache, check, randn
from kda_cases import np64

pytestmark = pytest.mark.gpu

INF = float("inf")


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
    (32, 1e-6, 0), (1000, 0.1, 10), (2100, 0.02, 12), (2100, 1.0, 12), (700, 0.02, 25), (700, 1e-6, 40), (40, 1e-24, 3), (700, 3e30, 30), (700, 1e-31, 20), (700, 1e-3, 60), (40, 1e-28, 1)])
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


# --- scores of -inf weigh nothing, wherever a row's tokens are worked on ---

@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("cut", [0, 16, 128, 256, 512, 1024, 1536])
@pytest.mark.parametrize("first", [True, False])
def test_step_scores_of_minus_infinity(layout, cut, first):
    """Keys on one side of `cut` score -inf: as if they were not there; only they: NaN (0 / 0), and
    a logarithm of -inf."""
    gen = torch.Generator().manual_seed(cut)
    n, HQ, HKV, D, P = 1601, 4, 2, 64, 16
    q, k, v = randn(gen, 1, HQ, D), randn(gen, n, HKV, D), randn(gen, n, HKV, D)
    q[..., 0] = 1.0
    hidden = np.arange(n) < cut if first else np.arange(n) >= cut
    k[torch.from_numpy(hidden)] = k[torch.from_numpy(hidden)].index_fill(2, torch.tensor([0]), -INF)
    cache = Cache(gen, [k], [v], P).cuda()
    o, lse = steps(cache, n, q, 0.125, layout)
    if hidden.all():
        assert torch.isnan(o.float()).all() and (lse == -INF).all()
        return
    keep = torch.from_numpy(~hidden)
    refs = ao.attend(np64(q), np64(k[keep]), np64(v[keep]), 0.125, [int(keep.sum())])
    for r in range(2):
        check(o[r:r + 1], lse[r:r + 1], refs, n, D)


@pytest.mark.parametrize("own", ["finite", "-inf", "none"])
@pytest.mark.parametrize("cut", [0, 128, 256, 384])
def test_step_prefix_scores_of_minus_infinity(own, cut):
    """A prefix whose keys from `cut` on score -inf: a split of it may have no others."""
    gen = torch.Generator().manual_seed(cut + 1)
    prefix, HQ, HKV, D, P = 400, 2, 1, 128, 16
    n = 0 if own == "none" else 20
    q = randn(gen, 1, HQ, D)
    q[..., 0] = 1.0
    ks, vs = ([randn(gen, m, HKV, D) for m in (n, prefix)] for _ in range(2))
    ks[1][cut:, :, 0] = -INF
    if own == "-inf":
        ks[0][:, :, 0] = -INF
    cache = Cache(gen, ks, vs, P).cuda()
    keys = np.concatenate([np64(ks[1][:cut]), np64(ks[0][:0 if own == "-inf" else n])])
    values = np.concatenate([np64(vs[1][:cut]), np64(vs[0][:0 if own == "-inf" else n])])
    for layout in ("few", "many"):
        o, lse = steps(cache, n, q, 0.09, layout, prefix=prefix)
        if len(keys) == 0:
            assert torch.isnan(o.float()).all() and (lse == -INF).all()
            continue
        refs = ao.attend(np64(q), keys, values, float(np.float32(0.09)), [len(keys)])
        for r in range(2):
            check(o[r:r + 1], lse[r:r + 1], refs, n + prefix, D)


def test_prompts_scores_of_minus_infinity():
    """Only scores of -inf give NaN and a logarithm of -inf; with others they weigh nothing."""
    gen = torch.Generator().manual_seed(2)
    T, HQ, HKV, D = 200, 2, 1, 64
    q, k, v = randn(gen, 1, T, HQ, D), randn(gen, 1, T, HKV, D), randn(gen, 1, T, HKV, D)
    q[..., 0] = 1.0
    k[:, :140, :, 0] = -INF
    lse = torch.zeros(1, T, HQ, device="cuda")
    o = kda.kda_attn_fwd(q.cuda(), k.cuda(), v.cuda(), scale=0.125, lse=lse)
    assert torch.isnan(o[0, :140].float()).all() and (lse[0, :140] == -INF).all()
    refs = ao.attend(np64(q[0, 140:]), np64(k[0, 140:]), np64(v[0, 140:]), 0.125, ao.seen_keys(60, 60, True))
    check(o[0, 140:], lse[0, 140:], refs, T, D)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("what", [INF, -INF, NAN])
@pytest.mark.parametrize("at", [3, 700, 1600])
def test_step_infinite_values(layout, what, at):
    """An infinity in a value, however small its weight, is that channel's result; the others stay."""
    gen = torch.Generator().manual_seed(at)
    n, HQ, HKV, D, P = 1601, 4, 2, 64, 16
    q, k, v = randn(gen, 1, HQ, D), randn(gen, n, HKV, D), randn(gen, n, HKV, D)
    q[..., 0], k[at, :, 0] = 30.0, -100.0  # a weight of exp(-375) and less
    v[at, 1, 17] = what
    cache = Cache(gen, [k], [v], P).cuda()
    o, lse = steps(cache, n, q, 0.125, layout)
    v[at, 1, 17] = 0.0
    refs = ao.attend(np64(q), np64(k), np64(v), 0.125, [n])
    got = o.float().cpu()
    want = torch.full((2, 2), what)
    assert torch.equal(torch.nan_to_num(got[:, 2:, 17], nan=5.0, posinf=6.0, neginf=7.0), torch.nan_to_num(want, nan=5.0, posinf=6.0, neginf=7.0))
    for r in range(2):
        fixed = got[r:r + 1].clone()
        fixed[:, 2:, 17] = torch.from_numpy(refs[0][:, 2:, 17]).float()
        check(fixed, lse[r:r + 1], refs, n, D)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_step_infinite_scores(layout):
    """A score of +inf gives NaN in its heads and leaves the others as they were."""
    gen = torch.Generator().manual_seed(3)
    n, HQ, HKV, D, P = 1601, 4, 2, 64, 16
    q, k, v = randn(gen, 1, HQ, D), randn(gen, n, HKV, D), randn(gen, n, HKV, D)
    q[..., 0] = 1.0
    k[900, 1, 0] = INF
    cache = Cache(gen, [k], [v], P).cuda()
    o, lse = steps(cache, n, q, 0.125, layout)
    assert torch.isnan(o[:, 2:].float()).all()
    refs = ao.attend(np64(q[:, :2]), np64(k[:, :1]), np64(v[:, :1]), 0.125, [n])
    for r in range(2):
        check(o[r:r + 1, :2], lse[r:r + 1, :2], refs, n, D)


@pytest.mark.parametrize("dtype,infinite", [(BF, False), (BF, True), (E4, False)])  # (8-bit values have no infinity)
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("n", [5, 700, 1601])
def test_step_large_values_without_weight(dtype, layout, n, infinite):
    """Values of 1e38 with weights of exp(-400) add nothing, in other tokens' parts of the row or beside
    them, also where an infinity makes the row one of a kind."""
    gen = torch.Generator().manual_seed(n)
    HQ, HKV, D, P = 4, 2, 64, 16
    q, k, v = randn(gen, 1, HQ, D), randn(gen, n, HKV, D), randn(gen, n, HKV, D)
    q[..., 0], k[..., 0] = 32.0, 0.0
    for at in (0, n // 2, n - 2):
        k[at, :, 0], v[at, :, 20:30] = -100.0, 1e38
    if infinite:
        v[n // 2, :, 3] = INF
    cache = Cache(gen, [k], [v], P, dtype)
    tokens = cache.tokens(0)
    if infinite:
        tokens[1][n // 2, :, 3] = 0.0
    refs = ao.attend(np64(q), *tokens, 0.125, [n])
    o, lse = steps(cache.cuda(), n, q, 0.125, layout)
    got = o.float().cpu()
    if infinite:
        assert (got[..., 3] == INF).all()
        got[..., 3] = torch.from_numpy(refs[0][..., 3]).float()
    for r in range(2):
        check(got[r:r + 1], lse[r:r + 1], refs, n, D)


def test_prompts_large_values_without_weight():
    """The same in rows of a prompt that are computed again."""
    gen = torch.Generator().manual_seed(8)
    T, HQ, HKV, D = 300, 4, 2, 128
    q, k, v = randn(gen, T, HQ, D), randn(gen, T, HKV, D), randn(gen, T, HKV, D)
    q[..., 0], k[..., 0] = 32.0, 0.0
    k[100, :, 0], v[100, :, 20:30] = -100.0, 1e38
    v[7, :, 3], v[100, :, 4] = INF, -INF
    lse = torch.zeros(1, T, HQ, device="cuda")
    o = kda.kda_attn_fwd(q[None].cuda(), k[None].cuda(), v[None].cuda(), scale=0.125, lse=lse)
    got = o[0].float().cpu()
    assert (got[7:, :, 3] == INF).all() and (got[100:, :, 4] == -INF).all()
    v[7, :, 3], v[100, :, 4] = 0.0, 0.0
    refs = ao.attend(np64(q), np64(k), np64(v), 0.125, ao.seen_keys(T, T, True))
    got[7:, :, 3], got[100:, :, 4] = (torch.from_numpy(refs[0][a:, :, c]).float() for a, c in ((7, 3), (100, 4)))
    check(got, lse[0], refs, T, D)


# --- values near the end of the range: their mean is there, their sum is not ---

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_prompts_largest_values(D, causal):
    gen = torch.Generator().manual_seed(D)
    T, HQ, HKV = 300, 4, 2
    q, k, v = randn(gen, 1, T, HQ, D) * 0.1, randn(gen, 1, T, HKV, D), (randn(gen, 1, T, HKV, D, dtype=F32).clamp(-1, 1) * 3.2e38).to(BF)
    v[..., :5] = 3.2e38
    lse = torch.zeros(1, T, HQ, device="cuda")
    o = kda.kda_attn_fwd(q.cuda(), k.cuda(), v.cuda(), scale=0.125, causal=causal, lse=lse)
    refs = ao.attend(np64(q[0]), np64(k[0]), np64(v[0]), 0.125, ao.seen_keys(T, T, causal))
    check(o[0], lse[0], refs, T, D)


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("n,big", [(2, 3.2e38), (4, 1e38), (70, 3.2e38), (3001, 1e38)])
def test_step_largest_values(dtype, layout, n, big):
    gen = torch.Generator().manual_seed(n)
    HQ, HKV, D, P = 4, 2, 128, 16
    q, k, v = randn(gen, 1, HQ, D), randn(gen, n, HKV, D), (randn(gen, n, HKV, D, dtype=F32).clamp(-1, 1) * big).to(BF)
    v[..., :5] = big
    v[..., 5:8] = -big
    cache = Cache(gen, [k], [v], P, dtype)
    refs = ao.attend(np64(q * 0.1), *cache.tokens(0), float(np.float32(0.09)), [n])
    o, lse = steps(cache.cuda(), n, q * 0.1, 0.09, layout)
    for r in range(2):
        check(o[r:r + 1], lse[r:r + 1], refs, n, D)


def test_step_8bit_values_past_the_largest_of_bf16():
    """A head of bf16's largest values is stored as 256 times 2^120, which bf16 does not hold: in the
    prefix, which bf16 copies of are made, as among the row's own tokens."""
    gen = torch.Generator().manual_seed(5)
    n, HQ, HKV, D, P = 48, 2, 1, 64, 16
    q, k, v = randn(gen, 1, HQ, D) * 0.1, randn(gen, n, HKV, D), torch.zeros(n, HKV, D, dtype=BF)
    v[1::3, :, :9] = 3.38e38
    v[2::3, :, 5:12] = -3.38e38
    cache = Cache(gen, [k], [v], P, E4)
    assert float(cache.v_scale[cache.v_scale == cache.v_scale].max()) == 2.0 ** 120
    refs = ao.attend(np64(q), *cache.tokens(0), 0.125, [n])
    cache.cuda()
    for layout in LAYOUTS:
        o, lse = steps(cache, n, q, 0.125, layout)
        for r in range(2):
            check(o[r:r + 1], lse[r:r + 1], refs, n, D)


# --- long rows ---

def repeated(q, k, v, scale, seen):
    """ao.attend of queries q [T, HQ, D] on the keys of one page, k and v [P, D], over and over: of
    `seen` [T] keys in all."""
    P = len(k)
    q, k, v = np64(q), np64(k), np64(v)
    count = np.asarray(seen)[:, None] // P + (np.arange(P)[None] < np.asarray(seen)[:, None] % P)
    s = np.einsum("thd,pd->thp", q, k) * scale + np.log(count)[:, None]
    m = s.max(-1, keepdims=True)
    e = np.exp(s - m)
    p = e / e.sum(-1, keepdims=True)
    return p @ v, (m + np.log(e.sum(-1, keepdims=True)))[..., 0], p @ np.abs(v), (np.abs(q) @ np.abs(k).T).max(-1) * scale


@pytest.mark.parametrize("T,D", [(32, 64), (512, 128)])
def test_prompts_rows_computed_again_for_long(T, D):
    """32 rows of 10^6 keys with an infinity among their values take longer to compute again than a
    wait may last, while the next tile of their CTA (of 512 rows and 128 channels: their pair of CTAs)
    is under way: the call ends with its results. (About 15 s each.)"""
    gen = torch.Generator().manual_seed(7)
    P, N, S = 128, 400 if T == 32 else 200, 2 ** 20 + (2 ** 18 if D == 64 else 0)
    k, v = (randn(gen, 1, 1, P, D).expand(2, -1, -1, -1).contiguous() for _ in range(2))
    v[1, 0, P - 32, 5] = INF  # in the last page of one sequence: of its last 32 queries only
    q = randn(gen, N * T, 1, D)
    table = torch.zeros(N, S // P, dtype=torch.int32, device="cuda")
    table[N - 1, -1] = 1  # (the last sequence starts first)
    err, lse = i32([0]), torch.zeros(1, N * T, 1, device="cuda")
    o = kda.kda_attn_fwd(q[None].cuda(), k.cuda(), v.cuda(), scale=0.09, cu_seqlens=i32([n * T for n in range(N + 1)]), block_table=table,
                         seq_lens_k=i32([S] * N), lse=lse, err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    bad = o[0, -32:, 0, 5].clone()
    assert (bad == INF).all() and torch.isinf(o).sum() == 32
    for a in (0, (N - 2) * T, (N - 1) * T):
        refs = repeated(q[a:a + T], k[0, 0], v[0, 0], float(np.float32(0.09)), S - T + 1 + np.arange(T))
        got = o[0, a:a + T].float().cpu()
        if a == (N - 1) * T:
            got[-32:, 0, 5] = torch.from_numpy(refs[0][-32:, 0, 5]).float()
        check(got, lse[0, a:a + T], refs, S, D)


def test_prompts_long_rows_computed_again():
    """More equal weights than fp32 can count one by one, in a row that is computed again (7 s)."""
    P, S, D = 128, 2 ** 24 + 2 ** 23, 64
    k, v = torch.zeros(3, 1, P, D, dtype=BF), torch.ones(3, 1, P, D, dtype=BF)
    v[1:] = 2.0
    v[2, 0, 0, 5] = INF
    table = torch.zeros(1, S // P, dtype=torch.int32, device="cuda")
    table[:, S // P // 3:] = 1
    table[:, -1] = 2
    lse = torch.zeros(1, 1, 1, device="cuda")
    o = kda.kda_attn_fwd(torch.zeros(1, 1, 1, D, dtype=BF, device="cuda"), k.cuda(), v.cuda(), scale=0.125, block_table=table,
                         seq_lens_k=i32([S]), lse=lse)
    o = o[0, 0, 0].float().cpu()
    assert o[5] == INF
    # a third of the values are 1: half a bf16 step, and 2 (2^10 + S / 2^10) fp32 additions
    bound = (2.0 ** -8 + 2 * (2 ** 10 + S / 2 ** 10) * 2.0 ** -24) * 5 / 3
    assert (o[torch.arange(D) != 5] - 5 / 3).abs().max() <= bound and bound < 0.02
    assert abs(float(lse) - np.log(S)) <= (2 ** 10 + S / 2 ** 10) * 2.0 ** -24 + 2.0 ** -20 * np.log(S)


def weighted(q, k, v, scale, count):
    """ao.attend of queries q [T, HQ, D] on keys k, v [S, HKV, D] of which each is there count [S] times."""
    T, HQ, D = q.shape
    S, G = len(k), HQ // k.shape[1]
    o, a, lse, top = np.zeros((T, HQ, D)), np.zeros((T, HQ, D)), np.zeros((T, HQ)), np.zeros((T, HQ))
    for h in range(HQ):
        kh, vh = np64(k[:, h // G]), np64(v[:, h // G])
        s = np64(q[:, h]) @ kh.T * scale + np.log(count)
        m = s.max(-1, keepdims=True)
        e = np.exp(s - m)
        p = e / e.sum(-1, keepdims=True)
        o[:, h], a[:, h], lse[:, h] = p @ vh, p @ np.abs(vh), (m + np.log(e.sum(-1, keepdims=True)))[:, 0]
        top[:, h] = (np.abs(np64(q[:, h])) @ np.abs(kh).T).max(-1) * scale
    return o, lse, a, top


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("S", [2 ** 15, 2 ** 15 + 128, 2 ** 16 + 1, 2 ** 20, 2 ** 22])
@pytest.mark.parametrize("equal", [True, False])
def test_prompts_long_rows(S, D, equal):
    """Values of one sign in long rows, whose sum the tensor core truncates with every product."""
    gen = torch.Generator().manual_seed(S % 1000 + D)
    P, T, HQ = 128, 45, 3
    q, k, v = randn(gen, T, HQ, D) * (0.0 if equal else 0.5), randn(gen, 1, 1, P, D), randn(gen, 1, 1, P, D).abs() + 0.5
    table = torch.zeros(1, -(-S // P), dtype=torch.int32, device="cuda")
    lse = torch.zeros(1, T, HQ, device="cuda")
    o = kda.kda_attn_fwd(q[None].cuda(), k.cuda(), v.cuda(), scale=0.125, causal=False, block_table=table, seq_lens_k=i32([S]), lse=lse)
    refs = weighted(q, k[0].transpose(0, 1), v[0].transpose(0, 1), 0.125, S // P + (np.arange(P) < S % P) + 0.0)
    # 2^15 keys are 2^11 truncated additions, of up to 2^-23 of the sum, and one of parts in fp32. Equal
    # weights are exact, and so is their sum; others are off as in attn_cases.errors
    sums = (2 ** 11 + S / 2 ** 15) * 2.0 ** -23
    each = 0.0 if equal else 2 * (np.expm1((D / 8 + 6) * 2.0 ** -23 * refs[3]) + 2.0 ** -21 + sums)[..., None] + 2.0 ** -8
    e = refs[2] * (each + sums)
    off = np.abs(np64(o[0]) - refs[0])
    assert (off <= e + 2.0 ** -8 * (np.abs(refs[0]) + e)).all(), f"worst {(off / np.abs(refs[0])).max():.1e}"
    assert np.abs(np64(lse[0]) - refs[1]).max() <= (0.0 if equal else each.max()) + 2.0 ** -20 * (1 + np.abs(refs[1]).max())


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,T", [(64, 200), (128, 40), (128, 512)])
def test_prompts_long_rows_whose_maximum_grows(D, T, causal):
    """Scores that grow after parts of a row's sum were put aside, and earlier keys that still count;
    512 rows of 128 channels, in 200 sequences: pairs of CTAs."""
    gen = torch.Generator().manual_seed(D + T)
    P, N, HQ = 128, 200 if T == 512 else 2, 1
    S = P * 820 + 31
    q, k, v = randn(gen, N * T, HQ, D) * 0.5, randn(gen, 3, 1, P, D), randn(gen, 3, 1, P, D).abs() + 0.5
    q[..., 0] = 8.0
    for page, score in enumerate((-7.0, 0.0, 6.5)):
        k[page, ..., 0] = score / (8.0 * 0.125)
    pages = torch.tensor([0] * 300 + [1] * 500 + [2] * 21, dtype=torch.int32)
    lse = torch.zeros(1, N * T, HQ, device="cuda")
    o = kda.kda_attn_fwd(q[None].cuda(), k.cuda(), v.cuda(), scale=0.125, causal=causal, cu_seqlens=i32([n * T for n in range(N + 1)]),
                         block_table=pages.cuda().repeat(N, 1), seq_lens_k=i32([S] * N), lse=lse)
    for n in (0, N - 1):
        for t in sorted({0, 1, 31, 127, 128, T // 2, T - 1} & set(range(T))):
            r = n * T + t
            seen = S - T + t + 1 if causal else S
            count = np.concatenate([[300.0] * P, [500.0] * P, (seen - 800 * P) // P + (np.arange(P) < (seen - 800 * P) % P)])
            keep = count > 0
            keys, values = (x.reshape(-1, 1, D)[torch.from_numpy(keep)] for x in (k.transpose(1, 2), v.transpose(1, 2)))
            refs = weighted(q[r:r + 1], keys, values, 0.125, count[keep])
            check(o[0, r:r + 1], lse[0, r:r + 1], refs, 2 ** 15, D)


def test_step_long_prefix():
    """Splits of a prefix that are long rows themselves."""
    gen = torch.Generator().manual_seed(9)
    P, B, HQ, HKV, D, prefix = 128, 640, 32, 8, 64, 2 ** 20 + 77
    q, k, v = randn(gen, B, HQ, D) * 0.5, randn(gen, 1, HKV, P, D), randn(gen, 1, HKV, P, D).abs() + 0.5
    lse = torch.zeros(B, HQ, device="cuda")
    o = kda.kda_attn_step(q.cuda(), k.cuda(), v.cuda(), torch.zeros(B, 1, dtype=torch.int32, device="cuda"), i32([0] * B), scale=0.125,
                          prefix_table=torch.zeros(-(-prefix // P), dtype=torch.int32, device="cuda"), prefix_len=prefix, lse=lse)
    rows = [0, 1, 63, 64, 300, 639]
    count = prefix // P + (np.arange(P) < prefix % P) + 0.0
    refs = weighted(q[rows], k[0].transpose(0, 1), v[0].transpose(0, 1), 0.125, count)
    check(o[rows], lse[rows], refs, 2 ** 15, D)


# --- prompts that pairs of CTAs work on: every row ---

def exact(q, k, v, scale, seen):
    """ao.attend on the GPU in 64 bits: q [T, HQ, D], k and v [S, HKV, D], seen [T] keys a query sees."""
    q, k, v = (x.cuda().double() for x in (q, k, v))
    T, HQ, D = q.shape
    S, G = len(k), q.shape[1] // k.shape[1]
    o, a, lse, top = (torch.zeros(T, HQ, *n, dtype=torch.float64, device="cuda") for n in ((D,), (D,), (), ()))
    hidden = torch.arange(S, device="cuda")[None] >= torch.as_tensor(seen, device="cuda")[:, None]
    for h in range(HQ):
        kh, vh = k[:, h // G], v[:, h // G]
        s = (q[:, h] @ kh.T * scale).masked_fill(hidden, -INF)
        lse[:, h] = torch.logsumexp(s, 1)
        p = torch.nan_to_num(torch.softmax(s, 1))
        o[:, h], a[:, h] = p @ vh, p @ vh.abs()
        if S:
            top[:, h] = (q[:, h].abs() @ kh.abs().T * scale).masked_fill(hidden, 0.0).amax(1)
    return tuple(x.cpu().numpy() for x in (o, lse, a, top))


@pytest.mark.parametrize("P", [0, 16, 64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_prompts_every_row_of_many_tiles(P, causal):
    """Outputs and logarithms of all rows: one key of 1400 too many or too few moves a logarithm by 7e-4."""
    gen = torch.Generator().manual_seed(43 + P)
    HQ, HKV, D = 64, 4, 128
    lens, lens_k = (701, 0, 1025, 3), (701, 9, 1400, 130)
    if not P:
        lens_k = (701, 9, 1025, 3)
    T, S = sum(lens), sum(lens_k)
    q, k, v = randn(gen, T, HQ, D), randn(gen, S, HKV, D), randn(gen, S, HKV, D)
    offs, offs_k = np.cumsum([0] + list(lens)), np.cumsum([0] + list(lens_k))
    ks, vs = ([x[a:b] for a, b in zip(offs_k[:-1], offs_k[1:])] for x in (k, v))
    lse = torch.zeros(1, T, HQ, device="cuda")
    kw = dict(scale=0.09, causal=causal, lse=lse, cu_seqlens=i32(offs.tolist()))
    if P:
        cache = Cache(gen, ks, vs, P).cuda()
        o = kda.kda_attn_fwd(q[None].cuda(), cache.k, cache.v, block_table=cache.table, seq_lens_k=cache.lens, **kw)
    else:
        o = kda.kda_attn_fwd(q[None].cuda(), k[None].cuda(), v[None].cuda(), cu_seqlens_k=i32(offs_k.tolist()), **kw)
    for n in range(4):
        a, b = offs[n], offs[n + 1]
        if a == b:
            continue
        refs = exact(q[a:b], ks[n], vs[n], float(np.float32(0.09)), ao.seen_keys(lens[n], lens_k[n], causal))
        check(o[0, a:b], lse[0, a:b], refs, lens_k[n], D)


@pytest.mark.parametrize("what", [INF, -INF, NAN])
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("at,channel", [(300, 17), (300, 100), (460, 17), (460, 100), (2499, 64)])
def test_prompts_hidden_values_of_many_tiles(what, where, at, channel):
    """A bad key or value in each half of a block's keys and of the channels, which two CTAs hold: only
    the queries that see it change, and those to what the definition gives."""
    gen = torch.Generator().manual_seed(at)
    T, HQ, HKV, D = 2500, 64, 4, 128
    q, k, v = randn(gen, T, HQ, D), randn(gen, T, HKV, D), randn(gen, T, HKV, D)
    own = slice(16, 32)  # the heads on key head 1
    clean_lse, lse = torch.zeros(1, T, HQ, device="cuda"), torch.zeros(1, T, HQ, device="cuda")
    clean = kda.kda_attn_fwd(q[None].cuda(), k[None].cuda(), v[None].cuda(), scale=0.09, lse=clean_lse)
    (k if where == "k" else v)[at, 1, channel] = what
    got = kda.kda_attn_fwd(q[None].cuda(), k[None].cuda(), v[None].cuda(), scale=0.09, lse=lse)
    others = [h for h in range(HQ) if not 16 <= h < 32]
    assert torch.equal(got[0][:, others], clean[0][:, others]) and torch.equal(lse[0][:, others], clean_lse[0][:, others])
    bad = (k if where == "k" else v)[:, 1:2].clone()
    (k if where == "k" else v)[at, 1, channel] = 0.0
    seen = ao.seen_keys(T, T, True)
    scale = float(np.float32(0.09))
    refs = exact(q[:, own], k[:, 1:2], v[:, 1:2], scale, seen)
    before, rest = got[0, :at, own], got[0, at:, own].float().cpu()
    # rows that do not see it: as if it were not there
    check(before, lse[0, :at, own], tuple(r[:at] for r in refs), T, D)
    if where == "v":
        want = torch.full((T - at, 16), what)
        assert torch.equal(torch.nan_to_num(rest[..., channel], nan=5.0, posinf=6.0, neginf=7.0), torch.nan_to_num(want, nan=5.0, posinf=6.0, neginf=7.0))
        keep = [d for d in range(D) if d != channel]
        check(rest[..., keep], lse[0, at:, own], tuple(r[at:][..., keep] if r.ndim == 3 else r[at:] for r in refs), T, D)
    elif what != what:
        assert torch.isnan(rest).all()
    else:  # scores of +inf or -inf by the sign of q: NaN, or the key left out
        pos = q[at:, own, channel].float() * what > 0
        assert torch.isnan(rest[pos]).all()
        without = [j for j in range(T) if j != at]
        refs = exact(q[at:, own], k[without, 1:2], v[without, 1:2], scale, seen[at:] - 1)
        fixed, fixed_lse = rest.clone(), lse[0, at:, own].cpu().clone()
        fixed[pos], fixed_lse[pos] = torch.from_numpy(refs[0]).float()[pos], torch.from_numpy(refs[1]).float()[pos]
        check(fixed, fixed_lse, refs, T, D)
    assert torch.isfinite(bad.float()).sum() == bad.numel() - 1
