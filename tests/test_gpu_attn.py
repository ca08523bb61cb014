"""GPU parity of the softmax attention calls (append to the paged cache, whole prompts,
single-token step) against the fp64 oracle through the public calls, within bounds
derived in attn_cases.errors."""

import numpy as np
import pytest
import torch

import kimi_delta_attention_04_gb300 as kda
from kimi_delta_attention_04_gb300 import _lib
from oracle import attn_oracle as ao

from attn_cases import BF, E4, F32, NAN, Cache, check, randn
from kda_cases import Canary, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kimi_delta_attention_04_gb300 import build
    build.build()
    kda.load()


def cu(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)


def err_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# --- append ---

def table_of(positions, rot):
    angle = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
    return torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1)).float()


def check_bf16(got, ref):
    # three fp32 roundings, then half a step of bf16
    assert np.all(np.abs(np64(got) - ref) <= (2.0 ** -8 + 2.0 ** -22) * (np.abs(ref) + 4 * 2.0 ** -24) + 4 * 2.0 ** -24)


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("T,HQ,HKV,D,P,rot,inter", [
    (1, 1, 1, 64, 16, 64, False), (5, 4, 2, 128, 16, 128, False), (37, 14, 2, 64, 32, 32, True), (9, 3, 3, 128, 64, 0, False),
    (33, 32, 8, 128, 128, 64, False), (7, 6, 2, 64, 16, 24, False), (11, 5, 1, 128, 32, 6, True), (3, 96, 16, 128, 16, 128, True),
    (130, 2, 1, 64, 16, 2, False), (4, 7, 7, 128, 16, 128, True), (65, 40, 8, 64, 64, 48, False)])
def test_append(dtype, T, HQ, HKV, D, P, rot, inter):
    gen = torch.Generator().manual_seed(T * 1009 + HQ * 31 + rot)
    packed = randn(gen, T, HQ + 2 * HKV, D)
    pages = -(-(T + 5) // P) + 2
    slots = torch.randperm(pages * P, generator=gen)[:T].int()
    if T > 3:
        slots[1] = -1
        slots[T - 1] = -(2 ** 31)
    positions = torch.randint(0, 500, (T,), generator=gen, dtype=torch.int32)
    if T > 4:
        positions[2], positions[3] = 0, 499
    table = table_of(500, rot) if rot else None
    cn = Canary()
    kc, vc = (cn.clone(randn(gen, pages, HKV, P, D).to(dtype).cuda()) for _ in range(2))
    before = [c.clone() for c in (kc, vc)]
    ks, vs = (cn.clone(torch.full((pages, HKV, P), 3.0).cuda()) if dtype == E4 else None for _ in range(2))
    q_out, k_out = cn.empty((T, HQ, D), BF, name="q_out"), cn.empty((T, HKV, D), BF, name="k_out")
    gpu = packed.cuda()
    err = err_word()
    got = kda.kda_kv_append(gpu[:, HQ:HQ + HKV], gpu[:, HQ + HKV:], slots.cuda(), kc, vc, q=gpu[:, :HQ],
                            positions=positions.cuda() if rot else None, cos_sin=table.cuda() if rot else None, interleaved=inter,
                            q_out=q_out, k_out=k_out, k_scale=ks, v_scale=vs, err=err, check_indices=True)
    assert got[0] is q_out and got[1] is k_out
    cn.check()
    assert int(err) == 0
    x = np64(packed)
    turn = (lambda y: ao.rotate(y, positions.numpy(), np64(table), inter)) if rot else (lambda y: y)
    q, k, v = turn(x[:, :HQ]), turn(x[:, HQ:HQ + HKV]), x[:, HQ + HKV:]
    check_bf16(q_out, q)
    check_bf16(k_out, k)
    for cache, scales, ref, old in ((kc, ks, k, before[0]), (vc, vs, v, before[1])):
        raw = cache.view(torch.uint8) if dtype == E4 else cache
        was = old.view(torch.uint8) if dtype == E4 else old
        touched = torch.zeros(pages, P, dtype=torch.bool)
        for t in range(T):
            s = int(slots[t])
            if s < 0:
                continue
            page, off = s // P, s % P
            touched[page, off] = True
            row = cache[page, :, off].float()
            if dtype == BF:
                check_bf16(row, ref[t])
            else:
                sc = np64(scales[page, :, off])
                # (the fp32 maximum may fall to the other side of 448 times a power of two)
                lo, hi = ao.power_scale(ref[t] * (1 - 2.0 ** -21)), ao.power_scale(ref[t] * (1 + 2.0 ** -21))
                assert np.all((sc >= lo) & (sc <= hi))
                y = ref[t] / sc[:, None]
                slack = 4 * 2.0 ** -24 * (np.max(np.abs(y), -1, keepdims=True) + 1)
                assert np.all(np.abs(np64(row) - y) <= slack + np.maximum(2.0 ** -4 * (np.abs(y) + slack), 2.0 ** -10))
        same = (raw.cpu() == was.cpu()).all(-1).all(1)
        assert (same | touched).all(), "places that no token has were written"
        if dtype == E4:
            assert ((scales.cpu() == 3.0).all(1) | touched).all()


def test_append_in_place_and_without_queries():
    gen = torch.Generator().manual_seed(5)
    T, HQ, HKV, D, P = 19, 8, 2, 128, 16
    packed = randn(gen, T, HQ + 2 * HKV, D)
    positions, table = torch.arange(T, dtype=torch.int32), table_of(T, D)
    slots = torch.arange(T, dtype=torch.int32)
    gpu = packed.cuda()
    q, k, v = gpu[:, :HQ], gpu[:, HQ:HQ + HKV], gpu[:, HQ + HKV:]
    caches = [torch.zeros(2, HKV, P, D, dtype=BF, device="cuda") for _ in range(2)]
    kw = dict(positions=positions.cuda(), cos_sin=table.cuda())
    out = kda.kda_kv_append(k, v, slots.cuda(), *caches, **kw)
    assert out == (None, None) and torch.equal(gpu.cpu(), packed)
    first = [c.clone() for c in caches]
    kda.kda_kv_append(k, v, slots.cuda(), *caches, q=q, q_out=q, k_out=k, **kw)
    assert all(torch.equal(a, b) for a, b in zip(first, caches))
    x = np64(packed)
    check_bf16(gpu[:, :HQ], ao.rotate(x[:, :HQ], positions.numpy(), np64(table)))
    check_bf16(gpu[:, HQ:HQ + HKV], ao.rotate(x[:, HQ:HQ + HKV], positions.numpy(), np64(table)))
    assert torch.equal(gpu[:, HQ + HKV:].cpu(), packed[:, HQ + HKV:])


def test_append_bad_slots_and_positions():
    gen = torch.Generator().manual_seed(6)
    HKV, D, P = 2, 64, 16
    k, v, q = randn(gen, 6, HKV, D).cuda(), randn(gen, 6, HKV, D).cuda(), randn(gen, 6, 4, D).cuda()
    table = table_of(10, D).cuda()
    for slots, positions, code, zero in (
            ([0, 1, 2, 3, 4, 32], [0, 1, 2, 3, 4, 5], 1, []),
            ([0, 1, 2, 3, 4, 2 ** 31 - 1], [0, 1, 2, 3, 4, 5], 1, []),
            ([0, 1, 2, 3, 4, 5], [0, 1, 10, 3, -1, 5], 1, [2, 4]),
            ([0, 1, -1, 3, 4, 5], [0, 1, 2 ** 30, 3, 4, 5], 0, [2])):  # padding may have any position
        cn = Canary()
        kc, vc = (cn.clone(torch.zeros(2, HKV, P, D, dtype=BF, device="cuda")) for _ in range(2))
        q_out = cn.empty((6, 4, D), BF)
        err = err_word()
        kda.kda_kv_append(k, v, torch.tensor(slots, dtype=torch.int32).cuda(), kc, vc, q=q, q_out=q_out,
                          positions=torch.tensor(positions, dtype=torch.int32).cuda(), cos_sin=table, err=err)
        cn.check()
        assert int(err) == code
        good = [t for t in range(6) if 0 <= slots[t] < 2 * P and 0 <= positions[t] < 10]
        assert sorted({int(i) for i in torch.nonzero(vc.float().abs().sum((1, 3)).view(-1))[:, 0]}) == [slots[t] for t in good]
        for t in range(6):
            assert (q_out[t] == 0).all() == (t in zero)
    err = err_word()
    kda.kda_kv_append(k, v, torch.tensor([0, 3, -1, 3, -1, 5], dtype=torch.int32).cuda(), kc, vc, err=err, check_indices=True)
    assert int(err) == 1


def test_append_8bit_extremes():
    """Zeros, the border of 448 times a power of two, tiny and huge heads, infinities and NaN."""
    D, P = 64, 16
    x = torch.zeros(8, 1, D)
    x[1, 0, 3], x[1, 0, 4] = 448.0, -1.0
    x[2, 0, 3] = 450.0                      # bf16's next value above 448
    x[3, 0, :] = 2.0 ** -126
    x[4, 0, 5] = 3.0e38
    x[5, 0, 1], x[5, 0, 2] = float("inf"), 1.0
    x[6, 0, 1], x[6, 0, 2] = NAN, 1.0
    x[7, 0, :] = 2.0 ** -133                # bf16 subnormal
    x = x.to(BF)
    kc, vc = (torch.zeros(1, 1, P, D, device="cuda").to(E4) for _ in range(2))
    ks, vs = (torch.zeros(1, 1, P, device="cuda") for _ in range(2))
    kda.kda_kv_append(x.cuda(), x.cuda(), torch.arange(8, dtype=torch.int32).cuda(), kc, vc, k_scale=ks, v_scale=vs)
    s, y = ks[0, 0, :8].cpu(), kc[0, 0, :8].float().cpu()
    assert s[:5].tolist() == [1.0, 1.0, 2.0, 2.0 ** -110, 2.0 ** 119 if 3.0e38 <= 448 * 2.0 ** 119 else 2.0 ** 120]
    assert torch.isnan(s[5]) and torch.isnan(s[6]) and s[7] == 2.0 ** -110
    assert y[1, 3] == 448 and y[1, 4] == -1 and y[2, 3] == 224 and (y[0] == 0).all()
    assert torch.equal(kc.view(torch.uint8), vc.view(torch.uint8))


# --- whole prompts ---

def run_prompts(gen, lens, lens_k, HQ, HKV, D, causal, P=0, spread=1.0, packed=True, pad=0):
    """Runs the call on packed sequences (or an equal batch), with NaN wherever no sequence
    has a token, and compares with the oracle; returns the output."""
    T, S = sum(lens), sum(lens_k)
    q = randn(gen, T + pad, HQ, D, dtype=F32)
    q = (q * spread).to(BF)
    k, v = randn(gen, S + pad, HKV, D), randn(gen, S + pad, HKV, D)
    q[T:], k[S:], v[S:] = NAN, NAN, NAN
    offs, offs_k = np.cumsum([0] + list(lens)), np.cumsum([0] + list(lens_k))
    ks, vs = ([x[a:b] for a, b in zip(offs_k[:-1], offs_k[1:])] for x in (k, v))
    cn, err = Canary(), err_word()
    B, Tb = (1, T + pad) if packed else (len(lens), lens[0])
    o = cn.empty((B, Tb, HQ, D), BF, name="o")
    lse = cn.empty((B, Tb, HQ), F32, name="lse")
    o.fill_(7.0), lse.fill_(7.0)
    kw = dict(scale=D ** -0.5, causal=causal, o=o, lse=lse, err=err)
    if packed:
        kw["cu_seqlens"] = cu(lens).cuda()
    if P:
        cache = Cache(gen, ks, vs, P).cuda()
        got = kda.kda_attn_fwd(q.view(B, Tb, HQ, D).cuda(), cache.k, cache.v, block_table=cache.table, seq_lens_k=cache.lens, **kw)
    else:
        if packed and list(lens) != list(lens_k):
            kw["cu_seqlens_k"] = cu(lens_k).cuda()
        shape = (1, S + pad, HKV, D) if packed else (len(lens), lens_k[0], HKV, D)
        got = kda.kda_attn_fwd(q.view(B, Tb, HQ, D).cuda(), k.view(shape).cuda(), v.view(shape).cuda(), **kw)
    assert got is o
    cn.check()
    assert int(err) == 0
    flat, flat_lse = o.view(-1, HQ, D), lse.view(-1, HQ)
    for n in range(len(lens)):
        a, b = offs[n], offs[n + 1]
        refs = ao.attend(np64(q[a:b]), np64(ks[n]), np64(vs[n]), D ** -0.5, ao.seen_keys(lens[n], lens_k[n], causal))
        check(flat[a:b], flat_lse[a:b], refs, lens_k[n], D)
    if pad:
        assert (flat[T:] == 7.0).all() and (flat_lse[T:] == 7.0).all(), "rows behind the last sequence were written"
    return o


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("HQ,HKV", [(1, 1), (4, 1), (6, 2), (14, 2), (32, 2)])
@pytest.mark.parametrize("lens", [(1,), (5, 1, 0, 130), (257, 64), (300,)])
def test_prompts_packed(lens, HQ, HKV, D, causal):
    gen = torch.Generator().manual_seed(sum(lens) * 131 + HQ * 7 + D)
    run_prompts(gen, lens, lens, HQ, HKV, D, causal, pad=3)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,lens_k", [((3, 7), (9, 2)), ((130, 1), (5, 400)), ((64, 0, 20), (0, 33, 20)), ((200,), (129,))])
def test_prompts_other_key_lengths(lens, lens_k, causal):
    """More keys than queries (earlier context) and fewer: rows that see nothing give zeros."""
    gen = torch.Generator().manual_seed(sum(lens) + 10 * sum(lens_k))
    run_prompts(gen, lens, lens_k, 4, 2, 64, causal, pad=2)
    run_prompts(gen, lens, lens_k, 3, 3, 128, causal)


@pytest.mark.parametrize("P", [0, 16, 32, 64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_prompts_many_tiles(P, causal):
    """Prompts long enough for the tiles that two CTAs share: first, last and border rows of tiles."""
    gen = torch.Generator().manual_seed(41 + P)
    HQ, HKV, D = 64, 4, 128
    lens, lens_k = (701, 0, 1025, 3), (701, 9, 1400, 130)
    if not P:
        lens_k = (701, 9, 1025, 3)
    T, S = sum(lens), sum(lens_k)
    q, k, v = randn(gen, T, HQ, D), randn(gen, S, HKV, D), randn(gen, S, HKV, D)
    offs, offs_k = np.cumsum([0] + list(lens)), np.cumsum([0] + list(lens_k))
    ks, vs = ([x[a:b] for a, b in zip(offs_k[:-1], offs_k[1:])] for x in (k, v))
    cn, err = Canary(), err_word()
    o, lse = cn.empty((1, T, HQ, D), BF, name="o"), cn.empty((1, T, HQ), F32, name="lse")
    kw = dict(scale=0.09, causal=causal, o=o, lse=lse, err=err, cu_seqlens=cu(lens).cuda())
    if P:
        cache = Cache(gen, ks, vs, P).cuda()
        kda.kda_attn_fwd(q[None].cuda(), cache.k, cache.v, block_table=cache.table, seq_lens_k=cache.lens, **kw)
    else:
        kda.kda_attn_fwd(q[None].cuda(), k[None].cuda(), v[None].cuda(), cu_seqlens_k=cu(lens_k).cuda(), **kw)
    cn.check()
    assert int(err) == 0
    for n in range(4):
        seen = ao.seen_keys(lens[n], lens_k[n], causal)
        for i in sorted({i for i in (0, 1, 7, 8, 15, 16, 31, 32, 33, 63, 64, 127, 128, 500, lens[n] - 2, lens[n] - 1) if 0 <= i < lens[n]}):
            row = offs[n] + i
            refs = ao.attend(np64(q[row:row + 1]), np64(ks[n]), np64(vs[n]), float(np.float32(0.09)), [seen[i]])
            check(o[0, row:row + 1], lse[0, row:row + 1], refs, lens_k[n], D)
    # and every row against the step's kernel, which shares nothing with it but the cache
    if P:
        rows = [(n, i) for n in (0, 2) for i in range(0, lens[n], 5)]
        step = kda.kda_attn_step(q[[offs[n] + i for n, i in rows]].cuda(), cache.k, cache.v, cache.table[[n for n, _ in rows]].contiguous(),
                                 torch.tensor([int(ao.seen_keys(lens[n], lens_k[n], causal)[i]) for n, i in rows], dtype=torch.int32).cuda(), scale=0.09)
        got = o[0, [int(offs[n] + i) for n, i in rows]]
        # both round the weights and the result to bf16
        big = step.float().abs().max()
        assert float((got.float() - step.float()).abs().max()) <= 2 * 2.0 ** -8 * float(big) + 2 * 2.0 ** -8 * float(v.float().abs().max())


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("lens,lens_k", [((5, 1, 130), (5, 200, 259)), ((1, 1), (1, 128)), ((140, 0), (400, 7)), ((9,), (4,))])
def test_prompts_paged(lens, lens_k, P):
    gen = torch.Generator().manual_seed(sum(lens) * 3 + P)
    run_prompts(gen, lens, lens_k, 8, 2, 128, True, P=P, pad=1)
    run_prompts(gen, lens, lens_k, 7, 1, 64, False, P=P)


def test_prompts_equal_batch():
    gen = torch.Generator().manual_seed(9)
    run_prompts(gen, (70, 70, 70), (70, 70, 70), 4, 2, 64, True, packed=False)
    run_prompts(gen, (33, 33), (150, 150), 2, 2, 128, True, packed=False)
    run_prompts(gen, (33, 33), (0, 0), 2, 2, 128, True, packed=False)
    run_prompts(gen, (20, 20), (150, 31), 4, 1, 128, True, packed=False, P=32)


@pytest.mark.parametrize("spread", [0.0, 8.0, 60.0])
def test_prompts_sharp_and_flat(spread):
    """Equal weights, and maxima that climb far along a row."""
    gen = torch.Generator().manual_seed(11)
    run_prompts(gen, (700,), (700,), 2, 1, 128, True, spread=spread)


def test_prompts_of_views():
    """Views of one packed projection, and an output with a stride of its own."""
    gen = torch.Generator().manual_seed(12)
    T, HQ, HKV, D = 150, 4, 2, 128
    packed = randn(gen, 1, T, HQ + 2 * HKV, D)
    gpu = packed.cuda()
    wide = torch.zeros(1, T, HQ + 3, D, dtype=BF, device="cuda")
    kda.kda_attn_fwd(gpu[:, :, :HQ], gpu[:, :, HQ:HQ + HKV], gpu[:, :, HQ + HKV:], scale=0.1, o=wide[:, :, 1:HQ + 1])
    x = np64(packed[0])
    refs = ao.attend(x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], float(np.float32(0.1)), ao.seen_keys(T, T, True))
    check(wide[0, :, 1:HQ + 1], None, refs, T, D)
    assert (wide[:, :, 0] == 0).all() and (wide[:, :, HQ + 1:] == 0).all()


@pytest.mark.parametrize("what", [float("inf"), -float("inf"), NAN])
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("at", [40, 200])
def test_prompts_hidden_values_have_no_effect(what, where, at):
    """An infinity or a NaN in a key or value changes only the queries that see it."""
    gen = torch.Generator().manual_seed(13)
    T, HQ, HKV, D = 300, 4, 2, 128
    q, k, v = randn(gen, 1, T, HQ, D), randn(gen, 1, T, HKV, D), randn(gen, 1, T, HKV, D)
    clean = kda.kda_attn_fwd(q.cuda(), k.cuda(), v.cuda(), scale=0.09)
    (k if where == "k" else v)[0, at, 1, 17] = what
    got = kda.kda_attn_fwd(q.cuda(), k.cuda(), v.cuda(), scale=0.09)
    x = [np64(t[0]) for t in (q, k, v)]
    refs = ao.attend(x[0][:at], x[1][:at], x[2][:at], float(np.float32(0.09)), ao.seen_keys(at, at, True))
    check(got[0, :at], None, refs, T, D)
    assert torch.equal(got[0, :, :2], clean[0, :, :2]), "another head changed"
    seen = got[0, at:, 2:].float().cpu()
    if where == "v":  # the one channel is what the definition gives; the others stay
        want = torch.full_like(seen[:, :, 17], what)
        assert torch.equal(torch.nan_to_num(seen[:, :, 17], nan=5.0, posinf=6.0, neginf=7.0), torch.nan_to_num(want, nan=5.0, posinf=6.0, neginf=7.0))
        keep = [d for d in range(D) if d != 17]
        x[2][at, 1, 17] = 0
        refs = ao.attend(x[0], x[1], x[2], float(np.float32(0.09)), ao.seen_keys(T, T, True))
        check(got[0, :, 2:][:, :, keep], None, tuple(r[:, 2:, ...] if r.ndim == 2 else r[:, 2:][:, :, keep] for r in refs), T, D)
    elif what != what:
        assert torch.isnan(seen).all()
    else:  # scores of +inf or -inf by the sign of q: NaN, or the key left out
        pos = (q[0, at:, 2:, 17].float() * what > 0)
        assert torch.isnan(seen[pos]).all()
        x[1][at, 1, 17] = 0
        for i in range(at, T):
            for h in (2, 3):
                if not pos[i - at, h - 2]:
                    keys = [j for j in range(i + 1) if j != at]
                    r = ao.attend(x[0][i:i + 1, h:h + 1], x[1][keys, 1:2], x[2][keys, 1:2], float(np.float32(0.09)), [len(keys)])
                    check(got[0, i:i + 1, h:h + 1], None, r, T, D)


def test_prompts_with_unwritten_padding():
    """A right-padded equal batch whose padding holds NaN: the rows before it are as without it."""
    gen = torch.Generator().manual_seed(16)
    B, T, HQ, HKV, D, real = 3, 400, 4, 2, 128, (400, 250, 1)
    q, k, v = randn(gen, B, T, HQ, D), randn(gen, B, T, HKV, D), randn(gen, B, T, HKV, D)
    for b, n in enumerate(real):
        for x in (q, k, v):
            x[b, n:] = NAN
    lse = torch.empty(B, T, HQ, device="cuda")
    o = kda.kda_attn_fwd(q.cuda(), k.cuda(), v.cuda(), scale=0.09, lse=lse)
    for b, n in enumerate(real):
        refs = ao.attend(np64(q[b, :n]), np64(k[b, :n]), np64(v[b, :n]), float(np.float32(0.09)), ao.seen_keys(n, n, True))
        check(o[b, :n], lse[b, :n], refs, n, D)
        assert torch.isnan(o[b, n:].float()).all() and torch.isnan(lse[b, n:]).all()


def test_prompts_refuse_bad_lengths():
    T, HQ, HKV, D = 20, 2, 1, 64
    gen = torch.Generator().manual_seed(14)
    q, k, v = (randn(gen, 1, T, n, D).cuda() for n in (HQ, HKV, HKV))
    for bad in ([1, 5, 20], [0, 7, 5], [0, 5, 21], [0, -1, 20]):
        err = err_word()
        o = torch.full((1, T, HQ, D), 3.0, dtype=BF, device="cuda")
        kda.kda_attn_fwd(q, k, v, scale=1.0, cu_seqlens=torch.tensor(bad, dtype=torch.int32).cuda(), o=o, err=err)
        assert int(err) == 1 and (o == 3.0).all()
    err = err_word()
    kda.kda_attn_fwd(q, k, v, scale=1.0, cu_seqlens=cu([20]).cuda(), cu_seqlens_k=torch.tensor([0, 21], dtype=torch.int32).cuda(), o=o, err=err)
    assert int(err) == 1 and (o == 3.0).all()
    cache = torch.zeros(4, HKV, 16, D, dtype=BF, device="cuda")
    for n in (33, -1):
        err = err_word()
        kda.kda_attn_fwd(q, cache, cache, scale=1.0, block_table=torch.zeros(1, 2, dtype=torch.int32, device="cuda"),
                         seq_lens_k=torch.tensor([n], dtype=torch.int32).cuda(), o=o, err=err)
        assert int(err) == 1 and (o == 3.0).all()


def test_prompts_leave_out_bad_pages():
    gen = torch.Generator().manual_seed(15)
    T, S, HQ, HKV, D, P = 100, 170, 4, 2, 64, 32
    q, k, v = randn(gen, 1, T, HQ, D), randn(gen, S, HKV, D), randn(gen, S, HKV, D)
    cache = Cache(gen, [k], [v], P)
    cache.table[0, 2] = len(cache.k)
    cache.table[0, 0] = -5
    cache.cuda()
    err = err_word()
    o = kda.kda_attn_fwd(q.cuda(), cache.k, cache.v, scale=0.125, block_table=cache.table, seq_lens_k=cache.lens, err=err)
    assert int(err) == 1
    for i in (0, 1, 40, 99):
        keys = [j for j in range(i + S - T + 1) if j // P not in (0, 2)]
        refs = ao.attend(np64(q[0, i:i + 1]), np64(k[keys]), np64(v[keys]), 0.125, [len(keys)])
        check(o[0, i:i + 1], None, refs, S, D)
    cache.table.fill_(-1)
    lse = torch.zeros(1, T, HQ, device="cuda")
    o = kda.kda_attn_fwd(q.cuda(), cache.k, cache.v, scale=0.125, block_table=cache.table, seq_lens_k=cache.lens, err=err, lse=lse)
    assert (o == 0).all() and torch.isinf(lse).all()


@pytest.mark.parametrize("P", [16, 64, 128])
def test_prompts_leave_out_bad_pages_of_many_tiles(P):
    """Where two CTAs hold half of a block's keys each: pages of one half, of the other, of
    both, and of the last blocks, which are not full."""
    gen = torch.Generator().manual_seed(16)
    T, HQ, HKV, D = 2500, 64, 4, 128
    q, k, v = randn(gen, 1, T, HQ, D), randn(gen, T, HKV, D), randn(gen, T, HKV, D)
    cache = Cache(gen, [k], [v], P)
    gone = [t // P for t in (0, 200, 330, 640, 767, 1500, 2499)]
    cache.table[0, gone] = torch.tensor([-1, len(cache.k), 2 ** 31 - 1, -2 ** 31, len(cache.k), -7, -1], dtype=torch.int32)
    cache.cuda()
    err = err_word()
    o = kda.kda_attn_fwd(q.cuda(), cache.k, cache.v, scale=0.09, block_table=cache.table, seq_lens_k=cache.lens, err=err)
    assert int(err) == 1
    for i in (0, 17, 129, 255, 256, 400, 700, 801, 1024, 1600, 2047, 2490, 2499):
        keys = [j for j in range(i + 1) if j // P not in gone]
        if not keys:
            assert (o[0, i] == 0).all()
            continue
        refs = ao.attend(np64(q[0, i:i + 1]), np64(k[keys]), np64(v[keys]), float(np.float32(0.09)), [len(keys)])
        check(o[0, i:i + 1], None, refs, T, D)


# --- the single-token step ---

def run_step(gen, lens, HQ, HKV, D, P, dtype, prefix=0, spread=1.0, width=None):
    B = len(lens)
    q = (randn(gen, B, HQ, D, dtype=F32) * spread).to(BF)
    seqs = [max(0, n) for n in lens] + [prefix]
    ks, vs = ([randn(gen, n, HKV, D) for n in seqs] for _ in range(2))
    cache = Cache(gen, ks, vs, P, dtype)
    tokens = [cache.tokens(n) for n in range(B + 1)]
    table = cache.table[:B]
    need = max(1, max(-(-max(0, n) // P) for n in lens))
    table = torch.cat([table, torch.full((B, 50), 2 ** 30, dtype=torch.int32)], 1)[:, :need if width is None else width].contiguous()
    prefix_table = cache.table[B, :-(-prefix // P)].contiguous() if prefix else None
    cache.cuda()
    cn, err = Canary(), err_word()
    o, lse = cn.empty((B, HQ, D), BF, name="o"), cn.empty((B, HQ), F32, name="lse")
    got = kda.kda_attn_step(q.cuda(), cache.k, cache.v, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), scale=D ** -0.5,
                            k_scale=cache.k_scale, v_scale=cache.v_scale, prefix_table=None if prefix_table is None else prefix_table.cuda(),
                            prefix_len=prefix, o=o, lse=lse, err=err)
    assert got is o
    cn.check()
    assert int(err) == 0
    for b in range(B):
        k, v = (np.concatenate([tokens[B][i], tokens[b][i]]) for i in range(2))
        seen = 0 if lens[b] < 0 else len(k)
        check(o[b:b + 1], lse[b:b + 1], ao.attend(np64(q[b:b + 1]), k, v, D ** -0.5, [seen]), len(k), D)
    return o


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("HQ,HKV,D", [(1, 1, 64), (4, 2, 128), (7, 1, 64), (16, 1, 128), (40, 2, 64), (33, 1, 128), (8, 8, 128)])
@pytest.mark.parametrize("P", [16, 64])
def test_step(dtype, HQ, HKV, D, P):
    gen = torch.Generator().manual_seed(HQ * 17 + D + P)
    run_step(gen, [1, 0, 5, 16, 17, -1, 64, 65, 200], HQ, HKV, D, P, dtype)


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("P,lens", [(16, [3000]), (32, [2049, 1]), (128, [2500, 4000, 130]), (64, [9000])])
def test_step_split(dtype, P, lens):
    """Long rows, whose tokens several CTAs share; table wider than any row."""
    gen = torch.Generator().manual_seed(sum(lens))
    run_step(gen, lens, 4, 1, 128, P, dtype, spread=3.0)
    run_step(gen, lens, 6, 2, 64, P, dtype, width=-(-max(lens) // P) + 40)


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("prefix", [0, 200])
def test_step_few_rows_on_long_tables(dtype, prefix):
    """Rows that several clusters work on; padding and empty rows among them."""
    gen = torch.Generator().manual_seed(31 + prefix)
    run_step(gen, [17000, 3], 3, 1, 64, 64, dtype, prefix=prefix, spread=2.0)
    run_step(gen, [5, -1, 0], 2, 2, 128, 16, dtype, prefix=prefix, width=1200)


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("prefix,HQ,HKV,D,P", [(1, 2, 1, 64, 16), (15, 8, 2, 128, 16), (128, 4, 4, 64, 32), (300, 14, 2, 128, 64), (1000, 32, 2, 128, 128)])
def test_step_prefix(dtype, prefix, HQ, HKV, D, P):
    gen = torch.Generator().manual_seed(prefix + HQ)
    run_step(gen, [1, 0, 70, -1, 33], HQ, HKV, D, P, dtype, prefix=prefix, spread=2.0)


def test_step_prefix_many_rows():
    gen = torch.Generator().manual_seed(21)
    run_step(gen, [int(n) for n in torch.randint(0, 40, (150,), generator=gen)], 4, 2, 64, 16, BF, prefix=333)


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("prefix", [0, 40])
@pytest.mark.parametrize("HQ,HKV,D,P", [(8, 4, 128, 16), (40, 4, 64, 32)])
def test_step_many_rows(dtype, prefix, HQ, HKV, D, P):
    """More CTAs than three rounds of the SMs take: smaller ones, and results that a launch joins."""
    gen = torch.Generator().manual_seed(HQ + prefix)
    lens = [int(x) for x in torch.randint(1, 70, (156,), generator=gen)]
    run_step(gen, lens + [0, -3, 1, 300], HQ, HKV, D, P, dtype, prefix=prefix)


def test_step_equals_the_last_prompt_row():
    """The last query of a causal prompt and the step on the same cache: the same keys."""
    gen = torch.Generator().manual_seed(22)
    S, HQ, HKV, D, P = 777, 8, 2, 128, 32
    q, k, v = randn(gen, 1, S, HQ, D), randn(gen, S, HKV, D), randn(gen, S, HKV, D)
    cache = Cache(gen, [k], [v], P).cuda()
    whole = kda.kda_attn_fwd(q.cuda(), cache.k, cache.v, scale=0.09, block_table=cache.table, seq_lens_k=cache.lens)
    step = kda.kda_attn_step(q[0, -1:].cuda(), cache.k, cache.v, cache.table, cache.lens, scale=0.09)
    refs = ao.attend(np64(q[0, -1:]), np64(k), np64(v), float(np.float32(0.09)), [S])
    check(whole[0, -1:], None, refs, S, D)
    check(step, None, refs, S, D)


def test_step_bad_pages_and_lengths():
    gen = torch.Generator().manual_seed(23)
    HQ, HKV, D, P, S = 4, 2, 64, 16, 100
    q = randn(gen, 3, HQ, D)
    ks, vs = ([randn(gen, S, HKV, D) for _ in range(3)] for _ in range(2))
    cache = Cache(gen, ks, vs, P)
    table = cache.table.clone()
    table[1, 3] = -1
    table[2].fill_(2 ** 31 - 1)
    cache.cuda()
    err, lse = err_word(), torch.zeros(3, HQ, device="cuda")
    o = kda.kda_attn_step(q.cuda(), cache.k, cache.v, table.cuda(), cache.lens, scale=0.125, err=err, lse=lse)
    assert int(err) == 1
    for b, keys in ((0, range(S)), (1, [j for j in range(S) if j // P != 3])):
        keys = list(keys)
        check(o[b:b + 1], lse[b:b + 1], ao.attend(np64(q[b:b + 1]), np64(ks[b][keys]), np64(vs[b][keys]), 0.125, [len(keys)]), S, D)
    assert (o[2] == 0).all() and torch.isinf(lse[2]).all()
    err = err_word()
    o = kda.kda_attn_step(q.cuda(), cache.k, cache.v, cache.table, torch.tensor([S, 7 * P + 1, 2 ** 31 - 1], dtype=torch.int32).cuda(), scale=0.125, err=err)
    assert int(err) == 1 and (o[1:] == 0).all() and not (o[0] == 0).any()
    # a prefix page out of range
    err = err_word()
    prefix = cache.table[0].clone()
    prefix[1] = len(cache.k)
    o = kda.kda_attn_step(q.cuda(), cache.k, cache.v, cache.table, torch.tensor([0, 5, -1], dtype=torch.int32).cuda(), scale=0.125, err=err,
                          prefix_table=prefix, prefix_len=S)
    assert int(err) == 1
    keys = [j for j in range(S) if j // P != 1]
    check(o[:1], None, ao.attend(np64(q[:1]), np64(ks[0][keys]), np64(vs[0][keys]), 0.125, [len(keys)]), S, D)
    assert (o[2] == 0).all()


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("prefix", [0, 64])
def test_step_infinities(dtype, prefix):
    gen = torch.Generator().manual_seed(24)
    HQ, HKV, D, P, S = 2, 1, 128, 16, 90
    q, k, v = randn(gen, 1, HQ, D), randn(gen, S, HKV, D), randn(gen, S, HKV, D)
    for where in ("k", "v"):
        c = Cache(gen, [k[prefix:], k[:max(1, prefix)]], [v[prefix:], v[:max(1, prefix)]], P, dtype)
        page = int(c.table[1 if prefix else 0, 1])
        if dtype == E4:  # (an 8-bit head with an infinity or a NaN has a NaN as its scale)
            getattr(c, where + "_scale")[page, 0, 3] = NAN
        else:
            getattr(c, where)[page, 0, 3, 9] = NAN
        pt = c.table[1, :prefix // P].contiguous().cuda() if prefix else None
        own = c.table[:1].contiguous().cuda()
        c.cuda()
        o = kda.kda_attn_step(q.cuda(), c.k, c.v, own, c.lens[:1].contiguous(), scale=0.09, k_scale=c.k_scale, v_scale=c.v_scale,
                              prefix_table=pt, prefix_len=prefix)
        nan = torch.isnan(o[0].float()).cpu()
        if where == "k" or dtype == E4:
            assert nan.all()
        else:
            assert nan[:, 9].all() and nan.sum() == HQ


# --- streams, graphs ---

def test_other_streams_and_graphs():
    """The three calls on a stream of their own, and captured: a decode step replayed on new inputs."""
    gen = torch.Generator().manual_seed(25)
    B, HQ, HKV, D, P, prefix = 5, 8, 2, 128, 16, 100
    lens = [30, 1, 64, 0, 17]
    seqs = lens + [prefix]
    ks, vs = ([randn(gen, n, HKV, D) for n in seqs] for _ in range(2))
    cache = Cache(gen, [torch.cat([x, x[:0]]) for x in ks], vs, P, spare=8).cuda()
    table = torch.full((B, 6), -1, dtype=torch.int32, device="cuda")
    table[:, :cache.table.shape[1]] = cache.table[:B, :6]
    used = {int(p) for b in range(B) for p in cache.table[b, :-(-lens[b] // P)]} | {int(p) for p in cache.table[B, :-(-prefix // P)]}
    free = [p for p in range(len(cache.k)) if p not in used]
    for b in range(B):
        if lens[b] % P == 0:
            table[b, lens[b] // P] = free.pop()
    slots = torch.tensor([int(table[b, n // P]) * P + n % P for b, n in enumerate(lens)], dtype=torch.int32, device="cuda")
    prefix_table = cache.table[B, :-(-prefix // P)].contiguous()
    packed = torch.zeros(B, HQ + 2 * HKV, D, dtype=BF, device="cuda")
    positions = torch.tensor([prefix + n for n in lens], dtype=torch.int32, device="cuda")
    cos_sin = table_of(400, D).cuda()
    seq_lens = torch.tensor([n + 1 for n in lens], dtype=torch.int32, device="cuda")
    q_out, o = torch.empty(B, HQ, D, dtype=BF, device="cuda"), torch.empty(B, HQ, D, dtype=BF, device="cuda")

    def step(stream=None):
        kda.kda_kv_append(packed[:, HQ:HQ + HKV], packed[:, HQ + HKV:], slots, cache.k, cache.v, q=packed[:, :HQ], positions=positions,
                          cos_sin=cos_sin, q_out=q_out, stream=stream)
        return kda.kda_attn_step(q_out, cache.k, cache.v, table, seq_lens, scale=0.09, prefix_table=prefix_table, prefix_len=prefix, o=o,
                                 stream=stream)

    def expect(x):
        t = np64(cos_sin)
        q = ao.rotate(np64(x[:, :HQ]), positions.cpu().numpy(), t)
        k = ao.rotate(np64(x[:, HQ:HQ + HKV]), positions.cpu().numpy(), t)
        rnd = lambda y: np64(torch.from_numpy(y).to(BF))  # noqa: E731
        return [ao.attend(rnd(q)[b:b + 1], np.concatenate([np64(ks[B]), np64(ks[b]), rnd(k)[b:b + 1]]),
                          np.concatenate([np64(vs[B]), np64(vs[b]), np64(x[b:b + 1, HQ + HKV:])]), 0.09, [prefix + lens[b] + 1]) for b in range(B)]

    def compare(x):
        # (the oracle rounds the turned heads from fp64, the call from fp32: a bf16 step apart at ties)
        for b, refs in enumerate(expect(x)):
            oo, lse, a, top = refs
            check(o[b:b + 1], None, (oo, lse, a * (1 + 2.0 ** -6) + 2.0 ** -7 * np.abs(a), top), 300, D)

    side = torch.cuda.Stream()
    x = randn(gen, B, HQ + 2 * HKV, D)
    packed.copy_(x)
    torch.cuda.synchronize()
    step(side)
    side.synchronize()
    compare(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        x = randn(gen, B, HQ + 2 * HKV, D)
        packed.copy_(x)
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        compare(x)
    # the same call twice gives the same bits
    again = step().clone()
    assert torch.equal(again, step())


def test_calls_with_nothing_to_do():
    z = lambda *s: torch.zeros(*s, dtype=BF, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    assert kda.kda_attn_fwd(z(1, 0, 4, 64), z(1, 0, 2, 64), z(1, 0, 2, 64), scale=1.0).shape == (1, 0, 4, 64)
    assert kda.kda_attn_step(z(0, 4, 64), z(3, 2, 16, 64), z(3, 2, 16, 64), i(0, 2), i(0), scale=1.0).shape == (0, 4, 64)
    assert kda.kda_kv_append(z(0, 2, 64), z(0, 2, 64), i(0), z(3, 2, 16, 64), z(3, 2, 16, 64)) == (None, None)
    # an empty cache and a table without pages
    o = kda.kda_attn_step(z(2, 4, 64) + 1, z(0, 2, 16, 64), z(0, 2, 16, 64), i(2, 0), i(2), scale=1.0)
    assert (o == 0).all()
    o = kda.kda_attn_fwd(z(1, 3, 4, 64) + 1, z(1, 0, 2, 64), z(1, 0, 2, 64), scale=1.0)
    assert (o == 0).all()
    assert _lib.KDA_ATTN_MAX_HEADS == 1024
