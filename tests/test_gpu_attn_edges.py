"""Softmax attention where it meets its surroundings: caches and strides past 32 bits, calls
on several streams at once, captured calls, repeated calls, largest and oddest groups."""

import numpy as np
import pytest
import torch

import kimi_delta_attention_04_gb300 as kda
from oracle import attn_oracle as ao

from attn_cases import BF, E4, F32, Cache, check, quantised, randn
from kda_cases import np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from kimi_delta_attention_04_gb300 import build
    build.build()
    kda.load()


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", [BF, E4])
def test_caches_past_32_bits(dtype):
    """The last pages of a cache of more than 2^32 bytes (bf16: more than 2^32 elements)."""
    gen = torch.Generator().manual_seed(1)
    HQ, HKV, D, P, S = 8, 4, 128, 128, 200
    pages = 2 ** 32 // (HKV * P * D) + 5
    big = [torch.zeros(pages, HKV, P, D, dtype=torch.uint8, device="cuda").view(E4) if dtype == E4
           else torch.zeros(pages, HKV, P, D, dtype=dtype, device="cuda") for _ in range(2)]
    assert big[0].numel() > 2 ** 32
    scales = [torch.ones(pages, HKV, P, device="cuda") if dtype == E4 else None for _ in range(2)]
    q, k, v = randn(gen, S, HQ, D), randn(gen, S, HKV, D), randn(gen, S, HKV, D)
    own = [pages - 1, pages - 3]
    slots = i32([own[t // P] * P + t % P for t in range(S)])
    kda.kda_kv_append(k.cuda(), v.cuda(), slots, *big, k_scale=scales[0], v_scale=scales[1])
    held = []
    for x, cache, scale in zip((k, v), big, scales):
        got = torch.stack([cache.view(torch.uint8)[own[t // P], :, t % P].view(E4) if dtype == E4 else cache[own[t // P], :, t % P] for t in range(S)])
        if dtype == E4:
            want, s = quantised(x)
            assert torch.equal(got.view(torch.uint8).cpu(), want.view(torch.uint8))
            held.append(np64(want.float()) * np64(s)[..., None])
        else:
            assert torch.equal(got.cpu(), x)
            held.append(np64(x))
        # nothing where a 32-bit offset would have put them
        assert not bool(cache.view(torch.uint8)[:pages - 3].any())
    table, lens = i32([own]), i32([S])
    o = kda.kda_attn_step(q[-1:].cuda(), *big, table, lens, scale=0.09, k_scale=scales[0], v_scale=scales[1])
    check(o, None, ao.attend(np64(q[-1:]), *held, float(np.float32(0.09)), [S]), S, D)
    o = kda.kda_attn_step(q[-1:].cuda(), *big, i32([[0]]), i32([0]), scale=0.09, k_scale=scales[0], v_scale=scales[1], prefix_table=table[0],
                          prefix_len=S)
    check(o, None, ao.attend(np64(q[-1:]), *held, float(np.float32(0.09)), [S]), S, D)
    if dtype == BF:
        o = kda.kda_attn_fwd(q[None].cuda(), *big, scale=0.09, block_table=table, seq_lens_k=lens)
        check(o[0], None, ao.attend(np64(q), *held, float(np.float32(0.09)), ao.seen_keys(S, S, True)), S, D)


def test_row_strides_past_32_bits():
    """Rows so far apart that the last ones start past 2^32 elements."""
    gen = torch.Generator().manual_seed(2)
    T, HQ, HKV, D = 270, 4, 2, 64
    step = 2 ** 24
    wide = torch.empty(T * step, dtype=BF, device="cuda")
    view = wide.view(T, step)[:, :(2 * HQ + 2 * HKV) * D].view(T, -1, D)
    x = randn(gen, T, 2 * HQ + 2 * HKV, D)
    x[:, HQ + 2 * HKV:] = 0
    view.copy_(x)
    q, k, v, o = (view[None, :, a:b] for a, b in ((0, HQ), (HQ, HQ + HKV), (HQ + HKV, HQ + 2 * HKV), (HQ + 2 * HKV, 2 * HQ + 2 * HKV)))
    assert kda.kda_attn_fwd(q, k, v, scale=0.125, o=o) is o
    same = kda.kda_attn_fwd(*(t.contiguous() for t in (q, k, v)), scale=0.125)
    assert torch.equal(o, same)
    refs = ao.attend(*(np64(t[0]) for t in (x[None, :, :HQ], x[None, :, HQ:HQ + HKV], x[None, :, HQ + HKV:HQ + 2 * HKV])), 0.125, ao.seen_keys(T, T, True))
    check(o[0], None, refs, T, D)
    caches = [torch.zeros(20, HKV, 16, D, dtype=BF, device="cuda") for _ in range(2)]
    kda.kda_kv_append(k[0], v[0], i32(range(T)), *caches, q=q[0], q_out=o[0])
    assert torch.equal(o[0], q[0])
    assert torch.equal(caches[0].transpose(1, 2).reshape(-1, HKV, D)[:T], k[0])
    lens = [T - 1] * T
    whole = kda.kda_attn_step(q[0], *caches, i32([list(range(17))] * T), i32(lens), scale=0.125, o=o[0])
    same = kda.kda_attn_step(q[0].contiguous(), *caches, i32([list(range(17))] * T), i32(lens), scale=0.125)
    assert torch.equal(whole, same)


def test_unwritten_rows_between():
    """What lies between strided rows is left as it was, and 16-byte rows off the 32-byte grid work."""
    gen = torch.Generator().manual_seed(3)
    T, HQ, HKV, D = 140, 3, 1, 64
    buf = torch.full((T, HQ * D + 8), 5.0, dtype=BF, device="cuda")
    o = buf[:, 8:].view(1, T, HQ, D)
    q, k, v = randn(gen, 1, T, HQ, D), randn(gen, 1, T, HKV, D), randn(gen, 1, T, HKV, D)
    kda.kda_attn_fwd(q.cuda(), k.cuda(), v.cuda(), scale=0.125, o=o)
    assert (buf[:, :8] == 5.0).all()
    check(o[0], None, ao.attend(*(np64(x[0]) for x in (q, k, v)), 0.125, ao.seen_keys(T, T, True)), T, D)


@pytest.mark.parametrize("HQ,HKV", [(128, 1), (130, 1), (65, 1), (26, 2), (9, 1), (17, 1), (11, 1)])
def test_groups(HQ, HKV):
    """Groups that divide a tile's rows evenly, nearly and badly, and more than a tile holds."""
    gen = torch.Generator().manual_seed(HQ)
    T, D, P = 37, 64, 16
    q, k, v = randn(gen, 1, T, HQ, D), randn(gen, T, HKV, D), randn(gen, T, HKV, D)
    cache = Cache(gen, [k], [v], P).cuda()
    refs = ao.attend(np64(q[0]), np64(k), np64(v), 0.125, ao.seen_keys(T, T, True))
    check(kda.kda_attn_fwd(q.cuda(), k[None].cuda(), v[None].cuda(), scale=0.125)[0], None, refs, T, D)
    check(kda.kda_attn_fwd(q.cuda(), cache.k, cache.v, scale=0.125, block_table=cache.table, seq_lens_k=cache.lens)[0], None, refs, T, D)
    last = tuple(r[-1:] for r in refs)
    check(kda.kda_attn_step(q[0, -1:].cuda(), cache.k, cache.v, cache.table, cache.lens, scale=0.125), None, last, T, D)
    o = kda.kda_attn_step(q[0, -1:].cuda(), cache.k, cache.v, i32([[0]]), i32([0]), scale=0.125, prefix_table=cache.table[0].contiguous(), prefix_len=T)
    check(o, None, last, T, D)


def test_many_sequences():
    """More sequences than a warp or a CTA has threads, most of them empty or of one token."""
    gen = torch.Generator().manual_seed(5)
    lens = [int(n) for n in torch.randint(0, 3, (2000,), generator=gen)]
    lens[777], lens[1999] = 150, 0
    T, HQ, HKV, D = sum(lens), 2, 1, 64
    q, k, v = randn(gen, T, HQ, D), randn(gen, T, HKV, D), randn(gen, T, HKV, D)
    offs = np.cumsum([0] + lens)
    o = kda.kda_attn_fwd(q[None].cuda(), k[None].cuda(), v[None].cuda(), scale=0.125, cu_seqlens=i32(offs.tolist()))[0]
    refs = [ao.attend(np64(q[a:b]), np64(k[a:b]), np64(v[a:b]), 0.125, ao.seen_keys(b - a, b - a, True)) for a, b in zip(offs[:-1], offs[1:]) if b > a]
    check(o, None, tuple(np.concatenate([r[i] for r in refs]) for i in range(4)), 150, D)


def test_calls_at_once():
    """Prompts, projections and steps on streams of their own at the same time give what they give alone."""
    gen = torch.Generator().manual_seed(6)
    T, HQ, HKV, D, P = 2000, 16, 4, 128, 64
    q, k, v = randn(gen, 1, T, HQ, D).cuda(), randn(gen, 1, T, HKV, D).cuda(), randn(gen, 1, T, HKV, D).cuda()
    x, w = randn(gen, 3000, 1024).cuda(), randn(gen, 2048, 1024).cuda()
    pages = T // P + 1
    cache = [torch.zeros(pages, HKV, P, D, dtype=BF, device="cuda") for _ in range(2)]
    kda.kda_kv_append(k[0], v[0], i32(range(T)), *cache)
    table = i32([list(range(pages))] * 40)
    lens = i32([T - 7 * b for b in range(40)])

    def prompt(s=None):
        return kda.kda_attn_fwd(q, k, v, scale=0.09, stream=s)

    def linear(s=None):
        return kda.kda_linear(x, w, stream=s)

    def step(s=None):
        return kda.kda_attn_step(q[0, :40], *cache, table, lens, scale=0.09, prefix_table=table[0], prefix_len=1000, stream=s)

    calls = (prompt, linear, step, prompt)
    alone = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        got = [[c(s) for _ in range(3)] for c, s in zip(calls, streams)]
        torch.cuda.synchronize()
        for a, g in zip(alone, got):
            assert all(torch.equal(a, y) for y in g)


def test_captured_calls():
    """Graphs of prompts, an 8-bit prefix and few rows on a long table, two of them in flight at once."""
    gen = torch.Generator().manual_seed(7)
    T, HQ, HKV, D, P = 300, 6, 2, 64, 32
    q, k, v = randn(gen, 1, T, HQ, D).cuda(), randn(gen, 1, T, HKV, D).cuda(), randn(gen, 1, T, HKV, D).cuda()
    pages = 600
    cache = [torch.zeros(pages, HKV, P, D, dtype=torch.uint8, device="cuda").view(E4) for _ in range(2)]
    scales = [torch.ones(pages, HKV, P, device="cuda") for _ in range(2)]
    table, lens = i32([list(range(520))] * 2), i32([T, T - 100])

    def all_of_it():
        kda.kda_kv_append(k[0], v[0], slots, *cache, k_scale=scales[0], v_scale=scales[1])
        a = kda.kda_attn_fwd(q, k, v, scale=0.125)
        b = kda.kda_attn_step(q[0, :2], *cache, table, lens, scale=0.125, k_scale=scales[0], v_scale=scales[1], prefix_table=table[0], prefix_len=77)
        return a, b

    slots = i32(range(T))
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(all_of_it())
        graphs.append(g)
    for round in range(3):
        q.copy_(randn(gen, 1, T, HQ, D)), k.copy_(randn(gen, 1, T, HKV, D)), v.copy_(randn(gen, 1, T, HKV, D))
        torch.cuda.synchronize()
        want = [x.clone() for x in all_of_it()]
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        for got in outs:
            assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_one_slot_for_several_rows():
    """Rows that read the same pages (a request forked) and the same row twice."""
    gen = torch.Generator().manual_seed(8)
    HQ, HKV, D, P, S = 4, 2, 128, 16, 60
    k, v, q = randn(gen, S, HKV, D), randn(gen, S, HKV, D), randn(gen, 1, HQ, D)
    cache = Cache(gen, [k], [v], P).cuda()
    one = kda.kda_attn_step(q.cuda(), cache.k, cache.v, cache.table, cache.lens, scale=0.1)
    three = kda.kda_attn_step(q.repeat(3, 1, 1).cuda(), cache.k, cache.v, cache.table.repeat(3, 1), cache.lens.repeat(3), scale=0.1)
    assert all(torch.equal(one[0], x) for x in three)
    # a prefix that is the row's own tokens too: each key counts twice, which changes nothing
    twice = kda.kda_attn_step(q.cuda(), cache.k, cache.v, cache.table, cache.lens, scale=0.1, prefix_table=cache.table[0].contiguous(), prefix_len=S)
    check(twice, None, ao.attend(np64(q), np64(k), np64(v), float(np.float32(0.1)), [S]), 2 * S, D)


def test_a_workspace_of_the_callers():
    gen = torch.Generator().manual_seed(9)
    HQ, HKV, D, P, S = 4, 2, 64, 16, 90
    k, v, q = randn(gen, S, HKV, D), randn(gen, S, HKV, D), randn(gen, 2, HQ, D).cuda()
    cache = Cache(gen, [k], [v], P).cuda()
    kw = dict(scale=0.125, prefix_table=cache.table[0].contiguous(), prefix_len=S)
    rows = (q, cache.k, cache.v, i32([[0], [0]]), i32([0, 0]))
    want = kda.kda_attn_step(*rows, **kw)
    space = torch.empty(1 << 20, dtype=torch.uint8, device="cuda").fill_(255)
    assert torch.equal(kda.kda_attn_step(*rows, workspace=space, **kw), want)
    with pytest.raises(ValueError):
        kda.kda_attn_step(*rows, workspace=space[:100], **kw)
    with pytest.raises(kda.KdaError):
        kda.kda_attn_step(*rows, workspace=space[16:], **kw)


def test_python_refusals():
    z = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    q, k = z(1, 8, 4, 64), z(1, 8, 2, 64)
    cache, table, lens = z(4, 2, 16, 64), torch.zeros(1, 2, dtype=torch.int32, device="cuda"), i32([8])
    for error, call in (
            (ValueError, lambda: kda.kda_attn_fwd(q, k, z(1, 9, 2, 64), scale=1.0)),
            (ValueError, lambda: kda.kda_attn_fwd(q.float(), k, k, scale=1.0)),
            (ValueError, lambda: kda.kda_attn_fwd(q, k.float(), k, scale=1.0)),
            (ValueError, lambda: kda.kda_attn_fwd(q, z(2, 8, 2, 64), z(2, 8, 2, 64), scale=1.0)),
            (kda.KdaError, lambda: kda.kda_attn_fwd(q, z(1, 8, 3, 64), z(1, 8, 3, 64), scale=1.0)),
            (kda.KdaError, lambda: kda.kda_attn_fwd(q, k, k, scale=0.0)),
            (kda.KdaError, lambda: kda.kda_attn_fwd(q, k, k, scale=1.0, o=q)),
            (kda.KdaError, lambda: kda.kda_attn_fwd(z(1, 8, 4, 96), z(1, 8, 2, 96), z(1, 8, 2, 96), scale=1.0)),
            (ValueError, lambda: kda.kda_attn_fwd(q, k, k, scale=1.0, cu_seqlens=torch.tensor([0, 8], device="cuda"))),
            (ValueError, lambda: kda.kda_attn_fwd(q, k, k, scale=1.0, lse=z(1, 8, 4))),
            (ValueError, lambda: kda.kda_attn_fwd(q, k, k, scale=1.0, seq_lens_k=lens)),
            (ValueError, lambda: kda.kda_attn_fwd(q, cache, cache, scale=1.0, block_table=table)),
            (ValueError, lambda: kda.kda_attn_fwd(q, cache.to(E4), cache.to(E4), scale=1.0, block_table=table, seq_lens_k=lens)),
            (ValueError, lambda: kda.kda_attn_fwd(q.transpose(1, 2), k, k, scale=1.0)),
            (kda.KdaError, lambda: kda.kda_attn_fwd(z(1, 8, 4 * 64 + 1)[..., 1:].view(1, 8, 4, 64), k, k, scale=1.0)),
            (ValueError, lambda: kda.kda_kv_append(k[0], k[0], i32(range(7)), cache, cache)),
            (ValueError, lambda: kda.kda_kv_append(k[0], k[0], i32(range(8)), cache, cache.to(E4))),
            (ValueError, lambda: kda.kda_kv_append(k[0], k[0], i32(range(8)), cache.to(E4), cache.to(E4))),
            (ValueError, lambda: kda.kda_kv_append(k[0], k[0], i32(range(8)), cache, cache, positions=i32(range(8)))),
            (ValueError, lambda: kda.kda_kv_append(k[0], k[0], i32(range(8)), cache, cache, q_out=q[0])),
            (kda.KdaError, lambda: kda.kda_kv_append(k[0], k[0], i32(range(8)), cache, cache, positions=i32(range(8)), cos_sin=z(9, 66, dtype=F32))),
            (kda.KdaError, lambda: kda.kda_kv_append(k[0], k[0], i32(range(8)), cache, cache, check_indices=True)),
            (ValueError, lambda: kda.kda_attn_step(q[0], cache, cache, table, lens, scale=1.0)),
            (ValueError, lambda: kda.kda_attn_step(q[0, :1], cache, cache, table, lens, scale=1.0, prefix_len=5)),
            (ValueError, lambda: kda.kda_attn_step(q[0, :1], cache, cache, table, lens, scale=1.0, k_scale=z(4, 2, 16, dtype=F32))),
            (kda.KdaError, lambda: kda.kda_attn_step(q[0, :1], z(4, 2, 8, 64), z(4, 2, 8, 64), table, lens, scale=1.0))):
        with pytest.raises(error):
            call()


@pytest.mark.parametrize("dtype", [BF, E4])
def test_results_that_wait_for_a_long_prefix(dtype):
    """Rows whose own tokens are done long before the prefix: run again and again, and captured,
    on workspaces that held other results; every time the same, and right."""
    gen = torch.Generator().manual_seed(31)
    B, HQ, HKV, D, P, prefix, pages = 160, 16, 4, 128, 64, 20000, 330
    own = [int(n) for n in torch.randint(1, 60, (B,), generator=gen)]
    kv = [randn(gen, pages, HKV, P, D) for _ in range(2)]
    scales = [None, None]
    stored = [np64(x) for x in kv]
    if dtype == E4:
        kv, scales = (list(x) for x in zip(*(quantised(x) for x in kv)))
        stored = [np64(x.float()) * np64(s)[..., None] for x, s in zip(kv, scales)]
    kc, vc = (x.cuda() for x in kv)
    ks, vs = (None if s is None else s.cuda() for s in scales)
    pre = torch.randperm(pages, generator=gen)[:-(-prefix // P)]
    rows = torch.randint(0, pages, (B, 1), generator=gen)
    lens = i32(own)
    q = randn(gen, B, HQ, D).cuda()
    call = dict(scale=0.09, k_scale=ks, v_scale=vs, prefix_table=pre.int().cuda(), prefix_len=prefix)
    table = rows.int().cuda()

    def step(lse):
        return kda.kda_attn_step(q, kc, vc, table, lens, lse=lse, **call)

    lse = torch.zeros(B, HQ, device="cuda")
    first = step(lse)
    torch.cuda.synchronize()
    for b in (0, 63, 64, 159):
        tokens = [np.concatenate([np.concatenate([x[p] for p in pre.tolist()], 1)[:, :prefix], x[int(rows[b])][:, :own[b]]], 1).transpose(1, 0, 2)
                  for x in stored]
        refs = ao.attend(np64(q[b:b + 1]), *tokens, float(np.float32(0.09)), [prefix + own[b]])
        check(first[b:b + 1], lse[b:b + 1], refs, prefix + own[b], D)
    queries = [q.clone(), randn(gen, B, HQ, D).cuda()]
    q.copy_(queries[1])
    second_lse = torch.zeros_like(lse)
    wanted = [(first, lse), (step(second_lse), second_lse)]
    graph, held = torch.cuda.CUDAGraph(), torch.zeros_like(lse)
    with torch.cuda.graph(graph):
        again = step(held)
    for i in range(20):
        q.copy_(queries[i % 2])
        graph.replay()
        other = torch.zeros_like(lse)
        eager = step(other)
        for o, l in ((again, held), (eager, other)):
            assert torch.equal(o, wanted[i % 2][0]) and torch.equal(l, wanted[i % 2][1])
