"""What the softmax attention calls compute, as elementary torch operations, and the
calls a user makes of the library for the same: attention over whole prompts (packed
sequences, grouped heads, keys in a paged cache), the append of rotated keys and of
values to that cache, and the single-token step on it, with a prefix that all rows
share.

Where ``own`` is false, run() takes the plain form, in 32 bits, rounded once at
the end; where it is true, the library's entry points."""

import math

import numpy as np
import torch

own = False

E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "e4m3": E4M3}
BYTES = {"bf16": 2, "e4m3": 1}
THETA = 10000.0


def listed():
    return [
        # one 8192-token prompt, 32 query heads of 128 on 8 key heads
        dict(name="prompt_long", op="prompt", N=1, T=8192, lens=0, ctx=0, HQ=32, HKV=8, D=128, P=0, causal=True),
        # 16 packed prompts of 512 to 8192 tokens, 16 heads on 2
        dict(name="prompt_packed", op="prompt", N=16, T=8192, lens=512, ctx=0, HQ=16, HKV=2, D=128, P=0, causal=True),
        # many short packed prompts, odd lengths from one token, heads of 64 in groups of 7
        dict(name="prompt_short", op="prompt", N=64, T=333, lens=1, ctx=0, HQ=14, HKV=2, D=64, P=0, causal=True),
        # the next 512 tokens of 4 prompts whose first 6000 are in the cache
        dict(name="prompt_extend", op="prompt", N=4, T=512, lens=0, ctx=6000, HQ=32, HKV=8, D=128, P=64, causal=True),
        # one decode step's keys and values of 256 rows into a bf16 cache, queries rotated on the way
        dict(name="append_decode", op="append", T=256, HQ=32, HKV=8, D=128, P=16, cache="bf16", rot=128, inter=False),
        # an 8192-token prefill into an 8-bit cache
        dict(name="append_prefill8", op="append", T=8192, HQ=32, HKV=8, D=128, P=64, cache="e4m3", rot=128, inter=False),
        # heads of 64 of which 32 channels are rotated in neighbouring pairs
        dict(name="append_partial", op="append", T=1777, HQ=14, HKV=2, D=64, P=32, cache="bf16", rot=32, inter=True),
        # 4 rows with short contexts: what a step costs before any work
        dict(name="step_small", op="step", B=4, least=1, most=500, HQ=32, HKV=8, D=128, P=16, prefix=0, cache="bf16"),
        # 64 rows with ragged contexts of up to 8192 tokens
        dict(name="step_ragged", op="step", B=64, least=1, most=8192, HQ=32, HKV=8, D=128, P=64, prefix=0, cache="bf16"),
        # 256 rows with contexts of about 2048 tokens in 8 bits
        dict(name="step_8bit", op="step", B=256, least=1500, most=2500, HQ=32, HKV=8, D=128, P=64, prefix=0, cache="e4m3"),
        # one row with a context of 131072 tokens
        dict(name="step_one", op="step", B=1, least=131072, most=131072, HQ=32, HKV=8, D=128, P=64, prefix=0, cache="bf16"),
        # 256 rows that share an 8192-token prefix and have up to 500 tokens of their own
        dict(name="step_prefix", op="step", B=256, least=1, most=500, HQ=32, HKV=8, D=128, P=64, prefix=8192, cache="bf16"),
    ]


def _size(rng, lo, hi):
    """A size spread over its logarithm; half of them rounded to a multiple of 8."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, n // 8 * 8 if rng.random() < 0.5 and n >= 8 else n))


def _heads(rng):
    hkv = rng.choice([1, 2, 4, 8])
    return hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 16][:8 if hkv < 4 else 7]), hkv


def draw(rng):
    op = rng.choice(["prompt", "prompt", "append", "step", "step"])
    HQ, HKV = _heads(rng)
    D, P = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    if op == "append":
        rot = rng.choice([D, D, D // 2, 0])
        return dict(op=op, T=_size(rng, 1, 8192), HQ=HQ, HKV=HKV, D=D, P=P, cache=rng.choice(["bf16", "e4m3"]),
                    rot=rot, inter=rng.random() < 0.3)
    if op == "prompt":
        paged = rng.random() < 0.4
        N = _size(rng, 1, 64)
        T = _size(rng, 1, 8192)
        case = dict(op=op, N=N, T=T, lens=1 if rng.random() < 0.6 else 0, ctx=rng.choice([0, _size(rng, 1, 8192)]) if paged else 0,
                    HQ=HQ, HKV=HKV, D=D, P=P if paged else 0, causal=rng.random() < 0.8)
        most = work(listed()[1])["flops"]
        # (no case costs more than the largest listed one: without the causal half a case has twice the products)
        while 2 * work(dict(case, causal=False))["flops"] > most:
            if case["T"] > 64 and case["T"] >= case["ctx"]:
                case["T"] = case["T"] * 2 // 3
            elif case["N"] > 1:
                case["N"] = case["N"] * 2 // 3
            else:
                case["ctx"] = case["ctx"] * 2 // 3
        return case
    cache = rng.choice(["bf16", "e4m3"])
    most = _size(rng, 1, 65536)
    B = max(1, min(_size(rng, 1, 256), 2 ** 22 // (most * HKV)))
    prefix = _size(rng, 1, 16384) if rng.random() < 0.4 else 0
    return dict(op=op, B=B, least=1, most=most, HQ=HQ, HKV=HKV, D=D, P=P, prefix=prefix, cache=cache)


def _lengths(n, least, most):
    """Lengths that belong to the case: outputs have the same shape for every seed."""
    rng = np.random.default_rng([n, least, most])
    return [int(v) for v in rng.integers(least, most + 1, n)]


def _queries(case):
    return _lengths(case["N"], case["lens"], case["T"]) if case["lens"] else [case["T"]] * case["N"]


def _quantised(v):
    """v in e4m3 with one scale for each last axis, the smallest power of two that
    brings its largest magnitude to 448 or less (1 for zeros)."""
    m = v.abs().amax(-1)
    f, e = torch.frexp(m / E4M3_MAX)
    s = torch.where(m > 0, torch.ldexp(torch.ones_like(m), torch.where(f > 0.5, e, e - 1)), torch.ones_like(m))
    return (v / s[..., None]).to(E4M3), s


def _table(positions, rot):
    """Cosines and sines of a rotary embedding, fp32 [positions, rot], angles in 64 bits."""
    f = THETA ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    st = dict(case)
    op, HQ, HKV, D, P = case["op"], case["HQ"], case["HKV"], case["D"], case["P"]
    st["scale"] = D ** -0.5

    def filled(pages, dtype):
        """A cache of keys (a common part in each channel, as trained keys have) and one of values."""
        k = randn(pages, HKV, P, D)
        k += randn(HKV, 1, D)
        v = randn(pages, HKV, P, D)
        if dtype == "bf16":
            st["k_cache"], st["v_cache"] = k.to(torch.bfloat16), v.to(torch.bfloat16)
            st["k_scale"] = st["v_scale"] = None
        else:
            st["k_cache"], st["k_scale"] = _quantised(k)
            st["v_cache"], st["v_scale"] = _quantised(v)

    def tables(lens, first=0):
        """Pages of the cache in random order for sequences of these lengths; unused entries are -1."""
        need = [-(-n // P) for n in lens]
        order = torch.randperm(sum(need) + first + 7, generator=g, device="cuda").to(torch.int32)
        table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
        at = first
        for i, n in enumerate(need):
            table[i, :n] = order[at:at + n]
            at += n
        return order, table

    if op == "prompt":
        lens = _queries(case)
        st["cu"] = ints([0] + list(np.cumsum(lens)))
        tokens = sum(lens)
        if P:
            keys = [n + case["ctx"] for n in lens]
            order, st["table"] = tables(keys)
            st["lens_k"] = ints(keys)
            st["q"] = (1.5 * randn(1, tokens, HQ, D)).to(torch.bfloat16)
            filled(order.numel(), "bf16")
        else:
            # views of one packed projection's output
            packed = randn(1, tokens, HQ + 2 * HKV, D)
            packed[:, :, :HQ] *= 1.5
            packed[:, :, HQ:HQ + HKV] += randn(HKV, D)
            packed = packed.to(torch.bfloat16)
            st["q"], st["k"], st["v"] = packed[:, :, :HQ], packed[:, :, HQ:HQ + HKV], packed[:, :, HQ + HKV:]
        return st
    if op == "append":
        T = case["T"]
        pages = -(-(T + T // 2 + 100) // P)
        packed = randn(T, HQ + 2 * HKV, D).to(torch.bfloat16)
        st["q"], st["k"], st["v"] = packed[:, :HQ], packed[:, HQ:HQ + HKV], packed[:, HQ + HKV:]
        slots = torch.randperm(pages * P, generator=g, device="cuda")[:T].to(torch.int32)
        slots[torch.rand(T, generator=g, device="cuda") < 0.05] = -1  # padding
        st["slots"] = slots
        st["cos_sin"] = _table(16384, case["rot"]) if case["rot"] else None
        st["positions"] = torch.randint(0, 16384, (T,), generator=g, device="cuda", dtype=torch.int32) if case["rot"] else None
        for name in ("k", "v"):
            st[name + "_cache"] = torch.zeros(pages, HKV, P, D, device="cuda").to(DTYPES[case["cache"]])
            st[name + "_scale"] = torch.ones(pages, HKV, P, device="cuda") if case["cache"] == "e4m3" else None
        return st
    lens = _lengths(case["B"], case["least"], case["most"])
    first = -(-case["prefix"] // P)
    order, st["table"] = tables(lens, first)
    st["prefix_table"] = order[:first].contiguous() if first else None
    st["lens_k"], st["longest"] = ints(lens), max(lens)
    st["q"] = (1.5 * randn(case["B"], HQ, D)).to(torch.bfloat16)
    filled(order.numel(), case["cache"])
    return st


def _softmax_rows(s, seen):
    """Softmax over the last axis of what `seen` lets through; rows that see nothing give zeros."""
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total == 0, torch.ones_like(total), total)


def _gathered(st, name, table, n):
    """The first n tokens of the cache's pages in a table [rows, pages]: fp32 [rows, HKV, n, D]."""
    pages = table[:, :-(-n // st["P"])].long().clamp_min(0)
    x = st[name + "_cache"][pages].float()  # [rows, pages, HKV, P, D]
    if st[name + "_scale"] is not None:
        x = x * st[name + "_scale"][pages][..., None]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)[:, :, :n]


def _plain_prompt(st):
    HQ, HKV, D = st["HQ"], st["HKV"], st["D"]
    G = HQ // HKV
    out = torch.empty_like(st["q"], memory_format=torch.contiguous_format)
    at = 0
    for i, T in enumerate(_queries(st)):
        q = st["q"][0, at:at + T].float().reshape(T, HKV, G, D)
        if st["P"]:
            S = T + st["ctx"]
            k, v = (_gathered(st, name, st["table"][i:i + 1], S)[0] for name in ("k", "v"))
        else:
            S = T
            k, v = (st[name][0, at:at + T].float().transpose(0, 1) for name in ("k", "v"))
        for a in range(0, T, 2048):  # (blocks of queries, for the memory the scores take)
            b = min(T, a + 2048)
            x = q[a:b].permute(1, 2, 0, 3).reshape(HKV, G * (b - a), D)
            s = (x @ k.transpose(1, 2)).view(HKV, G, b - a, S) * st["scale"]
            row = torch.arange(a, b, device="cuda")[:, None] + (S - T)
            col = torch.arange(S, device="cuda")
            p = _softmax_rows(s, (col <= row) if st["causal"] else (col >= 0))
            o = (p.view(HKV, G * (b - a), S) @ v).view(HKV, G, b - a, D)
            out[0, at + a:at + b] = o.permute(2, 0, 1, 3).reshape(b - a, HQ, D).to(out.dtype)
        at += T
    return out


def _rotated(x, st):
    """The first rot channels of x [T, heads, D] turned by their positions' angles."""
    rot = st["rot"]
    x = x.float()
    if not rot:
        return x
    c, s = (t[:, None] for t in st["cos_sin"][st["positions"].long()].split(rot // 2, 1))
    if st["inter"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _append_outputs(st, q):
    out = dict(q=q, k_cache=st["k_cache"], v_cache=st["v_cache"])
    if st["k_scale"] is not None:
        out |= dict(k_scale=st["k_scale"], v_scale=st["v_scale"])
    return out


def _plain_append(st):
    P = st["P"]
    idx = torch.nonzero(st["slots"] >= 0)[:, 0]
    slots = st["slots"][idx].long()
    page, offset = slots // P, slots % P
    for name, x in (("k", _rotated(st["k"], st)), ("v", st["v"].float())):
        x = x[idx]
        if st[name + "_scale"] is None:
            st[name + "_cache"][page, :, offset] = x.to(torch.bfloat16)
        else:
            x, s = _quantised(x)
            # (as bytes: torch has no indexed copy of 8-bit floats)
            st[name + "_cache"].view(torch.uint8)[page, :, offset] = x.view(torch.uint8)
            st[name + "_scale"][page, :, offset] = s
    return _append_outputs(st, _rotated(st["q"], st).to(torch.bfloat16))


def _plain_step(st):
    B, HQ, HKV, D, prefix = st["B"], st["HQ"], st["HKV"], st["D"], st["prefix"]
    G, n = HQ // HKV, st["longest"]
    q = st["q"].float().view(B, HKV, G, D)
    s = (q @ _gathered(st, "k", st["table"], n).transpose(2, 3)) * st["scale"]
    seen = (torch.arange(n, device="cuda") < st["lens_k"][:, None])[:, None, None].expand_as(s)
    if prefix:
        k = _gathered(st, "k", st["prefix_table"][None], prefix)[0]
        x = q.permute(1, 0, 2, 3).reshape(HKV, B * G, D)
        shared = (x @ k.transpose(1, 2)).view(HKV, B, G, prefix).transpose(0, 1) * st["scale"]
        s = torch.cat([shared, s], -1)
        seen = torch.cat([torch.ones_like(shared, dtype=torch.bool), seen], -1)
    p = _softmax_rows(s, seen)
    o = p[..., prefix:] @ _gathered(st, "v", st["table"], n)
    if prefix:
        v = _gathered(st, "v", st["prefix_table"][None], prefix)[0]
        x = p[..., :prefix].transpose(0, 1).reshape(HKV, B * G, prefix)
        o = o + (x @ v).view(HKV, B, G, D).transpose(0, 1)
    return o.reshape(B, HQ, D).to(torch.bfloat16)


def run(st):
    if own:
        return _run_own(st)
    return {"prompt": _plain_prompt, "append": _plain_append, "step": _plain_step}[st["op"]](st)


def _run_own(st):
    import kimi_delta_attention_04_gb300 as kda
    op = st["op"]
    if op == "prompt":
        if st["P"]:
            return kda.kda_attn_fwd(st["q"], st["k_cache"], st["v_cache"], scale=st["scale"], causal=st["causal"], cu_seqlens=st["cu"],
                                    block_table=st["table"], seq_lens_k=st["lens_k"])
        return kda.kda_attn_fwd(st["q"], st["k"], st["v"], scale=st["scale"], causal=st["causal"], cu_seqlens=st["cu"])
    if op == "append":
        q = kda.kda_kv_append(st["k"], st["v"], st["slots"], st["k_cache"], st["v_cache"], q=st["q"], positions=st["positions"],
                              cos_sin=st["cos_sin"], interleaved=st["inter"], k_scale=st["k_scale"], v_scale=st["v_scale"])[0]
        return _append_outputs(st, q)
    return kda.kda_attn_step(st["q"], st["k_cache"], st["v_cache"], st["table"], st["lens_k"], scale=st["scale"], k_scale=st["k_scale"],
                             v_scale=st["v_scale"], prefix_table=st["prefix_table"], prefix_len=st["prefix"])


def work(case):
    op, HQ, HKV, D = case["op"], case["HQ"], case["HKV"], case["D"]
    if op == "prompt":
        pairs = queries = keys = pages = 0
        for T in _queries(case):
            S = T + case["ctx"]
            pairs += T * S - T * (T - 1) // 2 if case["causal"] else T * S
            queries, keys = queries + T, keys + S
            pages += -(-S // case["P"]) if case["P"] else 0
        return {"bytes": 4 * queries * HQ * D + 4 * keys * HKV * D + 4 * pages, "flops": 4 * D * HQ * pairs}
    if op == "append":
        T, e = case["T"], BYTES[case["cache"]]
        b = 4 * T * HQ * D + 4 * T * HKV * D + 2 * T * HKV * D * e + 4 * T
        b += 8 * T * HKV if case["cache"] == "e4m3" else 0
        b += T * (4 * case["rot"] + 4) if case["rot"] else 0
        return {"bytes": b, "flops": 3 * T * (HQ + HKV) * case["rot"]}
    lens, P = _lengths(case["B"], case["least"], case["most"]), case["P"]
    keys = sum(lens) + case["prefix"]
    b = keys * HKV * (2 * D * BYTES[case["cache"]] + (8 if case["cache"] == "e4m3" else 0)) + 4 * case["B"] * HQ * D
    return {"bytes": b + 4 * (case["B"] + sum(-(-n // P) for n in lens + [case["prefix"]])),
            "flops": 4 * D * HQ * (sum(lens) + case["B"] * case["prefix"])}


# ---- the definitions, in 64 bits ----

def _attend(q, k, v, scale, hidden_after=None):
    """q [t, D], k and v [s, D]: softmax(scale q k^T) v; query i sees keys up to hidden_after + i."""
    s = torch.einsum("td,sd->ts", q, k) * scale
    if hidden_after is not None:
        s.masked_fill_(torch.ones_like(s, dtype=torch.bool).triu_(hidden_after + 1), -math.inf)
    return torch.softmax(s, 1) @ v


def _token_rows(st, name, pages, n, h):
    """Tokens 0 to n of key head h on these pages, in 64 bits."""
    x = st[name + "_cache"][pages, h].double()
    if st[name + "_scale"] is not None:
        x = x * st[name + "_scale"][pages, h].double().unsqueeze(-1)
    return x.reshape(-1, st["D"])[:n]


def exact(case, seed):
    st = prepare(case, seed)
    op, HQ, HKV, D, P = case["op"], case["HQ"], case["HKV"], case["D"], case["P"]
    G = HQ // HKV
    if op == "prompt":
        if work(dict(case, causal=False))["flops"] > 8e12:
            return None
        out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
        at = 0
        for i, T in enumerate(_queries(case)):
            S = T + case["ctx"]
            pages = st["table"][i, :-(-S // P)].long() if P else None
            for h in range(HQ):
                if h % G == 0:
                    k, v = (_token_rows(st, n, pages, S, h // G) if P else st[n][0, at:at + T, h // G].double() for n in ("k", "v"))
                for a in range(0, T, 4096):
                    b = min(T, a + 4096)
                    out[0, at + a:at + b, h] = _attend(st["q"][0, at + a:at + b, h].double(), k, v, case["D"] ** -0.5,
                                                       S - T + a if case["causal"] else None)
            at += T
        return out
    if op == "step":
        out = torch.empty(case["B"], HQ, D, dtype=torch.float64, device="cuda")
        shared = {}
        for h in range(HKV):
            for n in ("k", "v"):
                shared[n, h] = _token_rows(st, n, st["prefix_table"].long(), case["prefix"], h) if case["prefix"] else None
        for i, S in enumerate(_lengths(case["B"], case["least"], case["most"])):
            pages = st["table"][i, :-(-S // P)].long()
            for h in range(HKV):
                k, v = (_token_rows(st, n, pages, S, h) if shared[n, h] is None else torch.cat([shared[n, h], _token_rows(st, n, pages, S, h)])
                        for n in ("k", "v"))
                out[i, h * G:(h + 1) * G] = _attend(st["q"][i, h * G:(h + 1) * G].double(), k, v, D ** -0.5)
        return out

    def turned(x):
        x, rot = x.double(), case["rot"]
        if not rot:
            return x
        t = st["cos_sin"].double()[st["positions"].long()]
        z = torch.complex(t[:, :rot // 2], t[:, rot // 2:])[:, None]
        if case["inter"]:
            w = torch.view_as_real(torch.view_as_complex(x[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * z).flatten(-2)
        else:
            w = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * z
            w = torch.cat([w.real, w.imag], -1)
        return torch.cat([w, x[..., rot:]], -1)

    out = dict(q=turned(st["q"]))
    caches = {}
    for name, x in (("k", turned(st["k"])), ("v", st["v"].double())):
        top = x.abs().amax(-1)
        s = torch.where(top > 0, torch.exp2(torch.ceil(torch.log2(top / E4M3_MAX))), torch.ones_like(top))
        cache = st[name + "_cache"].double()
        scales = None if st[name + "_scale"] is None else st[name + "_scale"].double()
        live = st["slots"] >= 0
        slots = st["slots"][live].long()
        if scales is not None:
            flat = scales.transpose(1, 2).reshape(-1, HKV).clone()
            flat[slots] = s[live]
            scales = flat.view(-1, P, HKV).transpose(1, 2)
            x = x / s[..., None]
        flat = cache.transpose(1, 2).reshape(-1, HKV, D).clone()
        flat[slots] = x[live]
        caches[name] = flat.view(-1, P, HKV, D).transpose(1, 2), scales
    out |= dict(k_cache=caches["k"][0], v_cache=caches["v"][0])
    if caches["k"][1] is not None:
        out |= dict(k_scale=caches["k"][1], v_scale=caches["v"][1])
    return out
