"""A pre-norm softmax attention layer with a paged cache on the library's calls, as it
stands between KDA layers of a hybrid stack: whole prompts, the next part of a prompt
whose beginning is cached, and single-token steps of requests that share a prefix.

    r         = x + residual; n = norm(r)             kda_add_rmsnorm
    [q|k|v]   = n W_qkv^T                             kda_linear
    q, k      turned by their positions;
    k, v      into the cache's pages                  kda_kv_append
    h         = softmax(scale q k^T) v                kda_attn_fwd / kda_attn_step
    out       = h W_out^T + r                         kda_linear (residual in its epilogue)

Run on a GPU: python examples/attention_layer.py
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import kimi_delta_attention_04_gb300 as kda  # noqa: E402

BF, E4M3 = torch.bfloat16, torch.float8_e4m3fn


class PagedCache:
    """Pages of keys and values, handed out one by one. 8 bits with a scale for each token and head if asked for."""

    def __init__(self, pages, heads, page_size, D, dtype=BF, device="cuda"):
        self.page_size, self.free = page_size, list(range(pages))
        self.k, self.v = (torch.empty(pages, heads, page_size, D, device=device, dtype=dtype) for _ in range(2))
        self.k_scale, self.v_scale = (torch.empty(pages, heads, page_size, device=device) if dtype == E4M3 else None for _ in range(2))

    def grow(self, pages, tokens):
        """Adds pages to a request's list until it has room for so many tokens."""
        while len(pages) * self.page_size < tokens:
            pages.append(self.free.pop())

    def slots(self, pages, first, last):
        """Places of a request's tokens first .. last - 1."""
        return [pages[t // self.page_size] * self.page_size + t % self.page_size for t in range(first, last)]


def table_of(page_lists, device="cuda"):
    width = max(1, max(len(p) for p in page_lists))
    return torch.tensor([p + [-1] * (width - len(p)) for p in page_lists], dtype=torch.int32, device=device)


def ints(values, device="cuda"):
    return torch.tensor(values, dtype=torch.int32, device=device)


class AttentionLayer:
    """Weights of one layer: width D of the residual stream, HQ query heads on HKV key heads of `head` channels."""

    def __init__(self, D, HQ, HKV, head, positions, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def randn(*shape):
            return torch.randn(*shape, generator=g, device=device)

        self.HQ, self.HKV, self.head, self.scale = HQ, HKV, head, head ** -0.5
        self.norm = 1 + 0.1 * randn(D)
        self.w_qkv = (randn((HQ + 2 * HKV) * head, D) / D ** 0.5).to(BF)
        self.w_out = (randn(D, HQ * head) / (HQ * head) ** 0.5).to(BF)
        angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * 10000.0 ** (
            -torch.arange(0, head, 2, dtype=torch.float64, device=device) / head)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()

    def project(self, x, residual, cache, slots, positions):
        """Tokens [n, D] -> (turned queries [n, HQ, head], turned keys, values, r); keys and values go to the cache."""
        n, _, r = kda.kda_add_rmsnorm(x, self.norm, eps=1e-6, residual=residual)
        p = kda.kda_linear(n, self.w_qkv).view(-1, self.HQ + 2 * self.HKV, self.head)
        q, k, v = p[:, :self.HQ], p[:, self.HQ:self.HQ + self.HKV], p[:, self.HQ + self.HKV:]
        q, k = kda.kda_kv_append(k, v, slots, cache.k, cache.v, q=q, k_out=k, positions=positions, cos_sin=self.cos_sin,
                                 k_scale=cache.k_scale, v_scale=cache.v_scale)
        return q, k, v, r

    def finish(self, h, r):
        return kda.kda_linear(h.reshape(-1, self.HQ * self.head), self.w_out, residual=r)

    def prompts(self, x, residual, cache, slots, positions, cu_seqlens):
        """Packed whole prompts, tokens [n, D]."""
        q, k, v, r = self.project(x, residual, cache, slots, positions)
        h = kda.kda_attn_fwd(q[None], k[None], v[None], scale=self.scale, cu_seqlens=cu_seqlens)
        return self.finish(h, r)

    def extend(self, x, residual, cache, slots, positions, cu_seqlens, table, lens):
        """The next tokens of packed prompts whose first ones the cache holds (bf16 caches)."""
        q, _, _, r = self.project(x, residual, cache, slots, positions)
        h = kda.kda_attn_fwd(q[None], cache.k, cache.v, scale=self.scale, cu_seqlens=cu_seqlens, block_table=table, seq_lens_k=lens)
        return self.finish(h, r)

    def step(self, x, residual, cache, slots, positions, table, lens, prefix_table=None, prefix_len=0):
        """One token a row, [B, D]; lens count each row's own tokens, this one among them."""
        q, _, _, r = self.project(x, residual, cache, slots, positions)
        h = kda.kda_attn_step(q, cache.k, cache.v, table, lens, scale=self.scale, k_scale=cache.k_scale, v_scale=cache.v_scale,
                              prefix_table=prefix_table, prefix_len=prefix_len)
        return self.finish(h, r)


def main(dtype=BF):
    """Two requests with a common beginning: each as one prompt, and as the shared beginning computed
    once, (bf16 caches: a part each as an extension of it,) and single tokens."""
    D, HQ, HKV, head, page = 512, 8, 2, 128, 16
    shared, part, steps = 70, 0 if dtype == E4M3 else 45, 6
    layer = AttentionLayer(D, HQ, HKV, head, positions=400)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    common = torch.randn(shared, D, generator=g, device="cuda").to(BF)
    own = [torch.randn(part + steps, D, generator=g, device="cuda").to(BF) for _ in range(2)]
    total = shared + part + steps

    # each request as one prompt
    cache = PagedCache(60, HKV, page, head, dtype)
    pages = [[], []]
    for p in pages:
        cache.grow(p, total)
    x = torch.cat([common, own[0], common, own[1]])
    whole = layer.prompts(x, x, cache, ints(sum((cache.slots(p, 0, total) for p in pages), [])), ints(list(range(total)) * 2),
                          ints([0, total, 2 * total])).view(2, total, D)

    # the beginning once, then what each request adds, then tokens one by one
    cache = PagedCache(60, HKV, page, head, dtype)
    prefix, rows = [], [[], []]
    cache.grow(prefix, shared)
    layer.prompts(common, common, cache, ints(cache.slots(prefix, 0, shared)), ints(range(shared)), ints([0, shared]))
    outs = [[], []]
    if part:
        # (an extension reads one table a request: the shared pages, then its own; the shared
        # part's last page is not full, so its tokens are copied to the request's own first page)
        full = shared // page
        rest = shared - full * page
        for p in rows:
            cache.grow(p, rest + part + steps)
            for c in (cache.k, cache.v):
                c[p[0], :, :rest] = c[prefix[full], :, :rest]
        table = table_of([prefix[:full] + p for p in rows])
        x = torch.cat([o[:part] for o in own])
        slots = sum((cache.slots(p, rest, rest + part) for p in rows), [])
        out = layer.extend(x, x, cache, ints(slots), ints(list(range(shared, shared + part)) * 2), ints([0, part, 2 * part]), table,
                           ints([shared + part] * 2))
        for b in range(2):
            outs[b].append(out[b * part:(b + 1) * part])
        prefix_len, offset = full * page, rest + part
    else:
        for p in rows:
            cache.grow(p, steps)
        prefix_len, offset = shared, 0
    prefix_table = ints(prefix)
    table = table_of(rows)
    for t in range(steps):
        x = torch.stack([o[part + t] for o in own])
        slots = [cache.slots(p, offset + t, offset + t + 1)[0] for p in rows]
        out = layer.step(x, x, cache, ints(slots), ints([shared + part + t] * 2), table, ints([offset + t + 1] * 2), prefix_table, prefix_len)
        for b in range(2):
            outs[b].append(out[b:b + 1])
    again = torch.stack([torch.cat(o) for o in outs])
    off = float((again.float() - whole[:, shared:].float()).norm() / whole[:, shared:].float().norm())
    print(f"shared beginning, extension and {steps} steps against whole prompts ({dtype}): {off:.1e}")
    return off


if __name__ == "__main__":
    main()
    main(E4M3)
