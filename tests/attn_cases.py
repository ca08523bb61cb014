"""Inputs and error bounds of the softmax attention tests."""

import numpy as np
import torch

from kda_cases import np64
from oracle import attn_oracle as ao

BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
NAN = float("nan")


def randn(gen, *shape, dtype=BF):
    return torch.randn(*shape, generator=gen).to(dtype)


def quantised(x):
    """(stored e4m3, fp32 scales) of heads x [..., D] in fp32."""
    s = torch.from_numpy(ao.power_scale(np64(x))).float()
    return (x.float() / s[..., None]).to(E4), s


class Cache:
    """A paged cache that holds the given sequences (k, v: lists of [S_n, HKV, D]) on pages
    in random order. Places that no token has hold NaN, and so do the pages left over;
    table entries behind a sequence's last page are out of range."""

    def __init__(self, gen, ks, vs, P, dtype=BF, spare=3):
        HKV, D = ks[0].shape[1:]
        need = [-(-len(k) // P) for k in ks]
        order = torch.randperm(sum(need) + spare, generator=gen)
        pages = len(order)
        self.P, self.dtype = P, dtype
        self.table = torch.full((len(ks), max(1, max(need))), 2 ** 30, dtype=torch.int32)
        self.lens = torch.tensor([len(k) for k in ks], dtype=torch.int32)
        self.k = torch.full((pages, HKV, P, D), NAN).to(dtype)
        self.v = self.k.clone()
        self.k_scale = self.v_scale = None
        if dtype == E4:  # (the 8-bit NaN is the scale's: stored values are finite)
            self.k, self.v = (torch.full((pages, HKV, P, D), 448.0).to(E4) for _ in range(2))
            self.k_scale, self.v_scale = (torch.full((pages, HKV, P), NAN) for _ in range(2))
        at = 0
        for n, (k, v) in enumerate(zip(ks, vs)):
            self.table[n, :need[n]] = order[at:at + need[n]].int()
            for c in range(need[n]):
                page, a, b = int(order[at + c]), c * P, min(len(k), (c + 1) * P)
                for name, x in (("k", k), ("v", v)):
                    x = x[a:b].transpose(0, 1)
                    if dtype == E4:
                        x, s = quantised(x)
                        getattr(self, name + "_scale")[page, :, :b - a] = s
                        getattr(self, name).view(torch.uint8)[page, :, :b - a] = x.view(torch.uint8)
                    else:
                        getattr(self, name)[page, :, :b - a] = x
            at += need[n]

    def tokens(self, n):
        """Sequence n's keys and values as stored, fp64 [S, HKV, D]."""
        return tuple(ao.tokens_of(np64(x.float()), self.table[n].numpy(), int(self.lens[n]), None if s is None else np64(s))
                     for x, s in ((self.k, self.k_scale), (self.v, self.v_scale)))

    def cuda(self):
        for name in ("k", "v", "k_scale", "v_scale", "table", "lens"):
            x = getattr(self, name)
            setattr(self, name, None if x is None else x.cuda())
        return self


def errors(a, top, n, D):
    """(error of o, error of lse) of rows of up to n keys, before o is rounded.

    A score is a sum of D products in fp32, in steps of 16 and 8 that the tensor core may
    truncate (2^-23 of the terms' magnitudes each), times a rounded factor, minus a rounded
    maximum: at most (D / 8 + 6) 2^-23 top. A weight is off by that, relatively, by 2^-21 of
    the special function, and by bf16's 2^-8; its sum and the products' sums by the same and
    by n / 8 truncated fp32 additions; their quotient by both sides."""
    score = (D / 8 + 6) * 2.0 ** -23 * top
    sums = 2.0 ** -21 + (n / 8 + 8) * 2.0 ** -23
    each = 2 * (np.expm1(score) + sums)
    return a * (each[..., None] + 2.0 ** -8), each + 2.0 ** -22 * (1 + top)


def check(got, got_lse, refs, n, D):
    """Compares o [rows, HQ, D] (bf16) and lse with the oracle's results."""
    o, lse, a, top = refs
    e_o, e_lse = errors(a, top, n, D)
    got = np64(got)
    bound = e_o + 2.0 ** -8 * (np.abs(o) + e_o) + 1e-37
    bad = ~(np.abs(got - o) <= bound)
    assert not bad.any(), f"o: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - o) / bound):.2f} times the bound"
    if got_lse is not None:
        got_lse = np64(got_lse)
        with np.errstate(invalid="ignore"):  # -inf on both sides
            same = (got_lse == lse) | (np.abs(got_lse - lse) <= e_lse)
        assert same.all(), f"lse: worst {np.nanmax(np.abs(got_lse - lse) / e_lse):.2f} times the bound"
