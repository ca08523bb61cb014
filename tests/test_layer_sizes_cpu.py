"""Sizes past 32 bits at the layer calls' Python wrappers: the C structs hold 32-bit
counts, and a tensor with more rows or columns than that is refused, not cut short.
No GPU: views of one element stand for the tensors, and the C call is recorded."""

import pytest
import torch

import kimi_delta_attention_04_gb300 as kda
from kimi_delta_attention_04_gb300 import _lib

BIG = 2 ** 32 + 5  # 5 in 32 bits
BF = torch.bfloat16


@pytest.fixture
def calls(monkeypatch):
    """What reaches the C calls, with CPU tensors let through."""
    made = []
    monkeypatch.setattr(_lib, "_lib", type("Recorder", (), {
        n: None for n in ("kda_add_rmsnorm", "kda_linear", "kda_scan_fwd", "kda_scan_bwd", "kda_scan_step")} |
        {"kda_linear_workspace_size": lambda self, args: 0})())
    monkeypatch.setattr(_lib, "_device_of", lambda x: x.get_device())
    monkeypatch.setattr(_lib, "_call", lambda fn, args, *rest: made.append(args))
    # (a view of one element has no spacing of its own)
    monkeypatch.setattr(_lib, "_rows", lambda t, *a: (None, 0) if t is None else (t.data_ptr(), t.shape[-1]))
    monkeypatch.setattr(_lib, "_vec", lambda t, *a, **k: None if t is None else t.data_ptr())
    return made


def view(*shape, dtype=BF):
    return torch.zeros(1, dtype=dtype).expand(shape)


def packed(n, dtype=torch.float32):
    """Any contiguous tensor will do where only the shape is looked at."""
    return torch.zeros(n, dtype=dtype)


def scan_args(B, T, D):
    x = view(B, T, D)
    return dict(x=x, gate=x, y=x, output_final_state=False)


CALLS = {
    "norm columns": lambda: kda.kda_add_rmsnorm(view(2, BIG), view(BIG, dtype=torch.float32), eps=1e-6, out=view(2, BIG)),
    "linear rows": lambda: kda.kda_linear(view(BIG, 8), view(16, 8), out=view(BIG, 16)),
    "linear outputs": lambda: kda.kda_linear(view(3, 8), view(BIG, 8), out=view(3, BIG)),
    "linear terms": lambda: kda.kda_linear(view(3, BIG), view(16, BIG), out=view(3, 16)),
    "scan tokens": lambda: kda.kda_scan_fwd(**scan_args(1, BIG, 4)),
    "scan batch": lambda: kda.kda_scan_fwd(**scan_args(BIG, 1, 4)),
    "scan channels": lambda: kda.kda_scan_fwd(**scan_args(1, 2, BIG)),
    "scan gradient": lambda: kda.kda_scan_bwd(view(1, BIG, 4), view(1, BIG, 4), view(1, BIG, 4), None, dx=view(1, BIG, 4),
                                              dgate=view(1, BIG, 4), output_dh0=False),
    "step rows": lambda: kda.kda_scan_step(view(BIG, 4), view(BIG, 4), packed((7, 4)), view(BIG, dtype=torch.int32),
                                           y=view(BIG, 4)),
    "step slots": lambda: kda.kda_scan_step(view(3, 4), view(3, 4), view(BIG, 4, dtype=torch.float32),
                                            packed(3, torch.int32), y=view(3, 4)),
}


@pytest.mark.parametrize("what", list(CALLS))
def test_sizes_past_32_bits_are_refused(calls, what):
    with pytest.raises(ValueError, match="32 bits"):
        CALLS[what]()
    assert not calls


def test_sizes_of_32_bits_pass(calls):
    n = 2 ** 31 - 1
    kda.kda_linear(view(n, 8), view(16, 8), out=view(n, 16))
    kda.kda_scan_fwd(**scan_args(1, n, 4))
    kda.kda_add_rmsnorm(view(BIG, 4), packed(4), eps=1e-6, out=view(BIG, 4))  # (its rows are counted in 64 bits)
    assert (calls[0].M, calls[1].T, calls[2].R) == (n, n, BIG)
