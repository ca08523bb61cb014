"""A pre-norm gated recurrent layer on the library's calls, as it stands between
KDA layers of a hybrid stack: prefill, single-token decode, and the gradients of
its recurrence.

    r         = x + residual                          kda_add_rmsnorm
    n, scale  = norm(r) in 8 bits                          "
    [u | f]   = n W_in^T + b (8-bit operands)         kda_linear
    h_t       = a_t h_{t-1} + (1 - a_t) u_t,          kda_scan_fwd / kda_scan_step
                a = sigmoid(f)
    out       = h W_out^T + r                         kda_linear (residual in its epilogue)

Run on a GPU: python examples/gated_recurrent_layer.py
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import kimi_delta_attention_04_gb300 as kda  # noqa: E402

E4M3 = torch.float8_e4m3fn


class GatedRecurrentLayer:
    """Weights of one layer: D the width of the residual stream, C the channels of
    the recurrence. The input projection is kept in 8 bits, quantised once."""

    def __init__(self, D, C, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def randn(*shape):
            return torch.randn(*shape, generator=g, device=device)

        self.D, self.C = D, C
        self.norm = 1 + 0.1 * randn(D)
        w_in = randn(2 * C, D) / D ** 0.5
        self.w_in_scale = w_in.abs().amax(1) / 448
        self.w_in = (w_in / self.w_in_scale[:, None]).to(E4M3)
        # the gate's bias gives each channel a memory of its own
        self.b_in = torch.cat([torch.zeros(C, device=device), 6 * torch.rand(C, generator=g, device=device)])
        self.w_out = (randn(D, C) / C ** 0.5).to(torch.bfloat16)

    def project(self, x, residual):
        """(u, f, r): the recurrence's input and gate logits, and the residual stream."""
        n, scale, r = kda.kda_add_rmsnorm(x, self.norm, eps=1e-6, residual=residual, out_dtype=E4M3)
        p = kda.kda_linear(n, self.w_in, x_scale=scale, w_scale=self.w_in_scale, bias=self.b_in)
        return p[..., :self.C], p[..., self.C:], r

    def prefill(self, x, residual, h0=None, cu_seqlens=None):
        """x, residual [B, T, D] -> (out [B, T, D], final states [N, C])."""
        u, f, r = self.project(x, residual)
        h, hT = kda.kda_scan_fwd(u, f, gate_mode="logits", complement=True, h0=h0, cu_seqlens=cu_seqlens)
        return kda.kda_linear(h, self.w_out, residual=r), hT

    def step(self, x, residual, pool, indices):
        """x, residual [B, D], one token a row; pool [slots, C] is updated in place."""
        u, f, r = self.project(x, residual)
        h = kda.kda_scan_step(u, f, pool, indices, gate_mode="logits", complement=True)
        return kda.kda_linear(h, self.w_out, residual=r)

    def recurrence_gradients(self, x, residual, dy):
        """(du, df, dh0) of sum(dy * h): the recurrence's part of a training step."""
        u, f, _ = self.project(x, residual)
        states = torch.empty(kda.chunk_count(u.shape[0], u.shape[1]), self.C, device=u.device)
        kda.kda_scan_fwd(u, f, gate_mode="logits", complement=True, h_chunks=states)
        return kda.kda_scan_bwd(u, f, dy, states, gate_mode="logits", complement=True)


def main():
    D, C, B, T = 1024, 512, 2, 300
    layer = GatedRecurrentLayer(D, C)
    x = torch.randn(B, T, D, device="cuda", dtype=torch.bfloat16)
    res = torch.randn(B, T, D, device="cuda", dtype=torch.bfloat16)
    whole, hT = layer.prefill(x, res)

    # the same tokens as a prefill and then single-token steps on a pool of states
    n = T - 8
    first, h = layer.prefill(x[:, :n].contiguous(), res[:, :n].contiguous())
    pool = torch.zeros(5, C, device="cuda")
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    pool[slots.long()] = h
    steps = [layer.step(x[:, t].contiguous(), res[:, t].contiguous(), pool, slots) for t in range(n, T)]
    again = torch.cat([first, torch.stack(steps, 1)], 1)
    off = float((again.float() - whole.float()).norm() / whole.float().norm())
    state_off = float((pool[slots.long()] - hT).norm() / hT.norm())

    du, df, dh0 = layer.recurrence_gradients(x, res, torch.randn(B, T, C, device="cuda", dtype=torch.bfloat16))
    print(f"prefill + {T - n} steps against one prefill: outputs {off:.1e}, states {state_off:.1e}; "
          f"gradients {tuple(du.shape)} {tuple(df.shape)} {tuple(dh0.shape)}")
    return off, state_off


if __name__ == "__main__":
    main()
