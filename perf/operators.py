"""What the layer operators compute, as elementary torch operations, and the
calls a user makes of the library for the same: the residual add with RMS norm
(optionally to 8 bits with a scale per row), the projection with its epilogue,
and the gated linear recurrence (prefill, training step, single-token step).

Where ``own`` is false, run() takes the plain form, in 32 bits, rounded once at
the end; where it is true, the library's entry points."""

import math

import numpy as np
import torch

own = False

E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": E4M3}
BYTES = {"bf16": 2, "fp32": 4, "e4m3": 1}
CHUNK = 16  # tokens between the recurrence's saved states
EPS = 1e-6


def listed():
    return [
        # one decode step's norm in front of the packed q|k|v projection: 256 rows, 32 heads of 128
        dict(name="norm_decode", op="norm", R=256, D=4096, dtype="bf16", out="e4m3", res=True),
        # the same norm over an 8192-token prefill
        dict(name="norm_prefill", op="norm", R=8192, D=4096, dtype="bf16", out="e4m3", res=True),
        # a 32-bit residual stream of an odd width, first layer (nothing to add yet)
        dict(name="norm_odd", op="norm", R=1001, D=2501, dtype="fp32", out="bf16", res=False),
        # the packed q|k|v projection of a 256-row decode step
        dict(name="linear_decode", op="linear", M=256, K=4096, N=12288, dtype="bf16", act="none", bias=False, res=False),
        # the output projection of a 16-row decode step on 8-bit weights, into the residual stream
        dict(name="linear_decode8", op="linear", M=16, K=4096, N=4096, dtype="e4m3", act="none", bias=False, res=True),
        # the packed q|k|v projection of an 8192-token prefill
        dict(name="linear_prefill", op="linear", M=8192, K=4096, N=12288, dtype="bf16", act="none", bias=False, res=False),
        # a projection with its whole epilogue on 8-bit operands, 8192 tokens
        dict(name="linear_prefill8", op="linear", M=8192, K=4096, N=4096, dtype="e4m3", act="silu", bias=True, res=True),
        # odd sizes throughout: rows that start at no 16-byte boundary, ragged tiles on every side
        dict(name="linear_odd", op="linear", M=777, K=1001, N=1111, dtype="bf16", act="gelu", bias=True, res=True),
        # the recurrence over one long prompt
        dict(name="scan_prefill", op="scan", N=1, T=8192, D=4096, dtype="bf16", gate="bf16", mode="logits", comp=True, lens=0, train=False),
        # a training step of the recurrence: forward with saved states, then the gradients
        dict(name="scan_train", op="scan", N=4, T=4096, D=2048, dtype="bf16", gate="fp32", mode="log", comp=False, lens=0, train=True),
        # a training step on 16 packed sequences of 512 to 8192 tokens
        dict(name="scan_train_packed", op="scan", N=16, T=8192, D=1000, dtype="bf16", gate="bf16", mode="logits", comp=True, lens=512, train=True),
        # one token for each of 256 rows on a pool of state slots, a tenth of the rows padding
        dict(name="scan_step", op="step", B=256, D=4096, slots=512, dtype="bf16", gate="bf16", mode="logits", comp=True),
    ]


def _size(rng, lo, hi):
    """A size spread over its logarithm; half of them rounded to a multiple of 8."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, n // 8 * 8 if rng.random() < 0.5 and n >= 8 else n))


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "scan", "scan", "step"])
    if op == "norm":
        return dict(op=op, R=_size(rng, 1, 8192), D=_size(rng, 64, 8192), dtype=rng.choice(["bf16", "bf16", "fp32"]),
                    out=rng.choice(["e4m3", "e4m3", "bf16"]), res=rng.random() < 0.7)
    if op == "linear":
        return dict(op=op, M=_size(rng, 1, 8192), K=_size(rng, 128, 4096), N=_size(rng, 64, 12288),
                    dtype=rng.choice(["bf16", "e4m3"]), act=rng.choice(["none", "silu", "gelu", "sigmoid", "relu"]),
                    bias=rng.random() < 0.5, res=rng.random() < 0.5)
    mode, comp = rng.choice(["log", "logits"]), rng.random() < 0.5
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    gate = "fp32" if dtype == "fp32" else rng.choice(["bf16", "fp32"])
    if op == "step":
        B = _size(rng, 1, 512)
        return dict(op=op, B=B, D=_size(rng, 64, 8192), slots=B + _size(rng, 1, 512), dtype=dtype, gate=gate, mode=mode, comp=comp)
    D = _size(rng, 64, 4096)
    N = rng.randint(1, 16)
    T = _size(rng, 1, max(1, min(8192, 8192 * 4096 // (N * D))))
    return dict(op=op, N=N, T=T, D=D, dtype=dtype, gate=gate, mode=mode, comp=comp,
                lens=1 if rng.random() < 0.4 else 0, train=rng.random() < 0.5)


def _lengths(case):
    """Lengths of the packed sequences (lens to T tokens each), or None for N
    equal ones. They belong to the case: outputs have the same shape for every seed."""
    if not case["lens"]:
        return None
    rng = np.random.default_rng([case["N"], case["T"], case["D"]])
    return [int(v) for v in rng.integers(case["lens"], case["T"] + 1, case["N"])]


def _quantised(v):
    """Rows of v in e4m3 with one fp32 scale each."""
    s = v.abs().amax(1).clamp_min(1e-30) / E4M3_MAX
    return (v / s[:, None]).to(E4M3), s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    st = dict(case)
    op = case["op"]
    if op == "norm":
        R, D, dt = case["R"], case["D"], DTYPES[case["dtype"]]
        st["x"] = randn(R, D).to(dt)
        # residual streams grow with depth and have a few large channels
        st["residual"] = (3 * randn(R, D) * (1 + 10 * (torch.rand(D, generator=g, device="cuda") < 0.01))).to(dt) if case["res"] else None
        st["weight"] = 1 + 0.2 * randn(D)
        return st
    if op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        x, w = randn(M, K), randn(N, K) / math.sqrt(K)
        st["x_scale"] = st["w_scale"] = None
        if case["dtype"] == "e4m3":
            st["x"], st["x_scale"] = _quantised(x)
            st["w"], st["w_scale"] = _quantised(w)
        else:
            st["x"], st["w"] = x.to(torch.bfloat16), w.to(torch.bfloat16)
        st["bias"] = 0.1 * randn(N) if case["bias"] else None
        st["residual"] = randn(M, N).to(torch.bfloat16) if case["res"] else None
        return st
    D, dt, gt = case["D"], DTYPES[case["dtype"]], DTYPES[case["gate"]]
    # each channel has its own memory: decays from about 0.5 to 0.998 a token
    memory = 6 * torch.rand(D, generator=g, device="cuda")

    def gates(*lead):
        f = randn(*lead, D) + memory
        return (f if case["mode"] == "logits" else torch.nn.functional.logsigmoid(f)).to(gt)

    if op == "step":
        B, slots = case["B"], case["slots"]
        st["x"], st["gate_t"] = randn(B, D).to(dt), gates(B)
        st["pool"], st["pool_out"] = randn(slots, D), torch.zeros(slots, D, device="cuda")
        idx = torch.randperm(slots, generator=g, device="cuda")[:B].to(torch.int32)
        idx[torch.rand(B, generator=g, device="cuda") < 0.1] = -1
        st["indices"] = idx
        return st
    lens = _lengths(case)
    N = case["N"]
    if lens is None:
        shape = (N, case["T"])
        st["cu_seqlens"] = None
        st["chunks"] = N * -(-case["T"] // CHUNK)
    else:
        shape = (1, sum(lens))
        st["cu_seqlens"] = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")
        st["chunks"] = sum(-(-n // CHUNK) for n in lens)
    st["x"], st["gate_t"] = randn(*shape, D).to(dt), gates(*shape)
    st["h0"] = randn(N, D)
    if case["train"]:
        st["dy"], st["dhT"] = randn(*shape, D).to(dt), randn(N, D)
    return st


def _act(v, kind):
    if kind == "silu":
        return v / (1 + torch.exp(-v))
    if kind == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if kind == "sigmoid":
        return 1 / (1 + torch.exp(-v))
    return torch.where(v < 0, torch.zeros_like(v), v) if kind == "relu" else v


def _decay(gate, mode):
    f = gate.float()
    return torch.exp(f) if mode == "log" else 1 / (1 + torch.exp(-f))


def _scan(a, u):
    """h_t = a_t h_{t-1} + u_t from zero along dimension 1, by doubling: after the
    step of length s, (a, u) at t stand for the last 2 s tokens up to t. (An
    elementary operation for it does not exist; this takes log2 T rounds.)"""
    s = 1
    while s < u.shape[1]:
        u = torch.cat([u[:, :s], u[:, s:] + a[:, s:] * u[:, :-s]], 1)
        a = torch.cat([a[:, :s], a[:, s:] * a[:, :-s]], 1)
        s *= 2
    return u


def _plain_scan(st):
    dt, gt = st["x"].dtype, st["gate_t"].dtype
    x, a = st["x"].float(), _decay(st["gate_t"], st["mode"])
    cu, h0 = st["cu_seqlens"], st["h0"]
    u = (1 - a) * x if st["comp"] else x
    # where sequences start and end, as (row, token); a start takes a h0 into its
    # u and lets nothing of the sequence before it through
    if cu is None:
        rows = torch.arange(st["N"], device="cuda")
        first, last = torch.zeros_like(rows), torch.full_like(rows, st["T"] - 1)
    else:
        rows = torch.zeros(st["N"], dtype=torch.long, device="cuda")
        first, last = cu[:-1].long(), cu[1:].long() - 1
    a0 = a[rows, first]
    uh, ah = u.clone(), a.clone()
    uh[rows, first] += a0 * h0
    ah[rows, first] = 0
    h = _scan(ah, uh)
    out = dict(y=h.to(dt), hT=h[rows, last])
    if st["train"]:
        d = st["dy"].float().clone()
        d[rows, last] += st["dhT"]
        # d_t = dy_t + a_{t+1} d_{t+1}: the same scan over reversed time, the decays one token on
        an = torch.cat([ah[:, 1:], torch.zeros_like(ah[:, :1])], 1)
        d = _scan(an.flip(1), d.flip(1)).flip(1)
        hp = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
        hp[rows, first] = h0
        da = d * (hp - x) if st["comp"] else d * hp
        out["dx"] = ((1 - a) * d if st["comp"] else d).to(dt)
        out["dgate"] = (da * a * (1 if st["mode"] == "log" else 1 - a)).to(gt)
        out["dh0"] = a0 * d[rows, first]
    return out


def run(st):
    if own:
        return _run_own(st)
    op = st["op"]
    if op == "norm":
        r = st["x"].float()
        if st["residual"] is not None:
            r = r + st["residual"].float()
        y = r * torch.rsqrt((r * r).mean(1, keepdim=True) + EPS) * st["weight"]
        out = {}
        if st["residual"] is not None:
            out["residual"] = r.to(st["x"].dtype)
        if st["out"] == "e4m3":
            m = y.abs().amax(1)
            s = torch.where(m > 0, m / E4M3_MAX, torch.ones_like(m))
            out["y"], out["scale"] = (y / s[:, None]).to(E4M3), s
        else:
            out["y"] = y.to(DTYPES[st["out"]])
        return out
    if op == "linear":
        v = st["x"].float() @ st["w"].float().T
        if st["x_scale"] is not None:
            v = v * st["x_scale"][:, None] * st["w_scale"]
        if st["bias"] is not None:
            v = v + st["bias"]
        v = _act(v, st["act"])
        if st["residual"] is not None:
            v = v + st["residual"].float()
        return v.to(torch.bfloat16)
    if op == "step":
        idx = st["indices"].long()
        ok = (idx >= 0)[:, None]
        a, x = _decay(st["gate_t"], st["mode"]), st["x"].float()
        h = a * st["pool"][idx.clamp_min(0)] + ((1 - a) * x if st["comp"] else x)
        # (rows without a slot add nothing; slots are distinct)
        hit = torch.zeros(st["slots"], device="cuda").index_add(0, idx.clamp_min(0), ok[:, 0].float())
        new = torch.zeros_like(st["pool"]).index_add(0, idx.clamp_min(0), torch.where(ok, h, torch.zeros_like(h)))
        st["pool_out"].copy_(torch.where(hit[:, None] > 0, new, st["pool_out"]))
        return dict(y=torch.where(ok, h, torch.zeros_like(h)).to(st["x"].dtype), pool=st["pool_out"])
    return _plain_scan(st)


def _run_own(st):
    import kimi_delta_attention_04_gb300 as kda
    op = st["op"]
    if op == "norm":
        y, scale, r = kda.kda_add_rmsnorm(st["x"], st["weight"], eps=EPS, residual=st["residual"], out_dtype=DTYPES[st["out"]])
        out = {} if r is None else {"residual": r}
        out["y"] = y
        if scale is not None:
            out["scale"] = scale
        return out
    if op == "linear":
        return kda.kda_linear(st["x"], st["w"], bias=st["bias"], activation=st["act"], residual=st["residual"],
                              x_scale=st["x_scale"], w_scale=st["w_scale"])
    how = dict(gate_mode=st["mode"], complement=st["comp"])
    if op == "step":
        y = kda.kda_scan_step(st["x"], st["gate_t"], st["pool"], st["indices"], state_out=st["pool_out"], **how)
        return dict(y=y, pool=st["pool_out"])
    states = torch.empty(st["chunks"], st["D"], device="cuda") if st["train"] else None
    y, hT = kda.kda_scan_fwd(st["x"], st["gate_t"], h0=st["h0"], cu_seqlens=st["cu_seqlens"], h_chunks=states, **how)
    out = dict(y=y, hT=hT)
    if st["train"]:
        out["dx"], out["dgate"], out["dh0"] = kda.kda_scan_bwd(
            st["x"], st["gate_t"], st["dy"], states, dhT=st["dhT"], cu_seqlens=st["cu_seqlens"], **how)
    return out


def work(case):
    op = case["op"]
    if op == "norm":
        n, e = case["R"] * case["D"], BYTES[case["dtype"]]
        b = n * e * (3 if case["res"] else 1) + n * BYTES[case["out"]] + 4 * case["D"]
        return {"bytes": b + (4 * case["R"] if case["out"] == "e4m3" else 0), "flops": 6 * n}
    if op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        b = (M + N) * K * BYTES[case["dtype"]] + 2 * M * N * (2 if case["res"] else 1) + (4 * N if case["bias"] else 0)
        return {"bytes": b + (4 * (M + N) if case["dtype"] == "e4m3" else 0), "flops": 2 * M * N * K}
    e, f, D = BYTES[case["dtype"]], BYTES[case["gate"]], case["D"]
    if op == "step":
        return {"bytes": case["B"] * (D * (2 * e + f + 8) + 4), "flops": 8 * case["B"] * D}
    n = sum(_lengths(case) or [case["N"] * case["T"]]) * D
    b = n * (2 * e + f) + 8 * case["N"] * D
    if case["train"]:
        b += n * (3 * e + 2 * f) + 8 * case["N"] * D
    return {"bytes": b, "flops": (24 if case["train"] else 8) * n}


# ---- the definitions, in 64 bits ----

def _exact_scan(case, st):
    """Token by token over sequences laid side by side: [token, sequence, channel]."""
    D, N = case["D"], case["N"]
    lens = _lengths(case) or [case["T"]] * N
    L = max(lens)
    offs = np.concatenate([[0], np.cumsum(lens)])

    def apart(t):
        flat = t.reshape(-1, D).double()
        out = torch.zeros(L, N, D, dtype=torch.float64, device="cuda")
        for n in range(N):
            out[:lens[n], n] = flat[offs[n]:offs[n + 1]]
        return out

    def joined(t):
        return torch.cat([t[:lens[n], n] for n in range(N)]).reshape(st["x"].shape)

    f, x = apart(st["gate_t"]), apart(st["x"])
    a = f.exp() if case["mode"] == "log" else torch.sigmoid(f)
    w = 1 - a if case["comp"] else torch.ones_like(a)
    live = torch.tensor([[t < n for n in lens] for t in range(L)], device="cuda")[:, :, None]
    h, hs = st["h0"].double(), torch.empty_like(x)
    before = torch.empty_like(x)
    for t in range(L):
        before[t] = h
        h = torch.where(live[t], a[t] * h + w[t] * x[t], h)
        hs[t] = h
    out = dict(y=joined(hs), hT=h)
    if case["train"]:
        dy = apart(st["dy"])
        d = st["dhT"].double()
        dx, dg = torch.empty_like(x), torch.empty_like(x)
        for t in range(L - 1, -1, -1):
            e = d + dy[t]
            dx[t] = e * w[t]
            da = e * (before[t] - x[t] if case["comp"] else before[t])
            dg[t] = da * a[t] * (1 if case["mode"] == "log" else 1 - a[t])
            d = torch.where(live[t], a[t] * e, d)
        out |= dict(dx=joined(dx), dgate=joined(dg), dh0=d)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        r = st["x"].double() + (0 if st["residual"] is None else st["residual"].double())
        y = r / torch.sqrt(r.square().sum(1, keepdim=True) / case["D"] + EPS) * st["weight"].double()
        out = {} if st["residual"] is None else {"residual": r}
        if case["out"] != "e4m3":
            return out | {"y": y}
        top = y.abs().max(1).values
        scale = torch.where(top == 0, 1.0, top / E4M3_MAX)
        return out | {"y": y / scale[:, None], "scale": scale}
    if op == "linear":
        x, w = st["x"].double(), st["w"].double()
        if st["x_scale"] is not None:
            x, w = x * st["x_scale"].double()[:, None], w * st["w_scale"].double()[:, None]
        v = torch.matmul(x, w.t())
        if st["bias"] is not None:
            v += st["bias"].double()
        f = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu, "sigmoid": torch.sigmoid, "relu": torch.relu}.get(case["act"])
        v = v if f is None else f(v)
        return v if st["residual"] is None else v + st["residual"].double()
    if op == "step":
        y, pool = torch.zeros(case["B"], case["D"], dtype=torch.float64, device="cuda"), st["pool_out"].double()
        f = st["gate_t"].double()
        a = f.exp() if case["mode"] == "log" else torch.sigmoid(f)
        for i, slot in enumerate(st["indices"].tolist()):
            if slot >= 0:
                y[i] = a[i] * st["pool"][slot].double() + (1 - a[i] if case["comp"] else 1) * st["x"][i].double()
                pool[slot] = y[i]
        return dict(y=y, pool=pool)
    return _exact_scan(case, st)
