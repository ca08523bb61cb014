"""The layer operators without a GPU: struct layouts, host-side refusals, and
the fp64 oracle against closed forms and differences."""

import ctypes
import math
import subprocess
from pathlib import Path

import numpy as np
import pytest
import torch

import kimi_delta_attention_04_gb300 as kda
from kimi_delta_attention_04_gb300 import _lib
from kimi_delta_attention_04_gb300 import build as kbuild
from oracle import layer_oracle as lo

HEADER = Path(__file__).resolve().parents[1] / "include" / "kda.h"
FAKE = 0x10000
BF16, FP32, E4M3 = _lib.KDA_DTYPE_BF16, _lib.KDA_DTYPE_FP32, _lib.KDA_DTYPE_E4M3
INVALID, UNSUPPORTED = _lib.KDA_ERR_INVALID_ARG, _lib.KDA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return _lib.load()


STRUCTS = {"kda_add_rmsnorm_args": _lib.AddRmsNormArgs, "kda_linear_args": _lib.LinearArgs,
           "kda_scan_args": _lib.ScanArgs, "kda_scan_bwd_args": _lib.ScanBwdArgs,
           "kda_scan_step_args": _lib.ScanStepArgs}


def test_struct_layouts_match_c(tmp_path):
    lines = ['#include <stdio.h>', '#include <stddef.h>', f'#include "{HEADER}"', "int main(void){"]
    want = {}
    for name, st in STRUCTS.items():
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        want[name] = ctypes.sizeof(st)
        for f, _ in st._fields_:
            lines.append(f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));')
            want[f"{name}.{f}"] = getattr(st, f).offset
    for const in ("KDA_NORM_MAX_D", "KDA_DTYPE_E4M3", "KDA_ACT_RELU", "KDA_SCAN_LOGITS", "KDA_SCAN_FLAG_COMPLEMENT"):
        lines.append(f'printf("{const} %zu\\n", (size_t){const});')
    want |= {"KDA_NORM_MAX_D": _lib.KDA_NORM_MAX_D, "KDA_DTYPE_E4M3": E4M3, "KDA_ACT_RELU": _lib.KDA_ACTIVATIONS["relu"],
             "KDA_SCAN_LOGITS": _lib.KDA_SCAN_GATES["logits"], "KDA_SCAN_FLAG_COMPLEMENT": _lib.KDA_SCAN_FLAG_COMPLEMENT}
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0;}"]))
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    assert {k: int(v) for k, v in (line.split() for line in out.splitlines())} == want


def _fill(st, **kw):
    for k, v in kw.items():
        setattr(st, k, v)
    return st


def _norm(**over):
    return _fill(_lib.AddRmsNormArgs(), **(dict(
        R=4, D=100, dtype=BF16, y_dtype=E4M3, eps=1e-6, x_stride=100, residual_stride=100, residual_out_stride=100,
        y_stride=100, x=FAKE, residual=FAKE, weight=FAKE, residual_out=FAKE, y=FAKE, y_scale=FAKE) | over))


@pytest.mark.parametrize("over,status", [
    (dict(R=-1), INVALID), (dict(D=0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(dtype=7), INVALID), (dict(dtype=E4M3), UNSUPPORTED), (dict(D=_lib.KDA_NORM_MAX_D + 1), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(x=FAKE + 1), INVALID), (dict(weight=None), INVALID), (dict(weight=FAKE + 2), INVALID),
    (dict(y=None), INVALID), (dict(y_scale=None), INVALID), (dict(y_dtype=BF16), INVALID),  # a scale without 8 bits
    (dict(x_stride=99), INVALID), (dict(y_stride=-100), INVALID), (dict(residual_stride=1), INVALID),
    (dict(residual_out_stride=0), INVALID), (dict(y_scale=FAKE + 2), INVALID),
])
def test_add_rmsnorm_refuses(lib, over, status):
    assert lib.kda_add_rmsnorm(ctypes.byref(_norm(**over)), None) == status
    assert lib.kda_add_rmsnorm(None, None) == INVALID


def _linear(**over):
    return _fill(_lib.LinearArgs(), **(dict(
        M=5, N=7, K=33, dtype=BF16, y_dtype=BF16, activation=1, ldx=33, ldw=33, ld_residual=7, ldy=7, x=FAKE, w=FAKE,
        bias=FAKE, residual=FAKE, y=FAKE, err=FAKE) | over))


@pytest.mark.parametrize("over,status", [
    (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(activation=5), INVALID),
    (dict(activation=-1), INVALID), (dict(dtype=FP32), UNSUPPORTED), (dict(y_dtype=E4M3), UNSUPPORTED),
    (dict(dtype=9), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID),
    (dict(x=FAKE + 1), INVALID), (dict(ldx=32), INVALID), (dict(ldw=32), INVALID), (dict(ldy=6), INVALID),
    (dict(ld_residual=6), INVALID), (dict(bias=FAKE + 2), INVALID), (dict(err=FAKE + 2), INVALID),
    (dict(dtype=E4M3), INVALID),                                  # 8 bits need both scales
    (dict(dtype=E4M3, x_scale=FAKE), INVALID), (dict(dtype=E4M3, w_scale=FAKE), INVALID),
    (dict(x_scale=FAKE, w_scale=FAKE), INVALID),                  # bf16 takes none
])
def test_linear_refuses(lib, over, status):
    a = _linear(**over)
    assert lib.kda_linear(ctypes.byref(a), ctypes.c_void_p(FAKE), 1 << 30, None) == status
    assert lib.kda_linear_workspace_size(ctypes.byref(a)) == 0
    assert lib.kda_linear(None, None, 0, None) == INVALID


def test_linear_workspace(lib):
    """Nothing for rows on 16-byte boundaries; otherwise a copy at a pitch of 16 bytes, each rounded to 256."""
    def size(**over):
        return lib.kda_linear_workspace_size(ctypes.byref(_linear(**over)))
    assert size(K=40, ldx=40, ldw=48) == 0
    assert size(K=40, ldx=41, ldw=48) == 512           # 5 rows of 80 bytes
    assert size(K=40, ldx=40, ldw=41) == 768           # 7 rows of 80 bytes
    assert size() == 512 + 768                         # 33 values: 66 bytes, a pitch of 80
    assert size(M=1, K=40, ldx=41, ldw=40) == 0        # one row has no pitch
    assert size(M=1, K=40, ldx=41, ldw=40, x=FAKE + 2) == 256
    a = _linear()
    call = lambda ws, n: lib.kda_linear(ctypes.byref(a), ctypes.c_void_p(ws), n, None)  # noqa: E731
    assert call(None, 1 << 20) == INVALID and call(FAKE, 1279) == INVALID and call(FAKE + 16, 1 << 20) == INVALID


def _scan(**over):
    return _fill(_lib.ScanArgs(), **(dict(
        dtype=BF16, gate_dtype=FP32, B=2, T=40, D=30, N=2, gate_mode=1, flags=1, x_stride=30, gate_stride=30,
        y_stride=30, h_chunks_rows=6, x=FAKE, gate=FAKE, h0=FAKE, y=FAKE, hT=FAKE, h_chunks=FAKE, err=FAKE) | over))


SCAN_REFUSALS = [
    (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(D=0), INVALID), (dict(N=3), INVALID), (dict(flags=2), INVALID),
    (dict(gate_mode=2), INVALID), (dict(dtype=E4M3), UNSUPPORTED), (dict(dtype=FP32, gate_dtype=BF16), UNSUPPORTED),
    (dict(dtype=5), INVALID), (dict(cu_seqlens=FAKE), INVALID), (dict(cu_seqlens=FAKE + 2, B=1, N=3), INVALID),
    (dict(x=None), INVALID), (dict(gate=None), INVALID), (dict(x_stride=29), INVALID), (dict(gate_stride=0), INVALID),
    (dict(gate=FAKE + 2), INVALID), (dict(h_chunks_rows=5), INVALID), (dict(h_chunks=FAKE + 1), INVALID),
    (dict(err=FAKE + 1), INVALID),
]


@pytest.mark.parametrize("over,status", SCAN_REFUSALS + [
    (dict(y=None), INVALID), (dict(y_stride=3), INVALID), (dict(h0=FAKE + 2), INVALID), (dict(hT=FAKE + 2), INVALID)])
def test_scan_fwd_refuses(lib, over, status):
    assert lib.kda_scan_fwd(ctypes.byref(_scan(**over)), None) == status
    assert lib.kda_scan_fwd(None, None) == INVALID


@pytest.mark.parametrize("over,status", SCAN_REFUSALS + [(dict(h_chunks=None), INVALID)])
def test_scan_bwd_refuses_forward_arguments(lib, over, status):
    a = _fill(_lib.ScanBwdArgs(), fwd=_scan(**over), dy_stride=30, dx_stride=30, dgate_stride=30, dy=FAKE, dx=FAKE,
              dgate=FAKE)
    assert lib.kda_scan_bwd(ctypes.byref(a), None) == status


@pytest.mark.parametrize("over", [dict(dy=None), dict(dx=None), dict(dgate=None), dict(dy_stride=2), dict(dx_stride=29),
                                  dict(dgate_stride=29), dict(dgate=FAKE + 2), dict(dhT=FAKE + 2), dict(dh0=FAKE + 1)])
def test_scan_bwd_refuses(lib, over):
    a = _fill(_lib.ScanBwdArgs(), **(dict(fwd=_scan(), dy_stride=30, dx_stride=30, dgate_stride=30, dy=FAKE, dx=FAKE,
                                          dgate=FAKE) | over))
    assert lib.kda_scan_bwd(ctypes.byref(a), None) == INVALID
    assert lib.kda_scan_bwd(None, None) == INVALID


@pytest.mark.parametrize("over,status", [
    (dict(B=-1), INVALID), (dict(D=0), INVALID), (dict(num_slots=-1), INVALID), (dict(gate_mode=3), INVALID),
    (dict(flags=0x2), INVALID), (dict(flags=_lib.KDA_FLAG_CHECK_INDICES, err=None), INVALID),
    (dict(dtype=FP32, gate_dtype=BF16), UNSUPPORTED), (dict(x=None), INVALID), (dict(gate=None), INVALID),
    (dict(y=None), INVALID), (dict(indices=None), INVALID), (dict(indices=FAKE + 1), INVALID),
    (dict(state_in=None), INVALID), (dict(state_out=FAKE + 2), INVALID), (dict(x_stride=4), INVALID),
])
def test_scan_step_refuses(lib, over, status):
    a = _fill(_lib.ScanStepArgs(), **(dict(
        dtype=BF16, gate_dtype=BF16, B=3, D=20, num_slots=5, gate_mode=0, flags=0, x_stride=20, gate_stride=20,
        y_stride=20, x=FAKE, gate=FAKE, state_in=FAKE, state_out=FAKE, indices=FAKE, y=FAKE, err=FAKE) | over))
    assert lib.kda_scan_step(ctypes.byref(a), None) == status
    assert lib.kda_scan_step(None, None) == INVALID


def test_empty_calls_do_nothing(lib):
    """No rows: accepted on the host without a launch (there is no GPU here)."""
    assert lib.kda_add_rmsnorm(ctypes.byref(_norm(R=0, x=None, y=None)), None) == _lib.KDA_OK
    assert lib.kda_linear(ctypes.byref(_linear(M=0, x=None, y=None)), None, 0, None) == _lib.KDA_OK
    a = _fill(_lib.ScanStepArgs(), dtype=BF16, gate_dtype=BF16, B=0, D=20, num_slots=5)
    assert lib.kda_scan_step(ctypes.byref(a), None) == _lib.KDA_OK


def test_python_calls_refuse_cpu_tensors():
    x = torch.zeros(2, 3, 8)
    for call in (lambda: kda.kda_add_rmsnorm(x, x[0, 0], eps=1e-6), lambda: kda.kda_linear(x, x[0]),
                 lambda: kda.kda_scan_fwd(x, x), lambda: kda.kda_scan_bwd(x, x, x, x[0]),
                 lambda: kda.kda_scan_step(x[0], x[0], x[0], torch.zeros(3, dtype=torch.int32))):
        with pytest.raises(ValueError):
            call()


def test_python_calls_refuse_unknown_choices():
    x = torch.zeros(2, 3, 8)
    with pytest.raises(ValueError, match="activation"):
        kda.kda_linear(x, x[0], activation="tanh")
    with pytest.raises(ValueError, match="gate_mode"):
        kda.kda_scan_fwd(x, x, gate_mode="linear")
    with pytest.raises(ValueError, match="gate_mode"):
        kda.kda_scan_step(x[0], x[0], x[0], x[0], gate_mode="linear")


# --- the oracle ---

def test_oracle_norm_by_hand():
    y, r = lo.add_rmsnorm(np.array([[3.0, 4.0, 0.0, 0.0]]), np.array([[0.0, 0.0, 0.0, 0.0]]), np.array([1.0, 2, 3, 4]), 0.0)
    assert np.allclose(r, [[3, 4, 0, 0]]) and np.allclose(y, [[3 / 2.5, 8 / 2.5, 0, 0]])
    assert np.allclose(lo.row_scale(np.array([[0.0, -896.0], [0.0, 0.0]])), [2.0, 1.0])


def test_oracle_linear_by_hand():
    x, w = np.array([[1.0, 2.0]]), np.array([[3.0, -1.0], [-1.0, 0.0]])
    assert np.allclose(lo.linear(x, w, bias=np.array([1.0, 0.5]), activation="relu", residual=np.array([[10.0, 20]])),
                       [[12, 20]])
    assert np.allclose(lo.linear(x, w, x_scale=np.array([2.0]), w_scale=np.array([1.0, 4.0])), [[2, -8]])
    v = np.linspace(-4, 4, 9)
    assert np.allclose(lo.activate(v, "gelu"), torch.nn.functional.gelu(torch.from_numpy(v)).numpy())
    assert np.allclose(lo.activate(v, "silu"), torch.nn.functional.silu(torch.from_numpy(v)).numpy())


def test_oracle_scan_closed_form():
    """Constant decay: h_T = a^T h0 + sum a^(T-s) x_s."""
    rng = np.random.default_rng(0)
    x, a = rng.standard_normal((9, 3)), 0.7
    y, hT, _ = lo.scan(x, np.full((9, 3), math.log(a)), gate_mode="log", complement=False, h0=np.ones(3))
    want = a ** 9 + sum(a ** (8 - s) * x[s] for s in range(9))
    assert np.allclose(hT, want) and np.allclose(y[-1], want)
    z, _, _ = lo.scan(np.ones((50, 3)), rng.standard_normal((50, 3)), gate_mode="logits", complement=True, h0=np.ones(3))
    assert np.allclose(z, 1)  # a convex combination of ones


@pytest.mark.parametrize("gate_mode", ["log", "logits"])
@pytest.mark.parametrize("complement", [False, True])
def test_oracle_scan_gradient_against_differences(gate_mode, complement):
    rng = np.random.default_rng(1)
    T, D, eps = 7, 2, 1e-6
    x, gate, dy = rng.standard_normal((T, D)), -0.5 * rng.random((T, D)), rng.standard_normal((T, D))
    h0, dhT = rng.standard_normal(D), rng.standard_normal(D)

    def loss(x, gate, h0):
        y, hT, _ = lo.scan(x, gate, gate_mode=gate_mode, complement=complement, h0=h0)
        return (dy * y).sum() + (dhT * hT).sum()

    got = lo.scan_grad(x, gate, dy, gate_mode=gate_mode, complement=complement, h0=h0, dhT=dhT)
    for which, g in enumerate(got):
        for i in np.ndindex(g.shape):
            args = [[v.copy() for v in (x, gate, h0)] for _ in range(2)]
            args[0][which][i] += eps
            args[1][which][i] -= eps
            # central difference: error eps^2 f''' / 6 plus rounding 2^-52 |f| / eps ~ 1e-9
            assert abs((loss(*args[0]) - loss(*args[1])) / (2 * eps) - g[i]) < 1e-7
