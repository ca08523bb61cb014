"""The softmax attention calls without a GPU: struct layouts, host-side refusals, and the
fp64 oracle against closed forms and planted mistakes."""

import ctypes
import subprocess
from pathlib import Path

import numpy as np
import pytest
import torch

import kimi_delta_attention_04_gb300 as kda
from kimi_delta_attention_04_gb300 import _lib
from kimi_delta_attention_04_gb300 import build as kbuild
from oracle import attn_oracle as ao

import attn_cases
from attn_cases import BF, E4, Cache, errors

HEADER = Path(__file__).resolve().parents[1] / "include" / "kda.h"
FAKE = 0x10000
BF16, FP32, E4M3 = _lib.KDA_DTYPE_BF16, _lib.KDA_DTYPE_FP32, _lib.KDA_DTYPE_E4M3
INVALID, UNSUPPORTED = _lib.KDA_ERR_INVALID_ARG, _lib.KDA_ERR_UNSUPPORTED
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return _lib.load()


STRUCTS = {"kda_kv_append_args": _lib.KvAppendArgs, "kda_attn_fwd_args": _lib.AttnFwdArgs, "kda_attn_step_args": _lib.AttnStepArgs}


def test_struct_layouts_match_c(tmp_path):
    lines = ['#include <stdio.h>', '#include <stddef.h>', f'#include "{HEADER}"', "int main(void){"]
    want = {}
    for name, st in STRUCTS.items():
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        want[name] = ctypes.sizeof(st)
        for f, _ in st._fields_:
            lines.append(f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));')
            want[f"{name}.{f}"] = getattr(st, f).offset
    for const in ("KDA_KV_FLAG_INTERLEAVED", "KDA_ATTN_FLAG_CAUSAL", "KDA_ATTN_MAX_HEADS", "KDA_ATTN_LONG_TOKENS", "KDA_ATTN_MAX_TOKENS"):
        lines.append(f'printf("{const} %zu\\n", (size_t){const});')
        want[const] = getattr(_lib, const)
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0;}"]))
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    assert {k: int(v) for k, v in (line.split() for line in out.splitlines())} == want


def _fill(st, kw):
    for k, v in kw.items():
        setattr(st, k, v)
    return st


def _append(**over):
    return _fill(_lib.KvAppendArgs(), dict(
        tokens=4, HQ=4, HKV=2, D=64, pages=3, page_size=16, cache_dtype=BF16, rot=64, max_positions=10, q_stride=256, k_stride=128,
        v_stride=128, q_out_stride=256, k_out_stride=128, q=FAKE, k=FAKE, v=FAKE, slots=FAKE, positions=FAKE, cos_sin=FAKE, q_out=FAKE,
        k_out=FAKE, k_cache=FAKE, v_cache=FAKE) | over)


@pytest.mark.parametrize("over,status", [
    (dict(tokens=-1), INVALID), (dict(HQ=0), INVALID), (dict(HKV=0), INVALID), (dict(HQ=5), INVALID), (dict(D=96), UNSUPPORTED),
    (dict(D=0), INVALID), (dict(HQ=2048, q_stride=2 ** 20, q_out_stride=2 ** 20), UNSUPPORTED), (dict(pages=-1), INVALID),
    (dict(page_size=24), UNSUPPORTED), (dict(page_size=256), UNSUPPORTED), (dict(page_size=0), INVALID), (dict(page_size=-16), INVALID),
    (dict(pages=2 ** 27, page_size=16), INVALID), (dict(cache_dtype=FP32), UNSUPPORTED), (dict(cache_dtype=9), INVALID),
    (dict(cache_dtype=E4M3), INVALID), (dict(cache_dtype=E4M3, k_scale=FAKE), INVALID), (dict(k_scale=FAKE, v_scale=FAKE), INVALID),
    (dict(cache_dtype=E4M3, k_scale=FAKE + 4, v_scale=FAKE), INVALID), (dict(rot=-2), INVALID), (dict(rot=63), INVALID),
    (dict(rot=66), INVALID), (dict(max_positions=-1), INVALID), (dict(positions=None), INVALID), (dict(cos_sin=None), INVALID),
    (dict(cos_sin=FAKE + 4), INVALID), (dict(positions=FAKE + 2), INVALID), (dict(rot=0), INVALID), (dict(slots=None), INVALID),
    (dict(slots=FAKE + 1), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=FAKE + 8), INVALID),
    (dict(k_stride=127), INVALID), (dict(k_stride=132), INVALID), (dict(v_stride=-128), INVALID), (dict(q=None), INVALID),
    (dict(q_out=None), INVALID), (dict(q_out=FAKE + 8), INVALID), (dict(k_out=FAKE + 2), INVALID), (dict(k_out_stride=64), INVALID),
    (dict(k_cache=None), INVALID), (dict(v_cache=FAKE + 8), INVALID), (dict(flags=2), INVALID), (dict(flags=4), INVALID),
    (dict(err=FAKE + 2), INVALID), (dict(q_stride=2 ** 39), INVALID),
    (dict(q_out_stride=512), INVALID), (dict(k_out_stride=256), INVALID),  # in place at another stride
])
def test_append_refuses(lib, over, status):
    assert lib.kda_kv_append(ctypes.byref(_append(**over)), None) == status
    assert lib.kda_kv_append(None, None) == INVALID


def test_append_of_nothing_is_accepted(lib):
    assert lib.kda_kv_append(ctypes.byref(_append(tokens=0, slots=None, k=None, v=None, q=None, q_out=None)), None) == 0


def _fwd(**over):
    return _fill(_lib.AttnFwdArgs(), dict(
        B=2, T=8, S=8, N=2, HQ=4, HKV=2, D=64, flags=1, scale=0.1, q_stride=256, k_stride=128, v_stride=128, o_stride=256, q=FAKE, k=FAKE,
        v=FAKE, o=2 * FAKE) | over)


PACKED = dict(B=1, N=3, cu_seqlens=FAKE)
PAGED = dict(block_table=FAKE, seq_lens_k=FAKE, pages=4, page_size=16, table_width=2)


@pytest.mark.parametrize("over,status", [
    (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(S=-1), INVALID), (dict(N=0), INVALID), (dict(N=3), INVALID), (dict(HQ=3), INVALID),
    (dict(D=32), UNSUPPORTED), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=INF), INVALID), (dict(scale=NAN), INVALID),
    (dict(flags=2), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=FAKE + 8), INVALID), (dict(o=None), INVALID),
    (dict(o=FAKE + 4), INVALID), (dict(q_stride=255), INVALID), (dict(k_stride=0), INVALID), (dict(o_stride=-256), INVALID),
    (dict(cu_seqlens=FAKE), INVALID),                                # packed sequences in two rows
    (dict(cu_seqlens_k=FAKE), INVALID),                              # without the queries'
    (PACKED | dict(S=9), INVALID),                                   # other keys, and no array for them
    (PACKED | dict(cu_seqlens_k=FAKE + 1, S=9), INVALID), (PACKED | PAGED | dict(cu_seqlens_k=FAKE), INVALID),
    (PAGED | dict(seq_lens_k=None), INVALID), (dict(seq_lens_k=FAKE), INVALID), (PAGED | dict(page_size=8), UNSUPPORTED),
    (PAGED | dict(table_width=-1), INVALID), (PAGED | dict(table_width=2 ** 25 + 1), UNSUPPORTED), (PAGED | dict(table_width=2 ** 31 - 1), UNSUPPORTED), (PAGED | dict(k=None), INVALID),
    (PAGED | dict(pages=-1), INVALID), (dict(lse=FAKE + 2), INVALID), (dict(err=FAKE + 1), INVALID),
    (dict(T=2 ** 30, S=2 ** 30), INVALID), (dict(B=1, N=1, S=2 ** 29 + 1), UNSUPPORTED), (dict(q_stride=2 ** 39), INVALID), (dict(o=FAKE), INVALID),
])
def test_fwd_refuses(lib, over, status):
    assert lib.kda_attn_fwd(ctypes.byref(_fwd(**over)), None) == status
    assert lib.kda_attn_fwd(None, None) == INVALID


def test_fwd_of_no_queries_is_accepted(lib):
    assert lib.kda_attn_fwd(ctypes.byref(_fwd(T=0, q=None, o=None)), None) == 0


def _step(**over):
    return _fill(_lib.AttnStepArgs(), dict(
        B=3, HQ=4, HKV=2, D=128, pages=9, page_size=32, table_width=2, cache_dtype=BF16, prefix_len=0, prefix_pages=0, scale=0.1,
        q_stride=512, o_stride=512, q=FAKE, k_cache=FAKE, v_cache=FAKE, block_table=FAKE, seq_lens=FAKE, o=2 * FAKE) | over)


PREFIX = dict(prefix_len=33, prefix_pages=2, prefix_table=FAKE)


@pytest.mark.parametrize("over,status", [
    (dict(B=-1), INVALID), (dict(HQ=3), INVALID), (dict(D=256), UNSUPPORTED), (dict(table_width=-1), INVALID), (dict(scale=0.0), INVALID),
    (dict(cache_dtype=FP32), UNSUPPORTED), (dict(cache_dtype=E4M3), INVALID), (dict(k_cache=None), INVALID), (dict(v_cache=FAKE + 2), INVALID),
    (dict(page_size=20), UNSUPPORTED), (dict(q=None), INVALID), (dict(o=FAKE + 8), INVALID), (dict(q_stride=511), INVALID),
    (dict(o_stride=516), INVALID), (dict(block_table=None), INVALID), (dict(block_table=FAKE + 2), INVALID), (dict(seq_lens=None), INVALID),
    (dict(seq_lens=FAKE + 1), INVALID), (dict(table_width=2 ** 27), UNSUPPORTED), (dict(table_width=2 ** 31 - 1), UNSUPPORTED), (dict(prefix_len=-1), INVALID),
    (PREFIX | dict(prefix_len=2 ** 29 + 1, prefix_pages=2 ** 30), UNSUPPORTED), (dict(lse=FAKE + 1), INVALID),
    (dict(o=FAKE), INVALID), (PREFIX, INVALID),                      # no workspace
    (PREFIX | dict(prefix_table=None), INVALID), (PREFIX | dict(prefix_len=65), INVALID), (PREFIX | dict(prefix_table=FAKE + 2), INVALID),
    (dict(table_width=1024), INVALID),                               # few rows on long tables: no workspace
])
def test_step_refuses(lib, over, status):
    assert lib.kda_attn_step(ctypes.byref(_step(**over)), None, 0, None) == status
    assert lib.kda_attn_step(None, None, 0, None) == INVALID


def test_step_workspace(lib):
    size = lambda **over: lib.kda_attn_step_workspace_size(ctypes.byref(_step(**over)))  # noqa: E731
    assert size() == 0 and size(D=256) == 0 and size(B=0, **PREFIX) == 0
    assert size(**PREFIX) >= 3 * 4 * 129 * 4
    e4 = dict(cache_dtype=E4M3, k_scale=FAKE, v_scale=FAKE)
    assert size(**PREFIX, **e4) >= size(**PREFIX) + 2 * 2 * 2 * 32 * 128 * 2   # and the prefix in bf16
    # without a prefix, fewer tokens than KDA_ATTN_LONG_TOKENS never need one
    for B in (1, 2, 3, 50):
        for width in (1, 3, 100, _lib.KDA_ATTN_LONG_TOKENS // 32 - 1):
            for h in (1, 2, 4):
                assert size(B=B, table_width=width, HKV=h) == 0
    need = size(table_width=1024)
    assert need > 0
    assert lib.kda_attn_step(ctypes.byref(_step(table_width=1024)), FAKE, need - 1, None) == INVALID
    assert lib.kda_attn_step(ctypes.byref(_step(table_width=1024)), FAKE + 16, need, None) == INVALID
    assert lib.kda_attn_step(ctypes.byref(_step(B=0)), None, 0, None) == 0
    # largest sizes do not wrap
    assert size(B=2 ** 20, HQ=1024, HKV=8, prefix_len=2 ** 20, prefix_pages=2 ** 15, prefix_table=FAKE, q_stride=2 ** 17, o_stride=2 ** 17) > 2 ** 39


def test_python_calls_refuse_cpu_tensors():
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    kbuild.build()
    for call in (lambda: kda.kda_attn_fwd(z(1, 4, 2, 64), z(1, 4, 2, 64), z(1, 4, 2, 64), scale=1.0),
                 lambda: kda.kda_kv_append(z(4, 2, 64), z(4, 2, 64), i(4), z(1, 2, 16, 64), z(1, 2, 16, 64)),
                 lambda: kda.kda_attn_step(z(4, 2, 64), z(1, 2, 16, 64), z(1, 2, 16, 64), i(4, 1), i(4), scale=1.0)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


# --- the oracle ---

def test_rotation_keeps_lengths_and_depends_on_distance():
    rng = np.random.default_rng(0)
    D, rot = 16, 12
    angle = np.arange(50)[:, None] * 100.0 ** (-np.arange(rot // 2) / 6)
    table = np.concatenate([np.cos(angle), np.sin(angle)], 1)
    q, k = rng.standard_normal((1, 3, D)), rng.standard_normal((1, 3, D))
    for inter in (False, True):
        at = lambda x, p: ao.rotate(x, np.array([p]), table, inter)  # noqa: E731
        assert np.allclose(np.linalg.norm(at(q, 7), axis=-1), np.linalg.norm(q, axis=-1))
        assert np.allclose((at(q, 30) * at(k, 20)).sum(-1), (at(q, 15) * at(k, 5)).sum(-1))
        assert np.array_equal(at(q, 9)[..., rot:], q[..., rot:]) and np.array_equal(at(q, 0), q)
    # by hand: a quarter turn of the first pair
    quarter = np.array([[0.0, 1.0]])
    x = np.array([[[3.0, 5.0, 7.0]]])
    assert np.array_equal(ao.rotate(x, np.array([0]), quarter, False), [[[-5.0, 3.0, 7.0]]])


def test_power_scale_by_hand():
    x = np.array([[0.0, 0.0], [448.0, -1.0], [448.1, 0.0], [1.0, -0.5], [1e-40, 0.0], [-3.5, 2.0]])
    assert ao.power_scale(x).tolist() == [1.0, 1.0, 2.0, 2.0 ** -8, 2.0 ** -110, 2.0 ** -7]


def test_attend_by_hand_and_against_torch():
    # equal scores: the mean of what is seen; one key: its value
    q, k, v = np.zeros((3, 2, 4)), np.ones((3, 1, 4)), np.arange(12.0).reshape(3, 1, 4)
    o, lse, a, top = ao.attend(q, k, v, 0.5, ao.seen_keys(3, 3, True))
    assert np.allclose(o[2, 1], v[:, 0].mean(0)) and np.allclose(o[0, 0], v[0, 0]) and np.allclose(lse[:, 0], np.log([1, 2, 3]))
    assert np.allclose(a, o) and (top == 0).all()
    # fewer keys than queries: the first see none
    assert ao.seen_keys(5, 2, True).tolist() == [0, 0, 0, 1, 2] and ao.seen_keys(2, 5, True).tolist() == [4, 5]
    assert ao.seen_keys(2, 5, False).tolist() == [5, 5]
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((6, 4, 8)), rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8))
    o, lse, _, _ = ao.attend(q, k, v, 0.3, ao.seen_keys(6, 9, True))
    s = torch.einsum("thd,shd->hts", torch.from_numpy(q), torch.from_numpy(k).repeat_interleave(2, 1)) * 0.3
    s = s.masked_fill(torch.arange(9)[None] > torch.arange(6)[:, None] + 3, -INF)
    ref = torch.einsum("hts,shd->thd", s.softmax(-1), torch.from_numpy(v).repeat_interleave(2, 1))
    assert np.allclose(o, ref.numpy()) and np.allclose(lse, torch.logsumexp(s, -1).T.numpy())


@pytest.mark.parametrize("dtype", [BF, E4])
def test_paged_tokens_are_the_sequences(dtype):
    gen = torch.Generator().manual_seed(2)
    ks, vs = ([torch.randn(n, 2, 64, generator=gen).to(BF) for n in (5, 0, 33)] for _ in range(2))
    cache = Cache(gen, ks, vs, 16, dtype)
    for n in range(3):
        for got, x in zip(cache.tokens(n), (ks[n], vs[n])):
            step = 0.0 if dtype == BF else 2.0 ** -4
            assert got.shape == x.shape and np.all(np.abs(got - x.double().numpy()) <= step * np.abs(x.double().numpy()) + 2.0 ** -9 * (dtype == E4))


MISTAKES = {
    "a key too many": lambda q, k, v, s: ao.attend(q, k, v, s, np.minimum(ao.seen_keys(len(q), len(k), True) + 1, len(k))),
    "a key too few": lambda q, k, v, s: ao.attend(q, k, v, s, ao.seen_keys(len(q), len(k), True) - 1),
    "no scale": lambda q, k, v, s: ao.attend(q, k, v, 1.0, ao.seen_keys(len(q), len(k), True)),
    "another head's keys": lambda q, k, v, s: ao.attend(q, k[:, ::-1], v, s, ao.seen_keys(len(q), len(k), True)),
    "another head's values": lambda q, k, v, s: ao.attend(q, k, v[:, ::-1], s, ao.seen_keys(len(q), len(k), True)),
    "a value's neighbour": lambda q, k, v, s: ao.attend(q, k, np.roll(v, 1, 0), s, ao.seen_keys(len(q), len(k), True)),
    "a key's neighbour": lambda q, k, v, s: ao.attend(q, np.roll(k, 1, 0), v, s, ao.seen_keys(len(q), len(k), True)),
    "heads in another order": lambda q, k, v, s: tuple(x[:, ::-1] for x in ao.attend(q, k, v, s, ao.seen_keys(len(q), len(k), True))),
    "no mask": lambda q, k, v, s: ao.attend(q, k, v, s, ao.seen_keys(len(q), len(k), False)),
    "a block left out": lambda q, k, v, s: ao.attend(q, np.where(np.arange(len(k))[:, None, None] // 16 == 1, -k, k), v, s, ao.seen_keys(len(q), len(k), True)),
}


@pytest.mark.parametrize("mistake", MISTAKES)
def test_bounds_find_planted_mistakes(mistake):
    gen = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(n, h, 64, generator=gen).to(BF).double().numpy() for n, h in ((40, 4), (90, 2), (90, 2)))
    refs = ao.attend(q, k, v, 0.125, ao.seen_keys(40, 90, True))
    wrong = MISTAKES[mistake](q, k, v, 0.125)
    attn_cases.check(torch.from_numpy(refs[0]), torch.from_numpy(refs[1]), refs, 90, 64)
    with pytest.raises(AssertionError):
        attn_cases.check(torch.from_numpy(np.ascontiguousarray(wrong[0])).to(BF), None, refs, 90, 64)


def test_bounds_hold_for_a_rounded_computation():
    """The plain computation with bf16 weights, in fp32, is within the bounds."""
    gen = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(n, h, 64, generator=gen).to(BF) for n, h in ((40, 2), (90, 2), (90, 2)))
    refs = ao.attend(*(x.double().numpy() for x in (q, k, v)), 0.125, ao.seen_keys(40, 90, True))
    s = torch.einsum("thd,shd->hts", q.float(), k.float()) * 0.125
    s = s.masked_fill(torch.arange(90)[None] > torch.arange(40)[:, None] + 50, -INF)
    p = (s - s.amax(-1, keepdim=True)).exp()
    o = torch.einsum("hts,shd->thd", p.to(BF).float(), v.float()) / p.sum(-1).T[..., None]
    attn_cases.check(o.to(BF), torch.logsumexp(s, -1).T, refs, 90, 64)
    assert (errors(refs[2], refs[3], 90, 64)[0] < 0.02).all()
