"""ctypes binding of libkda.so (include/kda.h).

Argument marshalling only: every step of the computation runs in the library's
CUDA kernels. PyTorch supplies device memory, the current stream and the output
allocations. There is no CPU or PyTorch fallback: if libkda.so is missing or a
tensor is not on a CUDA device, the call raises.
"""

from __future__ import annotations

import ctypes
import threading
from pathlib import Path

import torch

_LIB_PATH = Path(__file__).resolve().parent / "libkda.so"
_lock = threading.Lock()
_lib = None

KDA_OK = 0
KDA_ERR_INVALID_ARG = 1
KDA_ERR_UNSUPPORTED = 2
KDA_ERR_CUDA = 3
KDA_ERR_TIMEOUT = 4
KDA_ERR_TOO_LARGE = 5
STATUS_NAMES = {0: "KDA_OK", 1: "KDA_ERR_INVALID_ARG", 2: "KDA_ERR_UNSUPPORTED", 3: "KDA_ERR_CUDA",
                4: "KDA_ERR_TIMEOUT", 5: "KDA_ERR_TOO_LARGE"}
KDA_NOALLOC_SCRATCH_BYTES = 16 << 20

KDA_DTYPE_BF16 = 0
KDA_DTYPE_FP32 = 1
KDA_DTYPE_E4M3 = 2
KDA_GATE_NONE, KDA_GATE_G, KDA_GATE_INPUTS, KDA_GATE_HEAD_G = 0, 1, 2, 3
KDA_BETA_VALUES, KDA_BETA_LOGITS = 0, 1
KDA_FLAG_L2NORM_QK = 0x1
KDA_FLAG_DELTA_OFF = 0x2
KDA_FLAG_CHECK_INDICES = 0x4
KDA_NORM_MAX_D = 32768
KDA_ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2, "sigmoid": 3, "relu": 4}
KDA_SCAN_GATES = {"log": 0, "logits": 1}
KDA_SCAN_FLAG_COMPLEMENT = 0x1
KDA_KV_FLAG_INTERLEAVED = 0x1
KDA_ATTN_FLAG_CAUSAL = 0x1
KDA_ATTN_MAX_HEADS = 1024
KDA_ATTN_LONG_TOKENS = 16384
KDA_ATTN_MAX_TOKENS = 1 << 29


class KdaError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)}")
        self.status = status


class ChunkArgs(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32), ("B", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32),
        ("dk", ctypes.c_int32), ("dv", ctypes.c_int32), ("N", ctypes.c_int32),
        ("gate_mode", ctypes.c_int32), ("beta_mode", ctypes.c_int32), ("flags", ctypes.c_uint32),
        ("scale", ctypes.c_float),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("g", ctypes.c_void_p),
        ("a", ctypes.c_void_p), ("A_log", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p),
        ("beta", ctypes.c_void_p), ("h0", ctypes.c_void_p), ("cu_seqlens", ctypes.c_void_p),
        ("o", ctypes.c_void_p), ("hT", ctypes.c_void_p), ("err", ctypes.c_void_p),
        ("h_chunks", ctypes.c_void_p),
    ]


class DecodeArgs(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("H", ctypes.c_int32), ("HV", ctypes.c_int32), ("K", ctypes.c_int32),
        ("V", ctypes.c_int32), ("num_slots", ctypes.c_int32), ("flags", ctypes.c_uint32),
        ("scale", ctypes.c_float),
        ("packed_qkv", ctypes.c_void_p), ("a", ctypes.c_void_p), ("b", ctypes.c_void_p),
        ("A_log", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p), ("state_pool", ctypes.c_void_p),
        ("indices", ctypes.c_void_p), ("o", ctypes.c_void_p), ("err", ctypes.c_void_p),
    ]


class DecodeConvArgs(ctypes.Structure):
    _fields_ = [
        ("dec", DecodeArgs), ("W", ctypes.c_int32), ("conv_state_in", ctypes.c_void_p),
        ("conv_state_out", ctypes.c_void_p), ("conv_weight", ctypes.c_void_p), ("conv_bias", ctypes.c_void_p),
    ]


class RecurrentArgs(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32), ("HV", ctypes.c_int32),
        ("K", ctypes.c_int32), ("V", ctypes.c_int32), ("num_slots", ctypes.c_int32), ("flags", ctypes.c_uint32),
        ("scale", ctypes.c_float),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("a", ctypes.c_void_p),
        ("b", ctypes.c_void_p), ("A_log", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p),
        ("state_pool", ctypes.c_void_p), ("indices", ctypes.c_void_p), ("o", ctypes.c_void_p),
        ("err", ctypes.c_void_p),
    ]


KDA_RECURRENT_MAX_T = 64


class RmsNormArgs(ctypes.Structure):
    _fields_ = [
        ("R", ctypes.c_int64), ("V", ctypes.c_int32), ("eps", ctypes.c_float),
        ("x", ctypes.c_void_p), ("weight", ctypes.c_void_p), ("y", ctypes.c_void_p),
    ]


class AddRmsNormArgs(ctypes.Structure):
    _fields_ = [
        ("R", ctypes.c_int64), ("D", ctypes.c_int32), ("dtype", ctypes.c_int32), ("y_dtype", ctypes.c_int32),
        ("eps", ctypes.c_float), ("x_stride", ctypes.c_int64), ("residual_stride", ctypes.c_int64),
        ("residual_out_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64), ("x", ctypes.c_void_p),
        ("residual", ctypes.c_void_p), ("weight", ctypes.c_void_p), ("residual_out", ctypes.c_void_p),
        ("y", ctypes.c_void_p), ("y_scale", ctypes.c_void_p),
    ]


class LinearArgs(ctypes.Structure):
    _fields_ = [
        ("M", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("y_dtype", ctypes.c_int32), ("activation", ctypes.c_int32), ("ldx", ctypes.c_int64), ("ldw", ctypes.c_int64),
        ("ld_residual", ctypes.c_int64), ("ldy", ctypes.c_int64), ("x", ctypes.c_void_p), ("w", ctypes.c_void_p),
        ("x_scale", ctypes.c_void_p), ("w_scale", ctypes.c_void_p), ("bias", ctypes.c_void_p),
        ("residual", ctypes.c_void_p), ("y", ctypes.c_void_p), ("err", ctypes.c_void_p),
    ]


class ScanArgs(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32), ("gate_dtype", ctypes.c_int32), ("B", ctypes.c_int32), ("T", ctypes.c_int32),
        ("D", ctypes.c_int32), ("N", ctypes.c_int32), ("gate_mode", ctypes.c_int32), ("flags", ctypes.c_uint32),
        ("x_stride", ctypes.c_int64), ("gate_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64),
        ("h_chunks_rows", ctypes.c_int64), ("x", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("h0", ctypes.c_void_p), ("cu_seqlens", ctypes.c_void_p),
        ("y", ctypes.c_void_p), ("hT", ctypes.c_void_p), ("h_chunks", ctypes.c_void_p), ("err", ctypes.c_void_p),
    ]


class ScanBwdArgs(ctypes.Structure):
    _fields_ = [
        ("fwd", ScanArgs), ("dy_stride", ctypes.c_int64), ("dx_stride", ctypes.c_int64),
        ("dgate_stride", ctypes.c_int64), ("dy", ctypes.c_void_p), ("dhT", ctypes.c_void_p), ("dx", ctypes.c_void_p),
        ("dgate", ctypes.c_void_p), ("dh0", ctypes.c_void_p),
    ]


class ScanStepArgs(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32), ("gate_dtype", ctypes.c_int32), ("B", ctypes.c_int32), ("D", ctypes.c_int32),
        ("num_slots", ctypes.c_int32), ("gate_mode", ctypes.c_int32), ("flags", ctypes.c_uint32),
        ("x_stride", ctypes.c_int64), ("gate_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64),
        ("x", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("state_in", ctypes.c_void_p),
        ("state_out", ctypes.c_void_p), ("indices", ctypes.c_void_p), ("y", ctypes.c_void_p), ("err", ctypes.c_void_p),
    ]


class KvAppendArgs(ctypes.Structure):
    _fields_ = [
        ("tokens", ctypes.c_int32), ("HQ", ctypes.c_int32), ("HKV", ctypes.c_int32), ("D", ctypes.c_int32),
        ("pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("cache_dtype", ctypes.c_int32), ("rot", ctypes.c_int32),
        ("max_positions", ctypes.c_int32), ("flags", ctypes.c_uint32), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64), ("q_out_stride", ctypes.c_int64), ("k_out_stride", ctypes.c_int64), ("q", ctypes.c_void_p),
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("slots", ctypes.c_void_p), ("positions", ctypes.c_void_p),
        ("cos_sin", ctypes.c_void_p), ("q_out", ctypes.c_void_p), ("k_out", ctypes.c_void_p), ("k_cache", ctypes.c_void_p),
        ("v_cache", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("err", ctypes.c_void_p),
    ]


class AttnFwdArgs(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("T", ctypes.c_int32), ("S", ctypes.c_int32), ("N", ctypes.c_int32), ("HQ", ctypes.c_int32),
        ("HKV", ctypes.c_int32), ("D", ctypes.c_int32), ("pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
        ("table_width", ctypes.c_int32), ("flags", ctypes.c_uint32), ("scale", ctypes.c_float), ("q_stride", ctypes.c_int64),
        ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64), ("o_stride", ctypes.c_int64), ("q", ctypes.c_void_p),
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("cu_seqlens", ctypes.c_void_p), ("cu_seqlens_k", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p), ("seq_lens_k", ctypes.c_void_p), ("o", ctypes.c_void_p), ("lse", ctypes.c_void_p),
        ("err", ctypes.c_void_p),
    ]


class AttnStepArgs(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("HQ", ctypes.c_int32), ("HKV", ctypes.c_int32), ("D", ctypes.c_int32), ("pages", ctypes.c_int32),
        ("page_size", ctypes.c_int32), ("table_width", ctypes.c_int32), ("cache_dtype", ctypes.c_int32),
        ("prefix_len", ctypes.c_int32), ("prefix_pages", ctypes.c_int32), ("scale", ctypes.c_float), ("q_stride", ctypes.c_int64),
        ("o_stride", ctypes.c_int64), ("q", ctypes.c_void_p), ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
        ("prefix_table", ctypes.c_void_p), ("o", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("err", ctypes.c_void_p),
    ]


class Tcgen05ProbeArgs(ctypes.Structure):
    _fields_ = [
        ("K", ctypes.c_int32), ("N", ctypes.c_int32), ("layout", ctypes.c_int32), ("a_from_tmem", ctypes.c_int32),
        ("reps", ctypes.c_int32), ("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("d", ctypes.c_void_p),
        ("cycles", ctypes.c_void_p), ("err", ctypes.c_void_p),
    ]


EXPORTS = ("kda_chunk_fwd", "kda_chunk_output", "kda_chunk_fwd_noalloc", "kda_chunk_workspace_size", "kda_decode_step",
           "kda_decode_conv_step", "kda_recurrent_step", "kda_head_rmsnorm", "kda_add_rmsnorm", "kda_linear",
           "kda_linear_workspace_size", "kda_scan_fwd",
           "kda_scan_bwd", "kda_scan_step", "kda_kv_append", "kda_attn_fwd", "kda_attn_step", "kda_attn_step_workspace_size",
           "kda_version",
           "kda_selftest_bounded_wait", "kda_selftest_tcgen05")


def lib_path() -> Path:
    return _LIB_PATH


def load() -> ctypes.CDLL:
    """Load libkda.so (once). Raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not _LIB_PATH.exists():
            raise RuntimeError(
                f"{_LIB_PATH} is missing: build the CUDA library first "
                "(python -m kimi_delta_attention_04_gb300.build). There is no fallback path.")
        lib = ctypes.CDLL(str(_LIB_PATH))
        lib.kda_chunk_fwd.restype = ctypes.c_int
        lib.kda_chunk_fwd.argtypes = [ctypes.POINTER(ChunkArgs), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        lib.kda_chunk_output.restype = ctypes.c_int
        lib.kda_chunk_output.argtypes = [ctypes.POINTER(ChunkArgs), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        lib.kda_chunk_workspace_size.restype = ctypes.c_size_t
        lib.kda_chunk_workspace_size.argtypes = [ctypes.POINTER(ChunkArgs)]
        lib.kda_decode_step.restype = ctypes.c_int
        lib.kda_decode_step.argtypes = [ctypes.POINTER(DecodeArgs), ctypes.c_void_p]
        lib.kda_recurrent_step.restype = ctypes.c_int
        lib.kda_recurrent_step.argtypes = [ctypes.POINTER(RecurrentArgs), ctypes.c_void_p]
        lib.kda_decode_conv_step.restype = ctypes.c_int
        lib.kda_decode_conv_step.argtypes = [ctypes.POINTER(DecodeConvArgs), ctypes.c_void_p]
        lib.kda_head_rmsnorm.restype = ctypes.c_int
        lib.kda_head_rmsnorm.argtypes = [ctypes.POINTER(RmsNormArgs), ctypes.c_void_p]
        for name, struct in (("kda_add_rmsnorm", AddRmsNormArgs), ("kda_scan_fwd", ScanArgs), ("kda_scan_bwd", ScanBwdArgs), ("kda_scan_step", ScanStepArgs),
                             ("kda_kv_append", KvAppendArgs), ("kda_attn_fwd", AttnFwdArgs)):
            getattr(lib, name).restype = ctypes.c_int
            getattr(lib, name).argtypes = [ctypes.POINTER(struct), ctypes.c_void_p]
        lib.kda_linear.restype = ctypes.c_int
        lib.kda_linear.argtypes = [ctypes.POINTER(LinearArgs), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        lib.kda_linear_workspace_size.restype = ctypes.c_size_t
        lib.kda_linear_workspace_size.argtypes = [ctypes.POINTER(LinearArgs)]
        lib.kda_attn_step.restype = ctypes.c_int
        lib.kda_attn_step.argtypes = [ctypes.POINTER(AttnStepArgs), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        lib.kda_attn_step_workspace_size.restype = ctypes.c_size_t
        lib.kda_attn_step_workspace_size.argtypes = [ctypes.POINTER(AttnStepArgs)]
        lib.kda_chunk_fwd_noalloc.restype = ctypes.c_int
        lib.kda_chunk_fwd_noalloc.argtypes = [ctypes.POINTER(ChunkArgs), ctypes.c_void_p]
        lib.kda_version.restype = ctypes.c_char_p
        lib.kda_version.argtypes = []
        lib.kda_selftest_bounded_wait.restype = ctypes.c_int
        lib.kda_selftest_bounded_wait.argtypes = [ctypes.c_void_p, ctypes.c_uint64, ctypes.c_void_p]
        lib.kda_selftest_tcgen05.restype = ctypes.c_int
        lib.kda_selftest_tcgen05.argtypes = [ctypes.POINTER(Tcgen05ProbeArgs), ctypes.c_void_p]
        _lib = lib
        return lib


def version() -> str:
    return load().kda_version().decode()


def selftest_bounded_wait(err, limit_ns, stream=None):
    """Run the bounded-wait self-test kernel: it waits on an mbarrier that nothing
    arrives on, gives up after limit_ns and writes KDA_ERR_TIMEOUT to err
    (a device int32 tensor). See include/kda.h."""
    with _on_device(err):
        st = load().kda_selftest_bounded_wait(_ptr(err), ctypes.c_uint64(int(limit_ns)), _stream_ptr(stream, err.device))
    if st != KDA_OK:
        raise KdaError(st, "kda_selftest_bounded_wait")


def selftest_tcgen05(a, b, *, layout=0, a_from_tmem=False, reps=0, err=None, stream=None):
    """One tcgen05 MMA, d [128, N] = a [128, K] @ b[N, K]^T (bf16 in, fp32 out),
    and its timed round trips (see include/kda.h). Returns (d, cycles) with
    cycles an int64 CUDA tensor [7]: summed issue->done and issue->data cycles
    over `reps` round trips, the cycles of a burst of `reps` back-to-back
    groups on one accumulator, reps, the cycles of a burst over independent
    accumulators and their count, and the issuing thread's own cycles for the
    first burst."""
    K, N = int(a.shape[1]), int(b.shape[0])
    if a.shape[0] != 128 or b.shape[1] != K or a.dtype != torch.bfloat16 or b.dtype != torch.bfloat16:
        raise ValueError("expects bf16 a [128, K] and b [N, K]")
    d = torch.empty(128, N, dtype=torch.float32, device=a.device)
    cycles = torch.zeros(7, dtype=torch.int64, device=a.device)
    args = Tcgen05ProbeArgs()
    args.K, args.N, args.layout, args.a_from_tmem, args.reps = K, N, int(layout), int(bool(a_from_tmem)), int(reps)
    args.a, args.b, args.d, args.cycles, args.err = _ptr(a), _ptr(b), _ptr(d), _ptr(cycles), _ptr(err)
    with _on_device(a):
        st = load().kda_selftest_tcgen05(ctypes.byref(args), _stream_ptr(stream, a.device))
    if st != KDA_OK:
        raise KdaError(st, "kda_selftest_tcgen05")
    return d, cycles


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"expected a torch.Tensor, got {type(t).__name__}")
    if not t.is_cuda:
        raise ValueError("libkda works on CUDA tensors only (no CPU fallback)")
    if not t.is_contiguous():
        raise ValueError("libkda needs contiguous tensors")
    return t.data_ptr()


def _stream_ptr(stream, device=None):
    """The stream to enqueue on: the given one, else the current stream of
    `device` (the device of the call's tensors)."""
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _on_device(t):
    """Context in which a C call runs: the device of tensor t is made current,
    so the library's per-device state (kernel attributes, the no-allocation
    scratch address) and its launches refer to the device that holds the data."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("libkda works on CUDA tensors only (no CPU fallback)")
    return torch.cuda.device(t.device)


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return KDA_DTYPE_BF16
    if dt == torch.float32:
        return KDA_DTYPE_FP32
    raise ValueError(f"unsupported input dtype {dt}; use torch.bfloat16 or torch.float32")


def make_chunk_args(q, k, v, *, scale, g=None, a=None, dt_bias=None, A_log=None, beta=None, b=None,
                    h0=None, cu_seqlens=None, l2norm_qk=False, delta=True, o=None, hT=None, err=None, g_head=None,
                    h_chunks=None):
    """Fill the C argument struct from tensors (no allocation, no launch)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if cu_seqlens is not None:
        N = cu_seqlens.numel() - 1
    else:
        N = B
    if g is not None:
        gate_mode = KDA_GATE_G
    elif g_head is not None:
        gate_mode, g = KDA_GATE_HEAD_G, g_head  # passed in the g field
    elif a is not None:
        gate_mode = KDA_GATE_INPUTS
    else:
        gate_mode = KDA_GATE_NONE
    if beta is not None:
        beta_mode, beta_t = KDA_BETA_VALUES, beta
    else:
        beta_mode, beta_t = KDA_BETA_LOGITS, b
    flags = (KDA_FLAG_L2NORM_QK if l2norm_qk else 0) | (0 if delta else KDA_FLAG_DELTA_OFF)
    args = ChunkArgs()
    args.dtype = _dtype_code(q.dtype)
    args.B, args.T, args.H, args.dk, args.dv, args.N = B, T, H, dk, dv, N
    args.gate_mode, args.beta_mode, args.flags = gate_mode, beta_mode, flags
    args.scale = float(scale)
    args.q, args.k, args.v = _ptr(q), _ptr(k), _ptr(v)
    args.g, args.a, args.A_log, args.dt_bias = _ptr(g), _ptr(a), _ptr(A_log), _ptr(dt_bias)
    args.beta = _ptr(beta_t)
    args.h0, args.cu_seqlens = _ptr(h0), _ptr(cu_seqlens)
    args.o, args.hT, args.err = _ptr(o), _ptr(hT), _ptr(err)
    args.h_chunks = _ptr(h_chunks)
    return args


def chunk_workspace_size(args: ChunkArgs) -> int:
    return int(load().kda_chunk_workspace_size(ctypes.byref(args)))


def kda_chunk_fwd(q, k, v, *, scale, g=None, a=None, dt_bias=None, A_log=None, beta=None, b=None,
                  h0=None, cu_seqlens=None, l2norm_qk=False, delta=True, o=None, hT=None,
                  output_final_state=True, workspace=None, err=None, stream=None, g_head=None, h_chunks=None):
    """Chunkwise KDA forward through libkda (see include/kda.h for the contract).

    q, k [B, T, H, dk]; v [B, T, H, dv] (bf16 or fp32, same dtype). The gate is
    g (fp32 [B, T, H, dk]) or gate inputs a (fp32 [B, T, H*dk]) + dt_bias
    (fp32 [H*dk]) + A_log (fp32 [H]), or the Gated DeltaNet per-head gate g_head
    (fp32 [B, T, H]), or none (g = 0). beta [B, T, H] is given
    as values (beta=) or logits (b=). h0 / returned hT are fp32 [N, H, dv, dk].
    h_chunks (fp32 [chunk_count(...), H, dv, dk], bf16 only) receives the state
    entering every 16-token chunk when given.
    Returns (o, hT) with hT None when output_final_state is False.
    """
    lib = load()
    B, T, H, _ = q.shape
    if o is None:
        o = torch.empty(B, T, H, v.shape[-1], dtype=q.dtype, device=q.device)
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else B
    if hT is None and output_final_state:
        hT = torch.empty(N, H, v.shape[-1], q.shape[-1], dtype=torch.float32, device=q.device)
    args = make_chunk_args(q, k, v, scale=scale, g=g, a=a, dt_bias=dt_bias, A_log=A_log, beta=beta, b=b,
                           h0=h0, cu_seqlens=cu_seqlens, l2norm_qk=l2norm_qk, delta=delta, o=o, hT=hT,
                           err=err, g_head=g_head, h_chunks=h_chunks)
    need = int(lib.kda_chunk_workspace_size(ctypes.byref(args)))
    with _on_device(q):
        if need == 0:
            st = lib.kda_chunk_fwd(ctypes.byref(args), None, 0, _stream_ptr(stream, q.device))
            raise KdaError(st if st != KDA_OK else KDA_ERR_INVALID_ARG, "kda_chunk_fwd")
        if workspace is None or workspace.numel() * workspace.element_size() < need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        st = lib.kda_chunk_fwd(ctypes.byref(args), ctypes.c_void_p(_ptr(workspace)), need,
                               _stream_ptr(stream, q.device))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_fwd")
    return o, hT


def kda_chunk_fwd_noalloc(q, k, v, *, scale, g=None, a=None, dt_bias=None, A_log=None, beta=None, b=None,
                          h0=None, cu_seqlens=None, l2norm_qk=False, delta=True, o=None, hT=None,
                          output_final_state=True, err=None, stream=None, g_head=None, h_chunks=None):
    """kda_chunk_fwd on the library's own scratch buffer: the C call allocates
    nothing (for callers that may not allocate device memory; see
    include/kda.h). Outputs o / hT are allocated here with torch unless given.
    Raises KdaError(KDA_ERR_TOO_LARGE) when the request needs more than
    KDA_NOALLOC_SCRATCH_BYTES of scratch."""
    lib = load()
    B, T, H, _ = q.shape
    if o is None:
        o = torch.empty(B, T, H, v.shape[-1], dtype=q.dtype, device=q.device)
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else B
    if hT is None and output_final_state:
        hT = torch.empty(N, H, v.shape[-1], q.shape[-1], dtype=torch.float32, device=q.device)
    args = make_chunk_args(q, k, v, scale=scale, g=g, a=a, dt_bias=dt_bias, A_log=A_log, beta=beta, b=b,
                           h0=h0, cu_seqlens=cu_seqlens, l2norm_qk=l2norm_qk, delta=delta, o=o, hT=hT,
                           err=err, g_head=g_head, h_chunks=h_chunks)
    with _on_device(q):
        st = lib.kda_chunk_fwd_noalloc(ctypes.byref(args), _stream_ptr(stream, q.device))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_fwd_noalloc")
    return o, hT


def make_decode_args(packed_qkv, a, b, A_log, dt_bias, state_pool, indices, *, H, HV, K, V, scale,
                     l2norm_qk=True, o=None, err=None, check_indices=False):
    args = DecodeArgs()
    args.B = packed_qkv.shape[0]
    args.H, args.HV, args.K, args.V = H, HV, K, V
    args.num_slots = state_pool.shape[0]
    args.flags = (KDA_FLAG_L2NORM_QK if l2norm_qk else 0) | (KDA_FLAG_CHECK_INDICES if check_indices else 0)
    args.scale = float(scale)
    args.packed_qkv, args.a, args.b = _ptr(packed_qkv), _ptr(a), _ptr(b)
    args.A_log, args.dt_bias = _ptr(A_log), _ptr(dt_bias)
    args.state_pool, args.indices = _ptr(state_pool), _ptr(indices)
    args.o, args.err = _ptr(o), _ptr(err)
    return args


def kda_decode_step(packed_qkv, a, b, A_log, dt_bias, state_pool, indices, *, H, HV, K, V, scale,
                    l2norm_qk=True, o=None, err=None, stream=None, check_indices=False):
    """Fused T=1 decode through libkda; state_pool is updated in place. Returns o [B, HV, V] bf16.
    check_indices (needs err): a debug check that the valid slot indices are distinct."""
    lib = load()
    if o is None:
        o = torch.empty(packed_qkv.shape[0], HV, V, dtype=torch.bfloat16, device=packed_qkv.device)
    args = make_decode_args(packed_qkv, a, b, A_log, dt_bias, state_pool, indices, H=H, HV=HV, K=K, V=V,
                            scale=scale, l2norm_qk=l2norm_qk, o=o, err=err, check_indices=check_indices)
    with _on_device(packed_qkv):
        st = lib.kda_decode_step(ctypes.byref(args), _stream_ptr(stream, packed_qkv.device))
    if st != KDA_OK:
        raise KdaError(st, "kda_decode_step")
    return o


def make_recurrent_args(q, k, v, a, b, A_log, dt_bias, state_pool, indices, *, scale, l2norm_qk=True,
                        o=None, err=None, check_indices=False):
    args = RecurrentArgs()
    args.B, args.T, args.H, args.K = (int(x) for x in q.shape)
    args.HV, args.V = int(v.shape[2]), int(v.shape[3])
    args.num_slots = state_pool.shape[0]
    args.flags = (KDA_FLAG_L2NORM_QK if l2norm_qk else 0) | (KDA_FLAG_CHECK_INDICES if check_indices else 0)
    args.scale = float(scale)
    args.q, args.k, args.v, args.a, args.b = _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b)
    args.A_log, args.dt_bias = _ptr(A_log), _ptr(dt_bias)
    args.state_pool, args.indices = _ptr(state_pool), _ptr(indices)
    args.o, args.err = _ptr(o), _ptr(err)
    return args


def kda_recurrent_step(q, k, v, a, b, A_log, dt_bias, state_pool, indices, *, scale, l2norm_qk=True,
                       o=None, err=None, stream=None, check_indices=False):
    """T tokens per row (q, k [B, T, H, K]; v [B, T, HV, V]; a [B, T, HV*K]; b [B, T, HV])
    through libkda on the slot pool, updated in place. Returns o [B, T, HV, V] bf16."""
    lib = load()
    if o is None:
        o = torch.empty(q.shape[0], q.shape[1], v.shape[2], v.shape[3], dtype=torch.bfloat16, device=q.device)
    args = make_recurrent_args(q, k, v, a, b, A_log, dt_bias, state_pool, indices, scale=scale,
                               l2norm_qk=l2norm_qk, o=o, err=err, check_indices=check_indices)
    with _on_device(q):
        st = lib.kda_recurrent_step(ctypes.byref(args), _stream_ptr(stream, q.device))
    if st != KDA_OK:
        raise KdaError(st, "kda_recurrent_step")
    return o


def kda_head_rmsnorm(x, weight, *, eps, out=None, stream=None):
    """Per-head RMSNorm over the last axis (V) of x (bf16, any leading shape) with
    an fp32 weight [V]; out may be x itself. Returns out."""
    lib = load()
    if out is None:
        out = torch.empty_like(x)
    args = RmsNormArgs()
    args.V = int(x.shape[-1])
    args.R = int(x.numel() // max(args.V, 1))
    args.eps = float(eps)
    args.x, args.weight, args.y = _ptr(x), _ptr(weight), _ptr(out)
    with _on_device(x):
        st = lib.kda_head_rmsnorm(ctypes.byref(args), _stream_ptr(stream, x.device))
    if st != KDA_OK:
        raise KdaError(st, "kda_head_rmsnorm")
    return out


def kda_decode_conv_step(mixed_qkv, conv_state_in, conv_weight, conv_bias, a, b, A_log, dt_bias, state_pool,
                         indices, *, H, HV, K, V, scale, conv_state_out=None, l2norm_qk=True, o=None, err=None,
                         stream=None, check_indices=False):
    """Decode with its causal conv1d + SiLU in front (see include/kda.h).
    mixed_qkv bf16 [B, C] is the conv input; conv_state_in bf16 [slots, W-1, C];
    conv_weight fp32 [C, W]; conv_bias fp32 [C] or None. conv_state_out defaults
    to conv_state_in (in place, allowed when HV == H). state_pool is updated in
    place. Returns o [B, HV, V] bf16."""
    lib = load()
    if o is None:
        o = torch.empty(mixed_qkv.shape[0], HV, V, dtype=torch.bfloat16, device=mixed_qkv.device)
    args = DecodeConvArgs()
    args.dec = make_decode_args(mixed_qkv, a, b, A_log, dt_bias, state_pool, indices, H=H, HV=HV, K=K, V=V,
                                scale=scale, l2norm_qk=l2norm_qk, o=o, err=err, check_indices=check_indices)
    args.W = int(conv_weight.shape[-1])
    args.conv_state_in = _ptr(conv_state_in)
    args.conv_state_out = _ptr(conv_state_in if conv_state_out is None else conv_state_out)
    args.conv_weight, args.conv_bias = _ptr(conv_weight), _ptr(conv_bias)
    with _on_device(mixed_qkv):
        st = lib.kda_decode_conv_step(ctypes.byref(args), _stream_ptr(stream, mixed_qkv.device))
    if st != KDA_OK:
        raise KdaError(st, "kda_decode_conv_step")
    return o


def chunk_count(B, T, cu_seqlens=None):
    """Number of 16-token chunks of a call: the first dimension of h_chunks."""
    if cu_seqlens is None:
        return B * ((T + 15) // 16)
    cu = cu_seqlens.detach().to("cpu").tolist()
    return sum((cu[i + 1] - cu[i] + 15) // 16 for i in range(len(cu) - 1))


def kda_chunk_output(q, k, v, h_chunks, *, scale, g=None, a=None, dt_bias=None, A_log=None, beta=None, b=None,
                     cu_seqlens=None, l2norm_qk=False, delta=True, o=None, workspace=None, err=None, stream=None,
                     g_head=None):
    """Chunk-parallel output pass: o from the inputs and the per-chunk entering
    states h_chunks that kda_chunk_fwd(h_chunks=...) wrote. Returns o."""
    lib = load()
    B, T, H, _ = q.shape
    if o is None:
        o = torch.empty(B, T, H, v.shape[-1], dtype=q.dtype, device=q.device)
    args = make_chunk_args(q, k, v, scale=scale, g=g, a=a, dt_bias=dt_bias, A_log=A_log, beta=beta, b=b,
                           cu_seqlens=cu_seqlens, l2norm_qk=l2norm_qk, delta=delta, o=o, err=err, g_head=g_head,
                           h_chunks=h_chunks)
    need = int(lib.kda_chunk_workspace_size(ctypes.byref(args)))
    with _on_device(q):
        if need == 0:
            st = lib.kda_chunk_output(ctypes.byref(args), None, 0, _stream_ptr(stream, q.device))
            raise KdaError(st if st != KDA_OK else KDA_ERR_INVALID_ARG, "kda_chunk_output")
        if workspace is None or workspace.numel() * workspace.element_size() < need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        st = lib.kda_chunk_output(ctypes.byref(args), ctypes.c_void_p(_ptr(workspace)), need,
                                  _stream_ptr(stream, q.device))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_output")
    return o


# --- the layer around the attention: norm, projections, gated recurrence ---


_DTYPE_CODES = {torch.bfloat16: KDA_DTYPE_BF16, torch.float32: KDA_DTYPE_FP32, torch.float8_e4m3fn: KDA_DTYPE_E4M3}


# These calls are short next to a launch (a decode step's norm takes 3 us), so the
# marshalling below avoids what costs microseconds: device contexts where the
# device is current already, stream objects, tuples of shapes.

def _code(dt):
    code = _DTYPE_CODES.get(dt)
    if code is None:
        raise ValueError(f"unsupported dtype {dt}; use torch.bfloat16, torch.float32 or torch.float8_e4m3fn")
    return code


def _device_of(x):
    """Device index of a call's first tensor."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"expected a torch.Tensor, got {type(x).__name__}")
    if not x.is_cuda:
        raise ValueError("libkda works on CUDA tensors only (no CPU fallback)")
    return x.get_device()


_I32_MAX = 2 ** 31 - 1


def _past_32_bits(**sizes):
    """Refuses what the C structs' 32-bit counts would be assigned cut short."""
    raise ValueError("sizes must fit 32 bits: " + ", ".join(f"{k} = {v}" for k, v in sizes.items() if v > _I32_MAX))


def _refuse(t, name, dev, dtype, shape):
    """Says what is wrong with a tensor that is not as expected (_rows and _vec ask)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, expected cuda:{dev} (libkda works on CUDA tensors only)")
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def _rows(t, name, dev, dtype, shape):
    """(pointer, row stride) of a tensor taken as rows of its last axis: that axis
    contiguous, the leading axes evenly spaced. None gives (None, 0)."""
    if t is None:
        return None, 0
    # (a CPU tensor's device index is -1)
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or t.dtype != dtype or t.shape != shape:
        _refuse(t, name, dev, dtype, shape)
    if t.is_contiguous():
        return t.data_ptr(), shape[-1]
    return _spaced_rows(t, name)


def _spaced_rows(t, name):
    size = t.shape
    if t.numel() == 0:
        return t.data_ptr(), size[-1]
    if size[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    step, span = None, None
    for n, stride in zip(reversed(size[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if step is None:
            step = stride
        elif stride != span:
            raise ValueError(f"{name}: the leading axes must be evenly spaced rows")
        span = stride * n
    return t.data_ptr(), size[-1] if step is None else step


def _vec(t, name, dev, shape, dtype=torch.float32):
    """Pointer of a contiguous tensor of the given shape, or None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or t.dtype != dtype or t.shape != shape:
        _refuse(t, name, dev, dtype, shape)
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


def _err_word(err, dev):
    if err is None:
        return None
    if not isinstance(err, torch.Tensor) or err.get_device() != dev or err.dtype != torch.int32 or err.numel() < 1:
        _refuse(err, "err", dev, torch.int32, (1,))
    return err.data_ptr()


def _empty(x, stream, shape, dtype):
    """An output on x's device, allocated on the stream that writes it, so that the
    caching allocator does not hand its memory on too early. (A device object is
    1.5 us cheaper than its index.)"""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=x.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=x.device)


def _output(t, name, x, stream, shape, dtype):
    """(tensor, pointer, row stride) of an output: the caller's, checked, or a new one."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=x.device) if stream is None else _empty(x, stream, shape, dtype)
        return t, t.data_ptr(), shape[-1]
    return t, *_rows(t, name, x.get_device(), dtype, shape)


def _state_output(t, name, x, stream, shape, wanted):
    """(tensor or None, pointer) of an fp32 state output."""
    if t is not None:
        return t, _vec(t, name, x.get_device(), shape)
    if not wanted:
        return None, None
    t = _empty(x, stream, shape, torch.float32)
    return t, t.data_ptr()


def _call(fn, args, dev, stream, *workspace):
    handle = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if torch.cuda.current_device() == dev:
        st = fn(args, *workspace, handle)
    else:
        with torch.cuda.device(dev):
            st = fn(args, *workspace, handle)
    if st != KDA_OK:
        raise KdaError(st, fn.__name__)


def kda_add_rmsnorm(x, weight, *, eps, residual=None, residual_out=None, out=None, out_scale=None, out_dtype=None,
                    stream=None):
    """r = x + residual; y = r / sqrt(mean(r^2) + eps) * weight over the last axis.

    x, residual (optional): bf16 or fp32 [..., D], rows evenly spaced; weight fp32
    [D]. out_dtype (default x.dtype) is torch.bfloat16, torch.float32 or
    torch.float8_e4m3fn; the last stores y / scale with one fp32 scale per row
    (largest |y| / 448). residual_out may be residual or x (in place).
    Returns (y, scale or None, residual_out or None): residual_out is made when
    there is a residual, or when it is given."""
    lib = _lib or load()
    dev = _device_of(x)
    shape, dtype = x.shape, x.dtype
    lead, D = shape[:-1], shape[-1]
    if D > _I32_MAX:
        _past_32_bits(D=D)
    if out is not None and out_dtype is not None and out.dtype != out_dtype:
        raise ValueError(f"out: expected {out_dtype}, got {out.dtype}")
    out_dtype = out.dtype if out is not None else (out_dtype or x.dtype)
    q8 = out_dtype == torch.float8_e4m3fn
    if out_scale is not None and not q8:
        raise ValueError("out_scale goes with an 8-bit output")
    args = AddRmsNormArgs()
    args.R, args.D = x.numel() // max(D, 1), D
    args.dtype, args.y_dtype, args.eps = _code(dtype), _code(out_dtype), eps
    args.x, args.x_stride = _rows(x, "x", dev, dtype, shape)
    args.weight = _vec(weight, "weight", dev, (D,))
    if residual is not None or residual_out is not None:
        args.residual, args.residual_stride = _rows(residual, "residual", dev, dtype, shape)
        residual_out, args.residual_out, args.residual_out_stride = _output(residual_out, "residual_out", x, stream, shape, dtype)
    out, args.y, args.y_stride = _output(out, "out", x, stream, shape, out_dtype)
    out_scale, args.y_scale = _state_output(out_scale, "out_scale", x, stream, lead, q8)
    _call(lib.kda_add_rmsnorm, args, dev, stream)
    return out, out_scale, residual_out


def kda_linear(x, w, *, bias=None, activation="none", residual=None, x_scale=None, w_scale=None, out=None,
               out_dtype=None, workspace=None, err=None, stream=None):
    """y = act((x w^T) * x_scale * w_scale + bias) + residual.

    x [..., K] and w [N, K], both bf16, or both torch.float8_e4m3fn with fp32
    scales x_scale [...] (one per row) and w_scale [N]. bias fp32 [N]; activation
    "none", "silu", "gelu", "sigmoid" or "relu"; residual [..., N] in the output's
    dtype, bf16 (default) or fp32; out may be residual. Rows of x or w that do not
    start on 16-byte boundaries are copied into workspace (a CUDA uint8 tensor of
    kda_linear_workspace_size bytes, made here unless given). Returns y [..., N]."""
    if activation not in KDA_ACTIVATIONS:
        raise ValueError(f"activation: expected one of {sorted(KDA_ACTIVATIONS)}, got {activation!r}")
    lib = _lib or load()
    dev = _device_of(x)
    dtype, lead, K = x.dtype, x.shape[:-1], x.shape[-1]
    if w.dim() != 2:
        raise ValueError("w: expected [N, K]")
    M, N = x.numel() // max(K, 1), w.shape[0]
    if M > _I32_MAX or N > _I32_MAX or K > _I32_MAX:
        _past_32_bits(M=M, N=N, K=K)
    shape = lead + (N,)
    if out is not None and out_dtype is not None and out.dtype != out_dtype:
        raise ValueError(f"out: expected {out_dtype}, got {out.dtype}")
    out_dtype = out.dtype if out is not None else (out_dtype or torch.bfloat16)
    args = LinearArgs()
    args.x, args.ldx = _rows(x, "x", dev, dtype, x.shape)
    args.w, args.ldw = _rows(w, "w", dev, dtype, (N, K))
    args.M, args.N, args.K = M, N, K
    args.dtype, args.y_dtype = _code(dtype), _code(out_dtype)
    args.activation = KDA_ACTIVATIONS[activation]
    args.x_scale, args.w_scale = _vec(x_scale, "x_scale", dev, lead), _vec(w_scale, "w_scale", dev, (N,))
    args.bias, args.err = _vec(bias, "bias", dev, (N,)), _err_word(err, dev)
    args.residual, args.ld_residual = _rows(residual, "residual", dev, out_dtype, shape)
    out, args.y, args.ldy = _output(out, "out", x, stream, shape, out_dtype)
    if ((args.x or 0) | (args.w or 0) | args.ldx * x.element_size() | args.ldw * x.element_size()) % 16 == 0:
        _call(lib.kda_linear, args, dev, stream, None, 0)
        return out
    need = lib.kda_linear_workspace_size(args)
    if need and workspace is None:
        workspace = _empty(x, stream, (need,), torch.uint8)
    elif need:
        _vec(workspace, "workspace", dev, (max(need, workspace.numel()),), torch.uint8)
    _call(lib.kda_linear, args, dev, stream, workspace.data_ptr() if need else None, need)
    return out


def _scan_args(x, gate, gate_mode, complement, h0, cu_seqlens, h_chunks, err, dev):
    if len(x.shape) != 3:
        raise ValueError("x: expected [B, T, D]")
    B, T, D = shape = x.shape
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1
    if B > _I32_MAX or T > _I32_MAX or D > _I32_MAX or N > _I32_MAX:
        _past_32_bits(B=B, T=T, D=D, N=N)
    args = ScanArgs()
    args.x, args.x_stride = _rows(x, "x", dev, x.dtype, shape)
    args.gate, args.gate_stride = _rows(gate, "gate", dev, gate.dtype, shape)
    args.dtype, args.gate_dtype = _code(x.dtype), _code(gate.dtype)
    args.B, args.T, args.D, args.N = B, T, D, N
    args.gate_mode, args.flags = KDA_SCAN_GATES[gate_mode], KDA_SCAN_FLAG_COMPLEMENT if complement else 0
    args.h0 = _vec(h0, "h0", dev, (N, D))
    args.cu_seqlens = _vec(cu_seqlens, "cu_seqlens", dev, (N + 1,), torch.int32)
    if h_chunks is not None:
        if h_chunks.dim() != 2:
            raise ValueError(f"h_chunks: expected [chunks, {D}]")
        args.h_chunks = _vec(h_chunks, "h_chunks", dev, (h_chunks.shape[0], D))
        args.h_chunks_rows = h_chunks.shape[0]
    args.err = _err_word(err, dev)
    return args


def kda_scan_fwd(x, gate, *, gate_mode="log", complement=False, h0=None, cu_seqlens=None, y=None, hT=None,
                 h_chunks=None, output_final_state=True, err=None, stream=None):
    """Gated linear recurrence h_t = a_t h_{t-1} + u_t over x [B, T, D], y_t = h_t.

    a = exp(gate) (gate_mode "log") or sigmoid(gate) ("logits"); u = x, or
    (1 - a) x with complement. x bf16 with a bf16 or fp32 gate, or both fp32; rows
    evenly spaced (views of one packed projection will do). h0, hT fp32 [N, D];
    cu_seqlens as for kda_chunk_fwd. h_chunks (fp32 [chunk_count(B, T,
    cu_seqlens), D]) receives the state entering every 16-token chunk, which
    kda_scan_bwd reads. Returns (y, hT), hT None when output_final_state is False."""
    if gate_mode not in KDA_SCAN_GATES:
        raise ValueError(f"gate_mode: expected one of {sorted(KDA_SCAN_GATES)}, got {gate_mode!r}")
    lib = _lib or load()
    dev = _device_of(x)
    args = _scan_args(x, gate, gate_mode, complement, h0, cu_seqlens, h_chunks, err, dev)
    y, args.y, args.y_stride = _output(y, "y", x, stream, x.shape, x.dtype)
    hT, args.hT = _state_output(hT, "hT", x, stream, (args.N, args.D), output_final_state)
    _call(lib.kda_scan_fwd, args, dev, stream)
    return y, hT


def kda_scan_bwd(x, gate, dy, h_chunks, *, gate_mode="log", complement=False, dhT=None, cu_seqlens=None, dx=None,
                 dgate=None, dh0=None, output_dh0=True, err=None, stream=None):
    """Gradients of kda_scan_fwd from dy (of y) and dhT (of hT; None for zero), with
    the h_chunks that the forward wrote. Returns (dx, dgate, dh0), dh0 None when
    output_dh0 is False. dx may be dy or x, and dgate may be gate."""
    if gate_mode not in KDA_SCAN_GATES:
        raise ValueError(f"gate_mode: expected one of {sorted(KDA_SCAN_GATES)}, got {gate_mode!r}")
    lib = _lib or load()
    dev = _device_of(x)
    shape, dtype = x.shape, x.dtype
    args = ScanBwdArgs()
    args.fwd = _scan_args(x, gate, gate_mode, complement, None, cu_seqlens, h_chunks, err, dev)
    N, D = args.fwd.N, args.fwd.D
    args.dy, args.dy_stride = _rows(dy, "dy", dev, dtype, shape)
    args.dhT = _vec(dhT, "dhT", dev, (N, D))
    dx, args.dx, args.dx_stride = _output(dx, "dx", x, stream, shape, dtype)
    dgate, args.dgate, args.dgate_stride = _output(dgate, "dgate", x, stream, shape, gate.dtype)
    dh0, args.dh0 = _state_output(dh0, "dh0", x, stream, (N, D), output_dh0)
    _call(lib.kda_scan_bwd, args, dev, stream)
    return dx, dgate, dh0


def kda_scan_step(x, gate, state_pool, indices, *, gate_mode="log", complement=False, state_out=None, y=None,
                  err=None, stream=None, check_indices=False):
    """One token of the recurrence for each row of x [B, D] on a pool of states
    (fp32 [slots, D]): row b uses slot indices[b] (int32; negative = padding, y = 0).
    state_out defaults to state_pool (in place); only the valid rows' slots are
    written. check_indices (needs err): a debug check that the valid slots are
    distinct. Returns y [B, D]."""
    if gate_mode not in KDA_SCAN_GATES:
        raise ValueError(f"gate_mode: expected one of {sorted(KDA_SCAN_GATES)}, got {gate_mode!r}")
    lib = _lib or load()
    dev = _device_of(x)
    if len(x.shape) != 2:
        raise ValueError("x: expected [B, D]")
    B, D = shape = x.shape
    slots = state_pool.shape[0]
    if B > _I32_MAX or D > _I32_MAX or slots > _I32_MAX:
        _past_32_bits(B=B, D=D, slots=slots)
    args = ScanStepArgs()
    args.dtype, args.gate_dtype, args.B, args.D = _code(x.dtype), _code(gate.dtype), B, D
    args.num_slots, args.gate_mode = slots, KDA_SCAN_GATES[gate_mode]
    args.flags = (KDA_SCAN_FLAG_COMPLEMENT if complement else 0) | (KDA_FLAG_CHECK_INDICES if check_indices else 0)
    args.x, args.x_stride = _rows(x, "x", dev, x.dtype, shape)
    args.gate, args.gate_stride = _rows(gate, "gate", dev, gate.dtype, shape)
    y, args.y, args.y_stride = _output(y, "y", x, stream, shape, x.dtype)
    args.state_in = _vec(state_pool, "state_pool", dev, (slots, D))
    args.state_out = args.state_in if state_out is None else _vec(state_out, "state_out", dev, (slots, D))
    args.indices, args.err = _vec(indices, "indices", dev, (B,), torch.int32), _err_word(err, dev)
    _call(lib.kda_scan_step, args, dev, stream)
    return y


# --- softmax attention with a paged cache ---


def _head_rows(t, name, dev, dtype, shape):
    """(pointer, row stride) of a tensor [..., heads, D] taken as rows of a token's heads:
    the last two axes contiguous, the leading ones evenly spaced. None gives (None, 0)."""
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or t.dtype != dtype or t.shape != shape:
        _refuse(t, name, dev, dtype, shape)
    st, H, D = t.stride(), shape[-2], shape[-1]
    n = len(st)
    # [tokens, heads, D] and [1, tokens, heads, D], whole or as a view of a wider row
    if st[-1] == 1 and st[-2] == D and (n == 3 or (n == 4 and shape[0] == 1)):
        return t.data_ptr(), st[-3] if shape[-3] > 1 else H * D
    if t.is_contiguous():
        return t.data_ptr(), H * D
    if t.numel() == 0:
        return t.data_ptr(), H * D
    if (D > 1 and st[-1] != 1) or (H > 1 and st[-2] != D):
        raise ValueError(f"{name}: the last two axes must be contiguous")
    ptr, step = _spaced_rows(t.select(-2, 0), name)
    return ptr, step if t.numel() > H * D else H * D


def _head_output(t, name, x, stream, shape):
    """(tensor, pointer, row stride) of a bf16 output [..., heads, D]: the caller's, checked, or a new one."""
    if t is None:
        t = torch.empty(shape, dtype=torch.bfloat16, device=x.device) if stream is None else _empty(x, stream, shape, torch.bfloat16)
        return t, t.data_ptr(), shape[-2] * shape[-1]
    return t, *_head_rows(t, name, x.get_device(), torch.bfloat16, shape)


def _cache(args, k_cache, v_cache, dev):
    """Checks a cache [pages, HKV, page_size, D] and fills the struct's part on it. Returns its shape."""
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache: expected [pages, HKV, page_size, D]")
    shape = k_cache.shape
    if max(shape) > _I32_MAX:
        _past_32_bits(**dict(zip(("pages", "HKV", "page_size", "D"), shape)))
    args.pages, args.page_size = shape[0], shape[2]
    return shape, _vec(k_cache, "k_cache", dev, shape, k_cache.dtype), _vec(v_cache, "v_cache", dev, shape, k_cache.dtype)


def _cache_scales(args, k_scale, v_scale, dtype, shape, dev):
    if (dtype == torch.float8_e4m3fn) != (k_scale is not None) or (k_scale is None) != (v_scale is None):
        raise ValueError("k_scale and v_scale go with an 8-bit cache")
    args.cache_dtype = _code(dtype)
    args.k_scale, args.v_scale = _vec(k_scale, "k_scale", dev, shape[:3]), _vec(v_scale, "v_scale", dev, shape[:3])


def kda_kv_append(k, v, slots, k_cache, v_cache, *, q=None, positions=None, cos_sin=None, interleaved=False, q_out=None,
                  k_out=None, k_scale=None, v_scale=None, err=None, stream=None, check_indices=False):
    """Rotary positions, and the append of keys and values to a paged cache.

    k, v bf16 [..., HKV, D] and q (optional) bf16 [..., HQ, D], a token a leading index
    (views of one packed projection will do); slots int32 [...] = page * page_size +
    offset, negative for padding. k_cache, v_cache [pages, HKV, page_size, D], bf16 or
    torch.float8_e4m3fn with k_scale, v_scale fp32 [pages, HKV, page_size], are updated in
    place. positions int32 [...] and cos_sin fp32 [positions, rot] (cosines, then sines)
    turn the first rot channels of q and k, in halves or in neighbouring pairs
    (interleaved). q_out may be q; k_out, filled when given, may be k. check_indices (needs
    err): a debug check that the valid slots are distinct. Returns (q_out or None, k_out),
    without gradients."""
    lib = _lib or load()
    dev = _device_of(k)
    if k.dim() < 2:
        raise ValueError("k: expected [..., HKV, D]")
    args = KvAppendArgs()
    cache, args.k_cache, args.v_cache = _cache(args, k_cache, v_cache, dev)
    _cache_scales(args, k_scale, v_scale, k_cache.dtype, cache, dev)
    lead, HKV, D = k.shape[:-2], cache[1], cache[3]
    shape = lead + (HKV, D)
    tokens = lead.numel()
    if tokens > _I32_MAX:
        _past_32_bits(tokens=tokens)
    args.tokens, args.HKV, args.D = tokens, HKV, D
    args.flags = (KDA_KV_FLAG_INTERLEAVED if interleaved else 0) | (KDA_FLAG_CHECK_INDICES if check_indices else 0)
    args.k, args.k_stride = _head_rows(k, "k", dev, torch.bfloat16, shape)
    args.v, args.v_stride = _head_rows(v, "v", dev, torch.bfloat16, shape)
    args.slots, args.err = _vec(slots, "slots", dev, lead, torch.int32), _err_word(err, dev)
    if (positions is None) != (cos_sin is None):
        raise ValueError("positions and cos_sin go together")
    if cos_sin is not None:
        if cos_sin.dim() != 2 or cos_sin.shape[0] > _I32_MAX:
            raise ValueError("cos_sin: expected [positions, rot]")
        args.max_positions, args.rot = cos_sin.shape
        args.cos_sin = _vec(cos_sin, "cos_sin", dev, cos_sin.shape)
        if args.rot:
            args.positions = _vec(positions, "positions", dev, lead, torch.int32)
        else:
            args.cos_sin = None
    if q is not None:
        if q.dim() < 2:
            raise ValueError("q: expected [..., HQ, D]")
        qshape = lead + (q.shape[-2], D)
        args.HQ = q.shape[-2]
        args.q, args.q_stride = _head_rows(q, "q", dev, torch.bfloat16, qshape)
        q_out, args.q_out, args.q_out_stride = _head_output(q_out, "q_out", k, stream, qshape)
    elif q_out is not None:
        raise ValueError("q_out goes with q")
    args.k_out, args.k_out_stride = _head_rows(k_out, "k_out", dev, torch.bfloat16, shape)
    _call(lib.kda_kv_append, args, dev, stream)
    return q_out, k_out


def kda_attn_fwd(q, k, v, *, scale, causal=True, cu_seqlens=None, cu_seqlens_k=None, block_table=None, seq_lens_k=None,
                 o=None, lse=None, err=None, stream=None):
    """Softmax attention over whole prompts: q bf16 [B, T, HQ, D] on keys and values bf16
    [B, S, HKV, D] (HQ a multiple of HKV, D 64 or 128), or on a bf16 cache [pages, HKV,
    page_size, D] with block_table int32 [N, width] and seq_lens_k int32 [N].

    cu_seqlens int32 [N + 1] packs N sequences along T (B = 1), cu_seqlens_k their keys
    (default: the same). causal: query i of a sequence of T sees keys up to i + S - T.
    lse (fp32 [B, T, HQ]) receives the logarithm of the sums when given. Rows of o and
    lse behind the last sequence are left as they were. Returns o [B, T, HQ, D], without
    gradients."""
    lib = _lib or load()
    dev = _device_of(q)
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k: expected [B, T, heads, D]")
    B, T, HQ, D = shape = q.shape
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1
    args = AttnFwdArgs()
    if block_table is not None:
        if block_table.dim() != 2:
            raise ValueError("block_table: expected [N, width]")
        kshape, args.k, args.v = _cache(args, k, v, dev)
        if k.dtype != torch.bfloat16:
            raise ValueError(f"k: expected {torch.bfloat16}, got {k.dtype}")
        HKV, S, width = kshape[1], 0, block_table.shape[1]
        if kshape[3] != D:
            raise ValueError(f"k: expected heads of {D}, got {kshape[3]}")
        if width > _I32_MAX:
            _past_32_bits(width=width)
        args.table_width = width
        args.block_table = _vec(block_table, "block_table", dev, (N, width), torch.int32)
        args.seq_lens_k = _vec(seq_lens_k, "seq_lens_k", dev, (N,), torch.int32)
        if seq_lens_k is None:
            raise ValueError("seq_lens_k goes with block_table")
    else:
        if seq_lens_k is not None:
            raise ValueError("seq_lens_k goes with block_table")
        S, HKV = k.shape[1], k.shape[2]
        args.k, args.k_stride = _head_rows(k, "k", dev, torch.bfloat16, (B, S, HKV, D))
        args.v, args.v_stride = _head_rows(v, "v", dev, torch.bfloat16, (B, S, HKV, D))
    if max(B, T, S, N, HQ, HKV) > _I32_MAX:
        _past_32_bits(B=B, T=T, S=S, N=N, HQ=HQ, HKV=HKV)
    args.B, args.T, args.S, args.N, args.HQ, args.HKV, args.D = B, T, S, N, HQ, HKV, D
    args.flags, args.scale = KDA_ATTN_FLAG_CAUSAL if causal else 0, scale
    args.q, args.q_stride = _head_rows(q, "q", dev, torch.bfloat16, shape)
    args.cu_seqlens = _vec(cu_seqlens, "cu_seqlens", dev, (N + 1,), torch.int32)
    args.cu_seqlens_k = _vec(cu_seqlens_k, "cu_seqlens_k", dev, (N + 1,), torch.int32)
    o, args.o, args.o_stride = _head_output(o, "o", q, stream, shape)
    args.lse, args.err = _vec(lse, "lse", dev, (B, T, HQ)), _err_word(err, dev)
    _call(lib.kda_attn_fwd, args, dev, stream)
    return o


def kda_attn_step(q, k_cache, v_cache, block_table, seq_lens, *, scale, k_scale=None, v_scale=None, prefix_table=None,
                  prefix_len=0, o=None, lse=None, workspace=None, err=None, stream=None):
    """One token of each row, q bf16 [B, HQ, D], against a paged cache [pages, HKV,
    page_size, D] (bf16, or torch.float8_e4m3fn with k_scale, v_scale fp32 [pages, HKV,
    page_size]): row b attends to the first prefix_len tokens on the pages of prefix_table
    (int32, shared by all rows and read once for them) and to its own seq_lens[b] tokens
    (int32; negative = padding, o = 0) on the pages of block_table[b] (int32 [B, width]).

    lse (fp32 [B, HQ]) receives the logarithm of the sums when given. With a prefix, or a
    table for KDA_ATTN_LONG_TOKENS tokens or more, workspace (a CUDA uint8 tensor of
    kda_attn_step_workspace_size bytes) is made here unless given. How rows are split goes by
    the table's width: one much wider than the rows costs time. Returns o [B, HQ, D],
    without gradients."""
    lib = _lib or load()
    dev = _device_of(q)
    if q.dim() != 3 or block_table.dim() != 2:
        raise ValueError("q: expected [B, HQ, D]; block_table: expected [B, width]")
    B, HQ, D = shape = q.shape
    args = AttnStepArgs()
    cache, args.k_cache, args.v_cache = _cache(args, k_cache, v_cache, dev)
    if cache[3] != D:
        raise ValueError(f"k_cache: expected heads of {D}, got {cache[3]}")
    _cache_scales(args, k_scale, v_scale, k_cache.dtype, cache, dev)
    width = block_table.shape[1]
    pages = 0 if prefix_table is None else prefix_table.numel()
    if max(B, HQ, width, pages, prefix_len) > _I32_MAX:
        _past_32_bits(B=B, HQ=HQ, width=width, prefix_pages=pages, prefix_len=prefix_len)
    if prefix_len > 0 and pages * cache[2] < prefix_len:
        raise ValueError(f"prefix_table: {pages} pages of {cache[2]} for {prefix_len} tokens")
    args.B, args.HQ, args.HKV, args.D, args.table_width = B, HQ, cache[1], D, width
    args.prefix_len, args.prefix_pages, args.scale = prefix_len, pages, scale
    args.q, args.q_stride = _head_rows(q, "q", dev, torch.bfloat16, shape)
    args.block_table = _vec(block_table, "block_table", dev, (B, width), torch.int32)
    args.seq_lens = _vec(seq_lens, "seq_lens", dev, (B,), torch.int32)
    args.prefix_table = _vec(prefix_table, "prefix_table", dev, (pages,), torch.int32)
    o, args.o, args.o_stride = _head_output(o, "o", q, stream, shape)
    args.lse, args.err = _vec(lse, "lse", dev, (B, HQ)), _err_word(err, dev)
    if prefix_len <= 0 and width * cache[2] < KDA_ATTN_LONG_TOKENS:
        _call(lib.kda_attn_step, args, dev, stream, None, 0)
        return o
    need = lib.kda_attn_step_workspace_size(args)
    if need and workspace is None:
        workspace = _empty(q, stream, (need,), torch.uint8)
    elif need:
        _vec(workspace, "workspace", dev, (max(need, workspace.numel()),), torch.uint8)
    _call(lib.kda_attn_step, args, dev, stream, workspace.data_ptr() if need else None, need)
    return o
