// Host side of the layer operators of include/kda.h (add + RMS norm, projection,
// gated recurrence): argument validation and dispatch. No allocation, no
// synchronisation.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/kda.h"
#include "kda_internal.h"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool is_float(int32_t dt) { return dt == KDA_DTYPE_BF16 || dt == KDA_DTYPE_FP32; }
bool is_dtype(int32_t dt) { return is_float(dt) || dt == KDA_DTYPE_E4M3; }
size_t bytes_of(int32_t dt) { return dt == KDA_DTYPE_BF16 ? 2 : dt == KDA_DTYPE_FP32 ? 4 : 1; }

// A [rows, cols] matrix the call needs: present, aligned to its element, and its
// rows neither overlapping (one row has no stride to get wrong) nor reaching
// past what 64-bit byte offsets hold.
bool matrix_ok(const void* p, int32_t dt, int64_t rows, int64_t cols, int64_t stride) {
  if (p == nullptr || !aligned(p, bytes_of(dt))) return false;
  if (rows > 1 && stride < cols) return false;
  return stride >= 0 && stride <= (INT64_C(1) << 40) && rows <= (INT64_C(1) << 52) / (stride > cols ? stride : cols);
}

kda_status done(cudaError_t e) {
  // a device that cannot run the launch's shape is a refusal, not a failure
  return e == cudaSuccess ? KDA_OK : e == cudaErrorNotSupported ? KDA_ERR_UNSUPPORTED : KDA_ERR_CUDA;
}

kda_status check_scan_common(int32_t dtype, int32_t gate_dtype, int32_t gate_mode) {
  if (!is_dtype(dtype) || !is_dtype(gate_dtype)) return KDA_ERR_INVALID_ARG;
  if (gate_mode != KDA_SCAN_LOG_DECAY && gate_mode != KDA_SCAN_LOGITS) return KDA_ERR_INVALID_ARG;
  if (!is_float(dtype) || !is_float(gate_dtype)) return KDA_ERR_UNSUPPORTED;
  if (dtype == KDA_DTYPE_FP32 && gate_dtype != KDA_DTYPE_FP32) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

kda_status check_scan(const kda_scan_args* a, bool forward) {
  if (a->B < 1 || a->T < 0 || a->D < 1 || a->N < 1) return KDA_ERR_INVALID_ARG;
  if (a->flags & ~KDA_SCAN_FLAG_COMPLEMENT) return KDA_ERR_INVALID_ARG;
  const kda_status st = check_scan_common(a->dtype, a->gate_dtype, a->gate_mode);
  if (st != KDA_OK) return st;
  if (a->cu_seqlens == nullptr) {
    if (a->N != a->B) return KDA_ERR_INVALID_ARG;
  } else if (a->B != 1 || !aligned(a->cu_seqlens, 4)) {
    return KDA_ERR_INVALID_ARG;
  }
  const int64_t tokens = static_cast<int64_t>(a->B) * a->T;
  if (tokens > INT32_MAX / 2) return KDA_ERR_INVALID_ARG;
  if (tokens > 0) {
    if (!matrix_ok(a->x, a->dtype, tokens, a->D, a->x_stride)) return KDA_ERR_INVALID_ARG;
    if (!matrix_ok(a->gate, a->gate_dtype, tokens, a->D, a->gate_stride)) return KDA_ERR_INVALID_ARG;
    if (forward && !matrix_ok(a->y, a->dtype, tokens, a->D, a->y_stride)) return KDA_ERR_INVALID_ARG;
    if (!forward && a->h_chunks == nullptr) return KDA_ERR_INVALID_ARG;
    // (packed sequences need at least this many; the device counts them)
    if (a->h_chunks && a->h_chunks_rows < ((static_cast<int64_t>(a->T) + 15) / 16) * a->B) return KDA_ERR_INVALID_ARG;
  }
  if (forward && (!aligned(a->h0, 4) || !aligned(a->hT, 4))) return KDA_ERR_INVALID_ARG;
  if (!aligned(a->h_chunks, 4) || !aligned(a->err, 4)) return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

kda_status check_linear(const kda_linear_args* a) {
  if (a == nullptr || a->M < 0 || a->N < 1 || a->K < 1) return KDA_ERR_INVALID_ARG;
  if (!is_dtype(a->dtype) || !is_dtype(a->y_dtype)) return KDA_ERR_INVALID_ARG;
  if (a->activation < KDA_ACT_NONE || a->activation > KDA_ACT_RELU) return KDA_ERR_INVALID_ARG;
  if (a->dtype == KDA_DTYPE_FP32 || a->y_dtype == KDA_DTYPE_E4M3) return KDA_ERR_UNSUPPORTED;
  if (!aligned(a->err, 4)) return KDA_ERR_INVALID_ARG;
  if (a->M == 0) return KDA_OK;
  if (!matrix_ok(a->x, a->dtype, a->M, a->K, a->ldx) || !matrix_ok(a->w, a->dtype, a->N, a->K, a->ldw) ||
      !matrix_ok(a->y, a->y_dtype, a->M, a->N, a->ldy))
    return KDA_ERR_INVALID_ARG;
  if (a->residual && !matrix_ok(a->residual, a->y_dtype, a->M, a->N, a->ld_residual)) return KDA_ERR_INVALID_ARG;
  const bool scaled = a->dtype == KDA_DTYPE_E4M3;
  if (scaled != (a->x_scale != nullptr) || scaled != (a->w_scale != nullptr)) return KDA_ERR_INVALID_ARG;
  if (!aligned(a->x_scale, 4) || !aligned(a->w_scale, 4) || !aligned(a->bias, 4)) return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_add_rmsnorm(const kda_add_rmsnorm_args* a, kda_stream_t stream) {
  if (a == nullptr || a->R < 0 || a->D < 1 || !(a->eps >= 0.f)) return KDA_ERR_INVALID_ARG;
  if (!is_dtype(a->dtype) || !is_dtype(a->y_dtype)) return KDA_ERR_INVALID_ARG;
  if (!is_float(a->dtype) || a->D > KDA_NORM_MAX_D || a->R > INT32_MAX) return KDA_ERR_UNSUPPORTED;
  if ((a->y_dtype == KDA_DTYPE_E4M3) != (a->y_scale != nullptr) && a->R > 0) return KDA_ERR_INVALID_ARG;
  if (!aligned(a->y_scale, 4)) return KDA_ERR_INVALID_ARG;
  if (a->R == 0) return KDA_OK;
  if (!matrix_ok(a->x, a->dtype, a->R, a->D, a->x_stride) || !matrix_ok(a->y, a->y_dtype, a->R, a->D, a->y_stride))
    return KDA_ERR_INVALID_ARG;
  if (a->residual && !matrix_ok(a->residual, a->dtype, a->R, a->D, a->residual_stride)) return KDA_ERR_INVALID_ARG;
  if (a->residual_out && !matrix_ok(a->residual_out, a->dtype, a->R, a->D, a->residual_out_stride))
    return KDA_ERR_INVALID_ARG;
  if (!a->weight || !aligned(a->weight, 4)) return KDA_ERR_INVALID_ARG;
  return done(kda::launch_add_rmsnorm(*a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kda_linear_workspace_size(const kda_linear_args* a) {
  return check_linear(a) == KDA_OK && a->M > 0 ? kda::linear_workspace_bytes(*a) : 0;
}

kda_status kda_linear(const kda_linear_args* a, void* workspace, size_t workspace_bytes, kda_stream_t stream) {
  const kda_status st = check_linear(a);
  if (st != KDA_OK || a->M == 0) return st;
  const size_t need = kda::linear_workspace_bytes(*a);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 256))) return KDA_ERR_INVALID_ARG;
  return done(kda::launch_linear(*a, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

kda_status kda_scan_fwd(const kda_scan_args* a, kda_stream_t stream) {
  if (a == nullptr) return KDA_ERR_INVALID_ARG;
  const kda_status st = check_scan(a, true);
  if (st != KDA_OK) return st;
  return done(kda::launch_scan_fwd(*a, reinterpret_cast<cudaStream_t>(stream)));
}

kda_status kda_scan_bwd(const kda_scan_bwd_args* a, kda_stream_t stream) {
  if (a == nullptr) return KDA_ERR_INVALID_ARG;
  const kda_status st = check_scan(&a->fwd, false);
  if (st != KDA_OK) return st;
  const int64_t tokens = static_cast<int64_t>(a->fwd.B) * a->fwd.T;
  if (tokens > 0) {
    if (!matrix_ok(a->dy, a->fwd.dtype, tokens, a->fwd.D, a->dy_stride) ||
        !matrix_ok(a->dx, a->fwd.dtype, tokens, a->fwd.D, a->dx_stride) ||
        !matrix_ok(a->dgate, a->fwd.gate_dtype, tokens, a->fwd.D, a->dgate_stride))
      return KDA_ERR_INVALID_ARG;
  }
  if (!aligned(a->dhT, 4) || !aligned(a->dh0, 4)) return KDA_ERR_INVALID_ARG;
  return done(kda::launch_scan_bwd(*a, reinterpret_cast<cudaStream_t>(stream)));
}

kda_status kda_scan_step(const kda_scan_step_args* a, kda_stream_t stream) {
  if (a == nullptr || a->B < 0 || a->D < 1 || a->num_slots < 0) return KDA_ERR_INVALID_ARG;
  if (a->flags & ~(KDA_SCAN_FLAG_COMPLEMENT | KDA_FLAG_CHECK_INDICES)) return KDA_ERR_INVALID_ARG;
  if ((a->flags & KDA_FLAG_CHECK_INDICES) && a->err == nullptr) return KDA_ERR_INVALID_ARG;
  const kda_status st = check_scan_common(a->dtype, a->gate_dtype, a->gate_mode);
  if (st != KDA_OK) return st;
  if (!aligned(a->err, 4)) return KDA_ERR_INVALID_ARG;
  if (a->B == 0) return KDA_OK;
  if (!matrix_ok(a->x, a->dtype, a->B, a->D, a->x_stride) || !matrix_ok(a->gate, a->gate_dtype, a->B, a->D, a->gate_stride) ||
      !matrix_ok(a->y, a->dtype, a->B, a->D, a->y_stride))
    return KDA_ERR_INVALID_ARG;
  if (!a->indices || !aligned(a->indices, 4)) return KDA_ERR_INVALID_ARG;
  if (a->num_slots > 0 && (!a->state_in || !a->state_out || !aligned(a->state_in, 4) || !aligned(a->state_out, 4)))
    return KDA_ERR_INVALID_ARG;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (a->flags & KDA_FLAG_CHECK_INDICES) e = kda::launch_check_indices(a->indices, a->B, a->num_slots, a->err, s);
  if (e == cudaSuccess) e = kda::launch_scan_step(*a, s);
  return done(e);
}

}  // extern "C"
