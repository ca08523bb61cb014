// Host side of the softmax attention calls of include/kda.h (append to the paged
// cache, whole prompts, single-token step): argument validation and dispatch. No
// allocation, no synchronisation.
#include <cmath>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/kda.h"
#include "kda_internal.h"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Rows of `cols` bf16 values (a token's heads): present, every row on a 16-byte
// boundary, not overlapping (one row has no stride to get wrong), within 64-bit
// byte offsets.
bool rows_ok(const void* p, int64_t rows, int64_t cols, int64_t stride) {
  if (p == nullptr || !aligned(p, 16)) return false;
  if (rows > 1 && (stride < cols || stride % 8 != 0)) return false;
  return stride >= 0 && stride < (INT64_C(1) << 39) && rows <= (INT64_C(1) << 52) / (stride > cols ? stride : cols);
}

kda_status done(cudaError_t e) {
  return e == cudaSuccess ? KDA_OK : e == cudaErrorNotSupported ? KDA_ERR_UNSUPPORTED : KDA_ERR_CUDA;
}

// Head counts and widths of one call. A row of heads stays below 2^31 values.
kda_status check_heads(int32_t HQ, int32_t HKV, int32_t D) {
  if (HQ < 1 || HKV < 1 || D < 1 || HQ % HKV != 0) return KDA_ERR_INVALID_ARG;
  if ((D != 64 && D != 128) || HQ > KDA_ATTN_MAX_HEADS) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

// A cache of `pages` pages. Slots and (page, head) pairs are counted in 32 bits.
kda_status check_cache(int32_t pages, int32_t page_size, int32_t HKV, int32_t dtype, const void* k, const void* v,
                       const float* ks, const float* vs) {
  if (pages < 0 || (dtype != KDA_DTYPE_BF16 && dtype != KDA_DTYPE_FP32 && dtype != KDA_DTYPE_E4M3)) return KDA_ERR_INVALID_ARG;
  if (dtype == KDA_DTYPE_FP32) return KDA_ERR_UNSUPPORTED;
  if (page_size < 1) return KDA_ERR_INVALID_ARG;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) return KDA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(pages) * page_size > INT32_MAX || static_cast<int64_t>(pages) * HKV > INT32_MAX) return KDA_ERR_INVALID_ARG;
  if (pages > 0 && (k == nullptr || v == nullptr)) return KDA_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16)) return KDA_ERR_INVALID_ARG;
  const bool scaled = dtype == KDA_DTYPE_E4M3;
  if (pages > 0 && (scaled != (ks != nullptr) || scaled != (vs != nullptr))) return KDA_ERR_INVALID_ARG;
  return aligned(ks, 16) && aligned(vs, 16) ? KDA_OK : KDA_ERR_INVALID_ARG;
}

// Tokens that a table has room for. At this limit counts of tokens past the last one stay
// below 2^31, and a prompt kernel's longest wait, for an item's whole work, below ten seconds
// (rows that are computed again take longer, which its limit counts in).
bool room_ok(int32_t width, int32_t page_size) { return static_cast<int64_t>(width) * page_size <= KDA_ATTN_MAX_TOKENS; }

// An output in place of an input: the same rows, or none of them.
bool place_ok(const void* out, int64_t out_stride, const void* in, int64_t in_stride, int64_t rows) {
  return out != in || out_stride == in_stride || rows <= 1;
}

bool scale_ok(float scale) { return scale > 0.f && std::isfinite(scale); }

kda_status check_step(const kda_attn_step_args* a) {
  if (a == nullptr || a->B < 0 || a->table_width < 0 || a->prefix_len < 0 || a->prefix_pages < 0 || !scale_ok(a->scale))
    return KDA_ERR_INVALID_ARG;
  kda_status st = check_heads(a->HQ, a->HKV, a->D);
  if (st != KDA_OK) return st;
  st = check_cache(a->pages, a->page_size, a->HKV, a->cache_dtype, a->k_cache, a->v_cache, a->k_scale, a->v_scale);
  if (st != KDA_OK) return st;
  if (!aligned(a->err, 4) || !aligned(a->lse, 4)) return KDA_ERR_INVALID_ARG;
  if (!room_ok(a->table_width, a->page_size) || a->prefix_len > KDA_ATTN_MAX_TOKENS) return KDA_ERR_UNSUPPORTED;
  if (a->B == 0) return KDA_OK;
  const int64_t cols = static_cast<int64_t>(a->HQ) * a->D;
  if (!rows_ok(a->q, a->B, cols, a->q_stride) || !rows_ok(a->o, a->B, cols, a->o_stride) || a->o == a->q) return KDA_ERR_INVALID_ARG;
  if (a->seq_lens == nullptr || !aligned(a->seq_lens, 4) || !aligned(a->block_table, 4)) return KDA_ERR_INVALID_ARG;
  if (a->table_width > 0 && a->block_table == nullptr) return KDA_ERR_INVALID_ARG;
  if (a->prefix_len > 0) {
    if (a->prefix_table == nullptr || !aligned(a->prefix_table, 4)) return KDA_ERR_INVALID_ARG;
    if (static_cast<int64_t>(a->prefix_pages) * a->page_size < a->prefix_len) return KDA_ERR_INVALID_ARG;
  }
  return KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_kv_append(const kda_kv_append_args* a, kda_stream_t stream) {
  if (a == nullptr || a->tokens < 0 || a->rot < 0 || a->max_positions < 0) return KDA_ERR_INVALID_ARG;
  if (a->flags & ~(KDA_KV_FLAG_INTERLEAVED | KDA_FLAG_CHECK_INDICES)) return KDA_ERR_INVALID_ARG;
  if ((a->flags & KDA_FLAG_CHECK_INDICES) && a->err == nullptr) return KDA_ERR_INVALID_ARG;
  const bool with_q = a->q != nullptr || a->q_out != nullptr;
  kda_status st = check_heads(with_q ? a->HQ : a->HKV, a->HKV, a->D);
  if (st != KDA_OK) return st;
  st = check_cache(a->pages, a->page_size, a->HKV, a->cache_dtype, a->k_cache, a->v_cache, a->k_scale, a->v_scale);
  if (st != KDA_OK) return st;
  if (a->rot % 2 != 0 || a->rot > a->D || !aligned(a->err, 4)) return KDA_ERR_INVALID_ARG;
  if (a->tokens == 0) return KDA_OK;
  if (a->rot > 0 ? (a->positions == nullptr || a->cos_sin == nullptr || !aligned(a->positions, 4) || !aligned(a->cos_sin, 16))
                 : (a->positions != nullptr || a->cos_sin != nullptr))
    return KDA_ERR_INVALID_ARG;
  if (a->slots == nullptr || !aligned(a->slots, 4)) return KDA_ERR_INVALID_ARG;
  const int64_t kv = static_cast<int64_t>(a->HKV) * a->D, qn = static_cast<int64_t>(a->HQ) * a->D;
  if (!rows_ok(a->k, a->tokens, kv, a->k_stride) || !rows_ok(a->v, a->tokens, kv, a->v_stride)) return KDA_ERR_INVALID_ARG;
  if (a->k_out && !rows_ok(a->k_out, a->tokens, kv, a->k_out_stride)) return KDA_ERR_INVALID_ARG;
  if (with_q && (!rows_ok(a->q, a->tokens, qn, a->q_stride) || !rows_ok(a->q_out, a->tokens, qn, a->q_out_stride)))
    return KDA_ERR_INVALID_ARG;
  if (!place_ok(a->q_out, a->q_out_stride, a->q, a->q_stride, a->tokens) || !place_ok(a->k_out, a->k_out_stride, a->k, a->k_stride, a->tokens))
    return KDA_ERR_INVALID_ARG;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (a->flags & KDA_FLAG_CHECK_INDICES) e = kda::launch_check_indices(a->slots, a->tokens, a->pages * a->page_size, a->err, s);
  if (e == cudaSuccess) e = kda::launch_kv_append(*a, s);
  return done(e);
}

kda_status kda_attn_fwd(const kda_attn_fwd_args* a, kda_stream_t stream) {
  if (a == nullptr || a->B < 1 || a->T < 0 || a->S < 0 || a->N < 1 || !scale_ok(a->scale)) return KDA_ERR_INVALID_ARG;
  if (a->flags & ~KDA_ATTN_FLAG_CAUSAL) return KDA_ERR_INVALID_ARG;
  kda_status st = check_heads(a->HQ, a->HKV, a->D);
  if (st != KDA_OK) return st;
  const bool packed = a->cu_seqlens != nullptr, paged = a->block_table != nullptr;
  if (packed ? a->B != 1 : a->N != a->B) return KDA_ERR_INVALID_ARG;
  if (a->cu_seqlens_k != nullptr && (!packed || paged)) return KDA_ERR_INVALID_ARG;
  if (paged != (a->seq_lens_k != nullptr)) return KDA_ERR_INVALID_ARG;
  if (!aligned(a->cu_seqlens, 4) || !aligned(a->cu_seqlens_k, 4) || !aligned(a->block_table, 4) || !aligned(a->seq_lens_k, 4) ||
      !aligned(a->lse, 4) || !aligned(a->err, 4))
    return KDA_ERR_INVALID_ARG;
  const int64_t queries = static_cast<int64_t>(a->B) * a->T, keys = static_cast<int64_t>(a->B) * a->S;
  if (queries > INT32_MAX / 2 || (!paged && keys > INT32_MAX / 2)) return KDA_ERR_INVALID_ARG;
  if (!paged && a->S > KDA_ATTN_MAX_TOKENS) return KDA_ERR_UNSUPPORTED;
  if (packed && !paged && a->cu_seqlens_k == nullptr && a->S != a->T) return KDA_ERR_INVALID_ARG;
  const int64_t qn = static_cast<int64_t>(a->HQ) * a->D, kv = static_cast<int64_t>(a->HKV) * a->D;
  if (paged) {
    st = check_cache(a->pages, a->page_size, a->HKV, KDA_DTYPE_BF16, a->k, a->v, nullptr, nullptr);
    if (st != KDA_OK) return st;
    if (a->table_width < 0) return KDA_ERR_INVALID_ARG;
    if (!room_ok(a->table_width, a->page_size)) return KDA_ERR_UNSUPPORTED;
  }
  if (queries == 0) return KDA_OK;
  if (!rows_ok(a->q, queries, qn, a->q_stride) || !rows_ok(a->o, queries, qn, a->o_stride) || a->o == a->q) return KDA_ERR_INVALID_ARG;
  if (!paged && keys > 0 && (!rows_ok(a->k, keys, kv, a->k_stride) || !rows_ok(a->v, keys, kv, a->v_stride))) return KDA_ERR_INVALID_ARG;
  return done(kda::launch_attn_fwd(*a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kda_attn_step_workspace_size(const kda_attn_step_args* a) {
  return check_step(a) == KDA_OK && a->B > 0 ? kda::attn_step_workspace_bytes(*a) : 0;
}

kda_status kda_attn_step(const kda_attn_step_args* a, void* workspace, size_t workspace_bytes, kda_stream_t stream) {
  const kda_status st = check_step(a);
  if (st != KDA_OK || a->B == 0) return st;
  const size_t need = kda::attn_step_workspace_bytes(*a);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 256))) return KDA_ERR_INVALID_ARG;
  return done(kda::launch_attn_step(*a, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
