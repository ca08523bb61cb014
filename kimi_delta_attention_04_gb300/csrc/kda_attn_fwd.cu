// Softmax attention over whole prompts: a warp for each query and head.
#include "kda_attn.cuh"

namespace kda {
namespace {

using namespace attn;

constexpr int kThreads = 256;

// Whether the arrays of lengths are as the contract has them (the whole block asks).
__device__ __forceinline__ bool lengths_ok(const kda_attn_fwd_args& p) {
  bool ok = true;
  for (int i = threadIdx.x; i <= p.N; i += blockDim.x) {
    if (p.cu_seqlens) ok &= i == 0 ? p.cu_seqlens[0] == 0 : p.cu_seqlens[i] >= p.cu_seqlens[i - 1] && p.cu_seqlens[i] <= p.T;
    if (p.cu_seqlens_k) ok &= i == 0 ? p.cu_seqlens_k[0] == 0 : p.cu_seqlens_k[i] >= p.cu_seqlens_k[i - 1] && p.cu_seqlens_k[i] <= p.S;
    if (p.seq_lens_k && i < p.N) ok &= p.seq_lens_k[i] >= 0 && p.seq_lens_k[i] <= p.table_width * p.page_size;
  }
  return __syncthreads_and(ok);
}

template <int D>
__global__ void __launch_bounds__(kThreads) kda_attn_rows_kernel(const kda_attn_fwd_args p) {
  if (!lengths_ok(p)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_err(p.err, KDA_ERR_INVALID_ARG);
    return;
  }
  const int lane = threadIdx.x % 32;
  const long long unit = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) / 32;
  const long long tok = unit / p.HQ;
  const int h = static_cast<int>(unit % p.HQ);
  if (tok >= static_cast<long long>(p.B) * p.T) return;
  int n, i, T, S;
  Keys keys = {p.k, p.v, nullptr, nullptr, nullptr, p.pages, p.page_size, p.HKV, p.k_stride, p.v_stride, 0};
  if (p.cu_seqlens) {
    if (tok >= p.cu_seqlens[p.N]) return;
    int lo = 0, hi = p.N - 1;  // the last n that starts at tok or before it
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (p.cu_seqlens[mid] <= tok) lo = mid; else hi = mid - 1;
    }
    n = lo;
    i = static_cast<int>(tok) - p.cu_seqlens[n];
    T = p.cu_seqlens[n + 1] - p.cu_seqlens[n];
    const int32_t* ck = p.cu_seqlens_k ? p.cu_seqlens_k : p.cu_seqlens;
    keys.first = ck[n];
    S = ck[n + 1] - ck[n];
  } else {
    n = static_cast<int>(tok / p.T);
    i = static_cast<int>(tok % p.T);
    T = p.T;
    S = p.S;
    keys.first = static_cast<long long>(n) * S;
  }
  if (p.block_table) {
    keys.table = p.block_table + static_cast<long long>(n) * p.table_width;
    S = p.seq_lens_k[n];
  }
  const int seen = p.flags & KDA_ATTN_FLAG_CAUSAL ? min(S, i + S - T + 1) : S;
  float q[D / 32], o[D / 32], m, l;
#pragma unroll
  for (int c = 0; c < D / 32; ++c)
    q[c] = __bfloat162float(static_cast<const __nv_bfloat16*>(p.q)[tok * p.q_stride + static_cast<long long>(h) * D + lane + 32 * c]);
  const int used = attend_row<D, false>(q, keys, h / (p.HQ / p.HKV), seen, p.scale * kLog2e, lane, p.err, m, l, o);
#pragma unroll
  for (int c = 0; c < D / 32; ++c)
    static_cast<__nv_bfloat16*>(p.o)[tok * p.o_stride + static_cast<long long>(h) * D + lane + 32 * c] =
        __float2bfloat16_rn(used == 0 ? 0.f : o[c] / l);
  if (p.lse && lane == 0) p.lse[tok * p.HQ + h] = used == 0 ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace

cudaError_t launch_attn_fwd(const kda_attn_fwd_args& a, cudaStream_t s) {
  const long long units = static_cast<long long>(a.B) * a.T * a.HQ, grid = (units + kThreads / 32 - 1) / (kThreads / 32);
  if (grid > INT32_MAX) return cudaErrorNotSupported;
  if (a.D == 64) kda_attn_rows_kernel<64><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(a);
  else kda_attn_rows_kernel<128><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kda
