// Gated linear recurrence, one fp32 state per sequence and channel:
//   h_t = a_t h_{t-1} + u_t,  u_t = x_t or (1 - a_t) x_t,  a_t = exp(g) or sigmoid(f),
// its gradients, and the single-token step on a pool of states.
//
// One thread per (sequence, channel) walks the tokens in order.
#include "kda_elem.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;
constexpr int kScanChunk = 16;  // tokens between the states of h_chunks

// sigmoid without overflow: e^-f = inf gives 0
__device__ __forceinline__ float decay_of(float f, int mode) {
  return mode == KDA_SCAN_LOG_DECAY ? expf(f) : 1.f / (1.f + expf(-f));
}

struct SeqPos {
  int start, end;        // tokens of the sequence
  long long chunk_base;  // its first chunk in h_chunks
};

// Finds sequence n, checking the whole of cu_seqlens on the way (all threads of
// the CTA call it). Returns false, after reporting, where the array is bad.
__device__ __forceinline__ bool find_sequence(const kda_scan_args& p, int n, SeqPos& pos) {
  if (p.cu_seqlens == nullptr) {
    pos.start = n * p.T;
    pos.end = pos.start + p.T;
    pos.chunk_base = static_cast<long long>(n) * ((p.T + kScanChunk - 1) / kScanChunk);
    return true;
  }
  __shared__ unsigned long long base, total;  // chunks before sequence n, of all
  if (threadIdx.x == 0) base = total = 0;
  bool bad = threadIdx.x == 0 && (p.cu_seqlens[0] != 0 || p.cu_seqlens[p.N] != p.T);
  unsigned long long mine = 0, all = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < p.N; i += blockDim.x) {
    const int s = p.cu_seqlens[i], e = p.cu_seqlens[i + 1];
    bad |= e < s || s < 0 || e > p.T;
    const unsigned chunks = bad ? 0u : static_cast<unsigned>(e - s + kScanChunk - 1) / kScanChunk;
    all += chunks;
    if (i < n) mine += chunks;
  }
  if (mine != 0) atomicAdd(&base, mine);
  if (all != 0) atomicAdd(&total, all);
  __syncthreads();
  bad |= p.h_chunks != nullptr && total > static_cast<unsigned long long>(p.h_chunks_rows);
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) set_err(p.err, KDA_ERR_INVALID_ARG);
    return false;
  }
  pos.start = p.cu_seqlens[n];
  pos.end = p.cu_seqlens[n + 1];
  pos.chunk_base = static_cast<long long>(base);
  return true;
}

template <typename X, typename G>
__global__ void __launch_bounds__(kThreads) kda_scan_fwd_kernel(const kda_scan_args p) {
  const int n = blockIdx.y, c = blockIdx.x * kThreads + threadIdx.x;
  SeqPos pos;
  if (!find_sequence(p, n, pos) || c >= p.D) return;
  const bool comp = p.flags & KDA_SCAN_FLAG_COMPLEMENT;
  float h = p.h0 ? p.h0[static_cast<long long>(n) * p.D + c] : 0.f;
  for (int t = pos.start; t < pos.end; ++t) {
    const int i = t - pos.start;
    if (p.h_chunks && i % kScanChunk == 0) p.h_chunks[(pos.chunk_base + i / kScanChunk) * p.D + c] = h;
    const float a = decay_of(load_f(static_cast<const G*>(p.gate) + t * p.gate_stride + c), p.gate_mode);
    const float x = load_f(static_cast<const X*>(p.x) + t * p.x_stride + c);
    h = a * h + (comp ? (1.f - a) * x : x);
    store_f(static_cast<X*>(p.y) + t * p.y_stride + c, h);
  }
  if (p.hT) p.hT[static_cast<long long>(n) * p.D + c] = h;
}

template <typename X, typename G>
__global__ void __launch_bounds__(kThreads) kda_scan_bwd_kernel(const kda_scan_bwd_args q) {
  const kda_scan_args& p = q.fwd;
  const int n = blockIdx.y, c = blockIdx.x * kThreads + threadIdx.x;
  SeqPos pos;
  if (!find_sequence(p, n, pos) || c >= p.D) return;
  const bool comp = p.flags & KDA_SCAN_FLAG_COMPLEMENT;
  const int len = pos.end - pos.start;
  float d = q.dhT ? q.dhT[static_cast<long long>(n) * p.D + c] : 0.f;
  for (int k = (len + kScanChunk - 1) / kScanChunk - 1; k >= 0; --k) {
    const int t0 = pos.start + k * kScanChunk, m = min(kScanChunk, len - k * kScanChunk);
    float a[kScanChunk], x[kScanChunk], hp[kScanChunk];  // decay, input, state before the token
    float h = p.h_chunks[(pos.chunk_base + k) * p.D + c];
#pragma unroll
    for (int i = 0; i < kScanChunk; ++i) {
      if (i < m) {
        a[i] = decay_of(load_f(static_cast<const G*>(p.gate) + (t0 + i) * p.gate_stride + c), p.gate_mode);
        x[i] = load_f(static_cast<const X*>(p.x) + (t0 + i) * p.x_stride + c);
        hp[i] = h;
        h = a[i] * h + (comp ? (1.f - a[i]) * x[i] : x[i]);
      }
    }
#pragma unroll
    for (int i = kScanChunk - 1; i >= 0; --i) {
      if (i < m) {
        const long long t = t0 + i;
        d += load_f(static_cast<const X*>(q.dy) + t * q.dy_stride + c);
        const float da = comp ? d * (hp[i] - x[i]) : d * hp[i];
        store_f(static_cast<X*>(q.dx) + t * q.dx_stride + c, comp ? (1.f - a[i]) * d : d);
        d *= a[i];
        store_f(static_cast<G*>(q.dgate) + t * q.dgate_stride + c,
                a[i] * (p.gate_mode == KDA_SCAN_LOG_DECAY ? da : (1.f - a[i]) * da));
      }
    }
  }
  if (q.dh0) q.dh0[static_cast<long long>(n) * p.D + c] = d;
}

template <typename X, typename G>
__global__ void __launch_bounds__(kThreads) kda_scan_step_kernel(const kda_scan_step_args p) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  const long long b = blockIdx.y;
  if (c >= p.D) return;
  const int slot = p.indices[b];
  X* y = static_cast<X*>(p.y) + b * p.y_stride + c;
  if (slot < 0 || slot >= p.num_slots) {
    if (slot >= 0 && c == 0) set_err(p.err, KDA_ERR_INVALID_ARG);
    store_f(y, 0.f);
    return;
  }
  const float a = decay_of(load_f(static_cast<const G*>(p.gate) + b * p.gate_stride + c), p.gate_mode);
  const float x = load_f(static_cast<const X*>(p.x) + b * p.x_stride + c);
  const long long at = static_cast<long long>(slot) * p.D + c;
  const float h = a * p.state_in[at] + (p.flags & KDA_SCAN_FLAG_COMPLEMENT ? (1.f - a) * x : x);
  p.state_out[at] = h;
  store_f(y, h);
}

}  // namespace

// The kernels' instances by tensor types: x bf16 with a bf16 or fp32 gate, or both fp32.
#define KDA_SCAN_LAUNCH(kernel, args, xt, gt, grid, s)                                                 \
  do {                                                                                                 \
    if ((xt) == KDA_DTYPE_FP32) kernel<float, float><<<grid, kThreads, 0, s>>>(args);                  \
    else if ((gt) == KDA_DTYPE_FP32) kernel<__nv_bfloat16, float><<<grid, kThreads, 0, s>>>(args);     \
    else kernel<__nv_bfloat16, __nv_bfloat16><<<grid, kThreads, 0, s>>>(args);                         \
  } while (0)

static unsigned blocks_of(int D) { return static_cast<unsigned>((D + kThreads - 1) / kThreads); }

cudaError_t launch_scan_fwd(const kda_scan_args& a, cudaStream_t s) {
  if (a.N > 65535) return cudaErrorNotSupported;
  const dim3 grid(blocks_of(a.D), a.N);
  KDA_SCAN_LAUNCH(kda_scan_fwd_kernel, a, a.dtype, a.gate_dtype, grid, s);
  return cudaGetLastError();
}

cudaError_t launch_scan_bwd(const kda_scan_bwd_args& a, cudaStream_t s) {
  if (a.fwd.N > 65535) return cudaErrorNotSupported;
  const dim3 grid(blocks_of(a.fwd.D), a.fwd.N);
  KDA_SCAN_LAUNCH(kda_scan_bwd_kernel, a, a.fwd.dtype, a.fwd.gate_dtype, grid, s);
  return cudaGetLastError();
}

cudaError_t launch_scan_step(const kda_scan_step_args& a, cudaStream_t s) {
  if (a.B > 65535) return cudaErrorNotSupported;
  const dim3 grid(blocks_of(a.D), a.B);
  KDA_SCAN_LAUNCH(kda_scan_step_kernel, a, a.dtype, a.gate_dtype, grid, s);
  return cudaGetLastError();
}

}  // namespace kda
