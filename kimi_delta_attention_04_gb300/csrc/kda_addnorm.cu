// Residual addition + root-mean-square norm of whole rows, optionally to e4m3
// with one scale per row: r = x + residual, y = r / sqrt(mean(r^2) + eps) * w.
//
// One CTA per row; the row stays in shared memory (fp32) between the sum of
// squares, the maximum and the store, so each input is read once.
#include "kda_elem.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;

template <bool MAX>
__device__ __forceinline__ float block_reduce(float v, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? max_nan(v, u) : v + u;
  }
  __syncthreads();  // the previous use of `part` is over
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = part[0];
  for (int w = 1; w < kThreads / 32; ++w) v = MAX ? max_nan(v, part[w]) : v + part[w];
  return v;
}

template <typename X, typename Y>
__global__ void __launch_bounds__(kThreads) kda_add_rmsnorm_kernel(const kda_add_rmsnorm_args p) {
  extern __shared__ float row_vals[];
  __shared__ float part[kThreads / 32];
  const long long row = blockIdx.x;
  const X* x = static_cast<const X*>(p.x) + row * p.x_stride;
  const X* res = p.residual ? static_cast<const X*>(p.residual) + row * p.residual_stride : nullptr;
  float ss = 0.f;
  for (int i = threadIdx.x; i < p.D; i += kThreads) {
    const float r = load_f(x + i) + (res ? load_f(res + i) : 0.f);
    row_vals[i] = r;
    ss += r * r;
  }
  ss = block_reduce<false>(ss, part);
  const float rstd = rsqrtf(ss / static_cast<float>(p.D) + p.eps);
  float inv = 1.f;
  if (sizeof(Y) == 1) {
    float m = 0.f;
    for (int i = threadIdx.x; i < p.D; i += kThreads) m = max_nan(m, fabsf(row_vals[i] * rstd * p.weight[i]));
    m = block_reduce<true>(m, part);
    const float scale = m > 0.f ? fmaxf(m / 448.f, 1.17549435e-38f) : 1.f;
    inv = 1.f / scale;
    if (threadIdx.x == 0) p.y_scale[row] = scale;
  }
  Y* y = static_cast<Y*>(p.y) + row * p.y_stride;
  X* ro = p.residual_out ? static_cast<X*>(p.residual_out) + row * p.residual_out_stride : nullptr;
  for (int i = threadIdx.x; i < p.D; i += kThreads) {
    const float r = row_vals[i];
    if (ro) store_f(ro + i, r);
    store_f(y + i, r * rstd * p.weight[i] * inv);
  }
}

template <typename X, typename Y>
cudaError_t launch(const kda_add_rmsnorm_args& a, cudaStream_t s) {
  static std::atomic<uint64_t> smem_set{0};
  cudaError_t e = set_smem_limit_once(kda_add_rmsnorm_kernel<X, Y>, KDA_NORM_MAX_D * sizeof(float), smem_set);
  if (e != cudaSuccess) return e;
  kda_add_rmsnorm_kernel<X, Y><<<static_cast<unsigned>(a.R), kThreads, a.D * sizeof(float), s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_add_rmsnorm(const kda_add_rmsnorm_args& a, cudaStream_t s) {
  if (a.dtype == KDA_DTYPE_BF16) {
    if (a.y_dtype == KDA_DTYPE_BF16) return launch<__nv_bfloat16, __nv_bfloat16>(a, s);
    if (a.y_dtype == KDA_DTYPE_FP32) return launch<__nv_bfloat16, float>(a, s);
    return launch<__nv_bfloat16, __nv_fp8_storage_t>(a, s);
  }
  if (a.y_dtype == KDA_DTYPE_BF16) return launch<float, __nv_bfloat16>(a, s);
  if (a.y_dtype == KDA_DTYPE_FP32) return launch<float, float>(a, s);
  return launch<float, __nv_fp8_storage_t>(a, s);
}

}  // namespace kda
