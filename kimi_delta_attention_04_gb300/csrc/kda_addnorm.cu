// Residual addition + root-mean-square norm of whole rows, optionally to e4m3
// with one scale per row: r = x + residual, y = r / sqrt(mean(r^2) + eps) * w.
//
// HBM-bound streaming: a row is read once, 8 values a thread and step with 16-byte
// accesses, and stays in registers (fp32) through the reduction and the stores.
// A CTA takes rows blockIdx, blockIdx + grid, ..: the weights stay in registers and
// the next row is on its way while this one is reduced and stored. One reduction
// gives the sum of squares and, for e4m3, the maximum of |r w| together (the row's
// largest |y| is rstd times it), so a row costs one barrier. Rows up to 512 values
// take a warp each and no barrier: 8192 x 4096 bf16 with residual to e4m3 in 36.5 us, 6.4
// TB/s; 256 rows in 2.6 us from L2. Rows whose pitch or address is off the 16-byte
// grid are read one value at a time, lane-contiguous.
//
// A finite row can have squares beyond fp32's range (values above 1e19, or all below
// 1e-15 without an eps to speak of); its sum is formed again from values scaled by a
// power of two, which scales the root likewise and costs other rows one comparison.
#include "kda_elem.cuh"

namespace kda {
namespace {

constexpr int kVec = 8;  // values a thread holds per step

// The sum of `sum` and the NaN-keeping maximum of `top` over the threads of a row
// (WARPS warps; one warp: no shared memory), each in one fixed order. `part` is not
// in use by a thread that is still reading an earlier result (callers alternate two).
template <bool TOP, int WARPS>
__device__ __forceinline__ void row_reduce(float& sum, float& top, float2* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (TOP) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
  if (WARPS == 1) return;
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = make_float2(sum, top);
  __syncthreads();
  sum = part[0].x;
  top = part[0].y;
#pragma unroll
  for (int w = 1; w < WARPS; ++w) {
    sum += part[w].x;
    if (TOP) top = max_nan(top, part[w].y);
  }
}

// 8 values as they lie in memory.
struct Raw8Bf16 {
  uint32_t w[4];
  __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0u; }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 r = *reinterpret_cast<const uint4*>(p);
    w[0] = r.x, w[1] = r.y, w[2] = r.z, w[3] = r.w;
  }
  __device__ __forceinline__ void put(int j, const __nv_bfloat16* p) {
    w[j / 2] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(p)) << (16 * (j % 2));
  }
  __device__ __forceinline__ float get(int j) const { return __uint_as_float(j % 2 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16); }
};
struct Raw8F32 {
  float w[8];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 0.f;
  }
  __device__ __forceinline__ void load(const float* p) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
  __device__ __forceinline__ void put(int j, const float* p) { w[j] = *p; }
  __device__ __forceinline__ float get(int j) const { return w[j]; }
};
template <typename T> struct RawOf;
template <> struct RawOf<__nv_bfloat16> { using type = Raw8Bf16; };
template <> struct RawOf<float> { using type = Raw8F32; };

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[kVec]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(Bf16::pack(v[0], v[1]), Bf16::pack(v[2], v[3]), Bf16::pack(v[4], v[5]), Bf16::pack(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[kVec]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_fp8_storage_t* p, const float (&v)[kVec]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_e4m3x2(v[0], v[1]) | (pack_e4m3x2(v[2], v[3]) << 16),
                                            pack_e4m3x2(v[4], v[5]) | (pack_e4m3x2(v[6], v[7]) << 16));
}

// What a row's values are scaled by where the sum of their squares, ss, tells too little:
// inf, or so small that some squares may have rounded away (above 2^-100 what those of
// 32768 values lose is below 2^-34 of it; beside an eps of 2^-80 it is nothing). Sums of
// squares of scaled values lie between 2^-98 and 2^120.
__device__ __forceinline__ float range_scale(float ss, float eps) {
  return ss > 3.40282347e+38f ? 0x1p-80f : ss < 0x1p-100f && eps < 0x1p-80f ? 0x1p100f : 1.f;
}

// Column of a thread's value j in step s. WIDE: 8 consecutive columns a thread;
// otherwise consecutive threads hold consecutive columns.
template <bool WIDE, int THREADS>
__device__ __forceinline__ int column(int s, int t, int j) {
  return WIDE ? (s * THREADS + t) * kVec + j : (s * kVec + j) * THREADS + t;
}

template <bool WIDE, int THREADS, typename T>
__device__ __forceinline__ void load_step(const T* row, int s, int t, int D, typename RawOf<T>::type& v) {
  if (WIDE) {
    if (column<WIDE, THREADS>(s, t, 0) < D) v.load(row + column<WIDE, THREADS>(s, t, 0));
    else v.zero();
  } else {
    v.zero();
#pragma unroll
    for (int j = 0; j < kVec; ++j)
      if (column<WIDE, THREADS>(s, t, j) < D) v.put(j, row + column<WIDE, THREADS>(s, t, j));
  }
}

template <bool WIDE, int THREADS, typename T>
__device__ __forceinline__ void store_step(T* row, int s, int t, int D, const float (&v)[kVec]) {
  if (WIDE) {
    if (column<WIDE, THREADS>(s, t, 0) < D) store8(row + column<WIDE, THREADS>(s, t, 0), v);
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int c = column<WIDE, THREADS>(s, t, j);
      if (c < D) store_f(row + c, v[j]);
    }
  }
}

// Warps of the kernel's CTAs on an SM that its registers are limited for: 24 leave
// 80 registers, enough for two steps with the next row and the weights; four steps
// have neither and one CTA's own limit.
template <int THREADS, int STEPS>
constexpr int min_ctas() { return STEPS <= 2 ? 768 / THREADS : 1; }

// WARPS warps on a row; ROWS rows (of one warp each) in a CTA.
template <typename X, typename Y, int WARPS, int ROWS, int STEPS, bool WIDE>
__global__ void __launch_bounds__(32 * WARPS * ROWS, min_ctas<32 * WARPS * ROWS, STEPS>())
    kda_add_rmsnorm_kernel(const kda_add_rmsnorm_args p) {
  static_assert(WARPS == 1 || ROWS == 1, "");
  constexpr int THREADS = 32 * WARPS;
  constexpr bool KEEP = STEPS <= 2;  // weights in registers, next row on its way
  using Raw = typename RawOf<X>::type;
  __shared__ float2 part[3][WARPS];  // by parity of the row; of a scaled row
  const int t = threadIdx.x % THREADS;
  const long long stride = static_cast<long long>(gridDim.x) * ROWS;
  long long row = static_cast<long long>(blockIdx.x) * ROWS + threadIdx.x / THREADS;
  Raw rx[STEPS], rr[STEPS];
  auto fetch = [&](long long at) {
    const X* x = static_cast<const X*>(p.x) + at * p.x_stride;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) load_step<WIDE, THREADS>(x, s, t, p.D, rx[s]);
    if (p.residual) {
      const X* r = static_cast<const X*>(p.residual) + at * p.residual_stride;
#pragma unroll
      for (int s = 0; s < STEPS; ++s) load_step<WIDE, THREADS>(r, s, t, p.D, rr[s]);
    }
  };
  Raw8F32 w[KEEP ? STEPS : 1];
  if (row < p.R) fetch(row);
  if (KEEP) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) load_step<WIDE, THREADS>(p.weight, s, t, p.D, w[s]);
  }
  for (int parity = 0; row < p.R; row += stride, parity ^= 1) {
    float v[STEPS][kVec];
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[s][j] = rx[s].get(j) + (p.residual ? rr[s].get(j) : 0.f);
    if (KEEP && row + stride < p.R) fetch(row + stride);
    float ss = 0.f, top = 0.f;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      if (!KEEP && sizeof(Y) == 1) load_step<WIDE, THREADS>(p.weight, s, t, p.D, w[0]);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        ss += v[s][j] * v[s][j];
        if (sizeof(Y) == 1) top = max_nan(top, fabsf(v[s][j] * w[KEEP ? s : 0].w[j]));
      }
    }
    row_reduce<sizeof(Y) == 1, WARPS>(ss, top, part[parity]);
    float eps = p.eps;
    const float by = range_scale(ss, eps);  // (the same in all threads of the row)
    if (by != 1.f) {
      ss = top = 0.f;
      eps *= by;
      eps *= by;
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        if (!KEEP && sizeof(Y) == 1) load_step<WIDE, THREADS>(p.weight, s, t, p.D, w[0]);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          const float u = v[s][j] * by;
          ss += u * u;
          if (sizeof(Y) == 1) top = max_nan(top, fabsf(u * w[KEEP ? s : 0].w[j]));
        }
      }
      row_reduce<sizeof(Y) == 1, WARPS>(ss, top, part[2]);
    }
    const float rstd = rsqrtf(ss / static_cast<float>(p.D) + eps);
    float inv = 1.f;
    if (sizeof(Y) == 1) {
      const float m = rstd * top;
      const float scale = m > 0.f ? fmaxf(m / 448.f, 1.17549435e-38f) : 1.f;
      inv = 1.f / scale;
      if (t == 0) p.y_scale[row] = scale;
    }
    if (p.residual_out) {
      X* ro = static_cast<X*>(p.residual_out) + row * p.residual_out_stride;
#pragma unroll
      for (int s = 0; s < STEPS; ++s) store_step<WIDE, THREADS>(ro, s, t, p.D, v[s]);
    }
    if (by != 1.f) {
#pragma unroll
      for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[s][j] *= by;
    }
    Y* y = static_cast<Y*>(p.y) + row * p.y_stride;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      if (!KEEP) load_step<WIDE, THREADS>(p.weight, s, t, p.D, w[0]);
#pragma unroll
      for (int j = 0; j < kVec; ++j) v[s][j] = v[s][j] * rstd * w[KEEP ? s : 0].w[j] * inv;
      store_step<WIDE, THREADS>(y, s, t, p.D, v[s]);
    }
    if (!KEEP && row + stride < p.R) fetch(row + stride);
  }
}

template <typename X, typename Y, bool WIDE, int WARPS, int ROWS, int STEPS>
cudaError_t launch_shape(const kda_add_rmsnorm_args& a, cudaStream_t s) {
  const long long groups = (a.R + ROWS - 1) / ROWS, resident = 152 * min_ctas<32 * WARPS * ROWS, STEPS>();
  const unsigned grid = static_cast<unsigned>(groups < resident ? groups : resident);
  kda_add_rmsnorm_kernel<X, Y, WARPS, ROWS, STEPS, WIDE><<<grid, 32 * WARPS * ROWS, 0, s>>>(a);
  return cudaGetLastError();
}

// The shape that holds a row of D values: up to 16 values a lane a warp of its own
// (four to a CTA), then CTAs of 2 to 32 warps with 16 or 32 values a thread. (The
// sizes in between powers of two leave fewer idle values: 1001 x 2501 fp32 on 5 warps
// instead of 8 takes 4.9 us instead of 5.7.)
template <typename X, typename Y, bool WIDE>
cudaError_t launch_row(const kda_add_rmsnorm_args& a, cudaStream_t s) {
  constexpr int kWarpValues = 32 * 2 * kVec;  // of a warp in two steps
  if (a.D <= kWarpValues / 2) return launch_shape<X, Y, WIDE, 1, 4, 1>(a, s);
  if (a.D <= kWarpValues) return launch_shape<X, Y, WIDE, 1, 4, 2>(a, s);
  if (a.D <= 2 * kWarpValues) return launch_shape<X, Y, WIDE, 2, 1, 2>(a, s);
  if (a.D <= 3 * kWarpValues) return launch_shape<X, Y, WIDE, 3, 1, 2>(a, s);
  if (a.D <= 4 * kWarpValues) return launch_shape<X, Y, WIDE, 4, 1, 2>(a, s);
  if (a.D <= 5 * kWarpValues) return launch_shape<X, Y, WIDE, 5, 1, 2>(a, s);
  if (a.D <= 8 * kWarpValues) return launch_shape<X, Y, WIDE, 8, 1, 2>(a, s);
  if (a.D <= 12 * kWarpValues) return launch_shape<X, Y, WIDE, 12, 1, 2>(a, s);
  if (a.D <= 16 * kWarpValues) return launch_shape<X, Y, WIDE, 16, 1, 2>(a, s);
  if (a.D <= 32 * kWarpValues) return launch_shape<X, Y, WIDE, 16, 1, 4>(a, s);
  return launch_shape<X, Y, WIDE, 32, 1, 4>(a, s);
}

// Whether rows start on the boundaries that 8 values at a time need.
bool wide_ok(const void* p, int64_t stride, size_t elem) {
  const size_t need = elem == 1 ? 8 : 16;
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % need == 0 && stride * static_cast<int64_t>(elem) % static_cast<int64_t>(need) == 0);
}

template <typename X, typename Y>
cudaError_t launch(const kda_add_rmsnorm_args& a, cudaStream_t s) {
  const bool wide = a.D % kVec == 0 && wide_ok(a.x, a.x_stride, sizeof(X)) && wide_ok(a.residual, a.residual_stride, sizeof(X)) &&
                    wide_ok(a.residual_out, a.residual_out_stride, sizeof(X)) && wide_ok(a.y, a.y_stride, sizeof(Y)) && wide_ok(a.weight, 0, sizeof(float));
  return wide ? launch_row<X, Y, true>(a, s) : launch_row<X, Y, false>(a, s);
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
