// Projection with its epilogue: y = act((x w^T) xs[m] ws[n] + bias[n]) + residual.
//
// One CTA computes a tile of 128 outputs (rows of w, the M side of the tensor
// core's product) x kTok tokens (rows of x, its N side): thread i of the four
// warps then holds output i of the tile in tensor-memory lane i, so bias and
// weight scale are one value per thread, and a warp's stores of one token are
// 32 consecutive outputs. Operands go through shared memory in blocks of 128
// bytes along K (64 bf16 or 128 e4m3 values), in the 128-byte swizzle.
//
// Plain loads, one buffer: every thread copies its share of both operand tiles,
// element by element (any stride and alignment; past the edges zeros).
#include "kda_cluster.cuh"
#include "kda_elem.cuh"
#include "kda_tcgen05.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;
constexpr int kOut = 128;       // outputs per tile (tensor-memory lanes)
constexpr int kTok = 64;        // tokens per tile (tensor-memory columns)
constexpr int kKBytes = 128;    // bytes of K per block: one row of the swizzle atom
constexpr uint64_t kWaitNs = 2000000000ull;

struct __align__(1024) LinearSmem {
  unsigned char w[kOut * kKBytes];
  unsigned char x[kTok * kKBytes];
  uint64_t bar;
  uint32_t tmem_base;
};

// One MMA of the 8-bit kind (e4m3 x e4m3, 32 values of K); its instruction
// descriptor is kind::f16's with operand formats 0 (e4m3).
__device__ __forceinline__ void mma_ss_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case KDA_ACT_SILU: return v / (1.f + expf(-v));
    case KDA_ACT_GELU: return 0.5f * v * (1.f + erff(v * 0.70710678f));
    case KDA_ACT_SIGMOID: return 1.f / (1.f + expf(-v));
    case KDA_ACT_RELU: return v < 0.f ? 0.f : v;
    default: return v;
  }
}

// Copies `rows` rows of one K block (elements k0 .. k0 + EPB - 1) into the
// swizzled tile: 16-byte chunk c of row r lies at chunk c ^ (r % 8).
template <typename E>
__device__ __forceinline__ void fill_tile(unsigned char* tile, const E* src, long long ld, int row0, int rows,
                                          int row_end, int k0, int K) {
  constexpr int EPB = kKBytes / sizeof(E);
  for (int i = threadIdx.x; i < rows * EPB; i += kThreads) {
    const int r = i / EPB, k = i % EPB, byte = k * static_cast<int>(sizeof(E));
    E v = 0;
    if (row0 + r < row_end && k0 + k < K) v = src[static_cast<long long>(row0 + r) * ld + k0 + k];
    *reinterpret_cast<E*>(tile + r * kKBytes + ((((byte >> 4) ^ r) & 7) << 4) + (byte & 15)) = v;
  }
}

template <typename E, typename Y>  // E: bits of an operand element (uint16_t bf16, uint8_t e4m3)
__global__ void __launch_bounds__(kThreads) kda_linear_kernel(const kda_linear_args p) {
  extern __shared__ unsigned char raw[];
  LinearSmem& sm = *reinterpret_cast<LinearSmem*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t{1023});
  const int tid = threadIdx.x, warp = tid >> 5;
  const int n0 = blockIdx.x * kOut, m0 = blockIdx.y * kTok;
  if (warp == 0) {
    tc05::tmem_alloc(&sm.tmem_base, kTok);
    tc05::tmem_relinquish();
  }
  if (tid == 0) {
    mbar_init(&sm.bar, 1);
    fence_mbarrier_init_cluster();
  }
  tc05::fence_before_sync();
  __syncthreads();
  tc05::fence_after_sync();
  const uint32_t tmem = sm.tmem_base;
  constexpr int EPB = kKBytes / sizeof(E);
  const uint32_t idesc = tc05::idesc_f16kind(kOut, kTok, sizeof(E) == 2);
  bool ok = true;
  uint32_t phase = 0;
  for (int k0 = 0; k0 < p.K; k0 += EPB) {
    fill_tile(sm.w, static_cast<const E*>(p.w), p.ldw, n0, kOut, p.N, k0, p.K);
    fill_tile(sm.x, static_cast<const E*>(p.x), p.ldx, m0, kTok, p.M, k0, p.K);
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      for (int s = 0; s < 4; ++s) {
        const uint64_t wd = tc05::smem_desc(smem_u32(sm.w) + 32 * s, 16, 1024, tc05::kSwizzle128B);
        const uint64_t xd = tc05::smem_desc(smem_u32(sm.x) + 32 * s, 16, 1024, tc05::kSwizzle128B);
        const uint32_t acc = k0 > 0 || s > 0;
        if (sizeof(E) == 2) tc05::mma_ss(tmem, wd, xd, idesc, acc);
        else mma_ss_f8(tmem, wd, xd, idesc, acc);
      }
      tc05::commit(&sm.bar);
    }
    ok = mbar_wait_bounded(smem_u32(&sm.bar), phase, kWaitNs);
    ok = __syncthreads_and(ok);
    if (!ok) break;
    phase ^= 1u;
  }
  tc05::fence_after_sync();
  const int n = n0 + tid;
  if (ok) {
    const float ws = p.w_scale && n < p.N ? p.w_scale[n] : 1.f;
    const float bias = p.bias && n < p.N ? p.bias[n] : 0.f;
    for (int c0 = 0; c0 < kTok && m0 + c0 < p.M; c0 += 16) {
      uint32_t r[16];
      tc05::ld16_wait(tmem + (static_cast<uint32_t>(32 * warp) << 16) + c0, r);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const long long m = m0 + c0 + j;
        if (m < p.M && n < p.N) {
          float v = __uint_as_float(r[j]);
          if (p.x_scale) v *= p.x_scale[m] * ws;
          v = activate(v + bias, p.activation);
          if (p.residual) v += load_f(static_cast<const Y*>(p.residual) + m * p.ld_residual + n);
          store_f(static_cast<Y*>(p.y) + m * p.ldy + n, v);
        }
      }
    }
  } else if (tid == 0) {
    set_err(p.err, KDA_ERR_TIMEOUT);
  }
  tc05::fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc05::fence_after_sync();
    tc05::tmem_dealloc(tmem, kTok);
  }
}

template <typename E, typename Y>
cudaError_t launch(const kda_linear_args& a, cudaStream_t s) {
  const long long gx = (a.N + kOut - 1) / kOut, gy = (static_cast<long long>(a.M) + kTok - 1) / kTok;
  if (gy > 65535) return cudaErrorNotSupported;
  kda_linear_kernel<E, Y><<<dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), kThreads,
                            sizeof(LinearSmem) + 1024, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear(const kda_linear_args& a, cudaStream_t s) {
  if (a.dtype == KDA_DTYPE_BF16)
    return a.y_dtype == KDA_DTYPE_BF16 ? launch<uint16_t, __nv_bfloat16>(a, s) : launch<uint16_t, float>(a, s);
  return a.y_dtype == KDA_DTYPE_BF16 ? launch<uint8_t, __nv_bfloat16>(a, s) : launch<uint8_t, float>(a, s);
}

}  // namespace kda
