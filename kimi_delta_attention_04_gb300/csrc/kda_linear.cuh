// Device code shared by the projection's kernels (kda_linear.cu, kda_linear_pair.cu):
// the 8-bit MMA, TMA loads of operand tiles, and the epilogue
// y = act((x w^T) xs[m] ws[n] + bias[n]) + residual.
#pragma once

#include "kda_cluster.cuh"
#include "kda_elem.cuh"
#include "kda_tcgen05.cuh"
#include "kda_tma.h"

namespace kda {
namespace linear {

constexpr int kOut = 128;       // outputs per CTA (tensor-memory lanes)
constexpr int kKBytes = 128;    // bytes of K per block: one row of the swizzle atom
constexpr uint64_t kLinearWaitNs = 2000000000ull;

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

__device__ __forceinline__ void tma_load_2d(uint32_t smem, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(smem),
      "l"(map), "r"(x), "r"(y), "r"(bar)
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

// What one thread needs to finish its output n of a tile's tokens.
template <typename Y>
struct Epilogue {
  const kda_linear_args& p;
  int n;
  float ws, bias;
  __device__ __forceinline__ Epilogue(const kda_linear_args& args, int out) : p(args), n(out), ws(1.f), bias(0.f) {
    if (n < p.N) {
      if (p.w_scale) ws = p.w_scale[n];
      if (p.bias) bias = p.bias[n];
    }
  }
  // Tokens m .. m + C - 1 (those below M). What the tokens need is read before
  // anything is stored: y may be the residual, so no load passes a store.
  template <int C>
  __device__ __forceinline__ void operator()(const float (&acc)[C], long long m) const {
    const int live = n < p.N ? static_cast<int>(p.M - m < C ? p.M - m : C) : 0;
    if (live <= 0) return;
    float xs[C], res[C];
    const Y* r = static_cast<const Y*>(p.residual) + m * p.ld_residual + n;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      xs[j] = p.x_scale && j < live ? p.x_scale[m + j] : 1.f;
      res[j] = p.residual && j < live ? load_f(r + j * p.ld_residual) : 0.f;
    }
    Y* y = static_cast<Y*>(p.y) + m * p.ldy + n;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const float v = activate(acc[j] * (xs[j] * ws) + bias, p.activation) + res[j];
      if (j < live) store_f(y + j * p.ldy, v);
    }
  }
};

template <int C>
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&v)[C]);
template <>
__device__ __forceinline__ void tmem_load<16>(uint32_t addr, float (&v)[16]) {
  uint32_t r[16];
  tc05::ld16_wait(addr, r);
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]);
}
template <>
__device__ __forceinline__ void tmem_load<32>(uint32_t addr, float (&v)[32]) {
  tc05::ld32_wait(addr, v);
}

}  // namespace linear
}  // namespace kda
