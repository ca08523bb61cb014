// Device code shared by the projection's kernels (kda_linear.cu, kda_linear_wide.cu):
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

// The wait for a whole tile's sum: a block takes 0.2 to 0.4 us (K = 2^31 is 2^25 of them).
__device__ __forceinline__ uint64_t tile_wait_ns(int blocks) { return kLinearWaitNs + 2000ull * blocks; }

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

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Until the copy of an operand, if the launch before was one, has ended and its writes
// can be read.
__device__ __forceinline__ void wait_for_copy() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Clusters of `cluster` CTAs; after the copy of an operand, a launch while the copy
// still runs: barriers and tensor memory are set up meanwhile, and only the loads wait
// (777 x 1001 -> 1111 bf16: 12.4 us instead of 13.4; 40 x 51 -> 30: 5.2 instead of 6.7).
inline void set_attributes(cudaLaunchConfig_t& cfg, cudaLaunchAttribute (&attrs)[2], int cluster, bool after_copy) {
  attrs[0].id = cudaLaunchAttributeClusterDimension;
  attrs[0].val.clusterDim.x = cluster;
  attrs[0].val.clusterDim.y = attrs[0].val.clusterDim.z = 1;
  attrs[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = after_copy ? 2 : 1;
}

// 1 / (1 + e^-v) from the special-function unit (ex2, rcp): off by a few steps of fp32 and,
// for v < 0, by what half a step of v comes to, |v| half steps; v is rounded itself.
// e^-v = inf gives 0.
__device__ __forceinline__ float fast_sigmoid(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2_approx(-1.44269504f * v)));
  return r;
}

// v (1 + erf(v / sqrt 2)) / 2 through erfc(z) = (c0 t + .. + c7 t^8) e^(-z^2) for z = |v| /
// sqrt 2, t = 1 / (1 + 0.431 z): on the negative side the small result is formed directly,
// not as a difference. The coefficients are fitted for the least relative error of
// e^(z^2) erfc(z) up to z = 9.4 (9e-8), so that what is left is fp32's own: some steps of
// the result, and what half a step of v comes to, v^2 of its half steps. Half the
// instructions of erff, which had been a third of 8192 x 4096 outputs' time at e4m3.
// Two values at a time, so that the longer polynomial costs no more than five terms alone.
__device__ __forceinline__ float2 gelu2(float2 v) {
  auto both = [](float c) { return make_float2(c, c); };
  const float2 m = make_float2(fminf(fabsf(v.x), 100.f), fminf(fabsf(v.y), 100.f));  // (inf * 0 would be NaN; e^-5000 is 0)
  const float2 q = fma2(both(0.304763019f), m, both(1.f));
  float2 t;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t.x) : "f"(q.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t.y) : "f"(q.y));
  float2 c = fma2(both(0.0734755993f), t, both(-0.307073146f));
  c = fma2(c, t, both(0.374484748f));
  c = fma2(c, t, both(-0.0783652589f));
  c = fma2(c, t, both(0.243221879f));
  c = fma2(c, t, both(0.206376895f));
  c = fma2(c, t, both(0.244791761f));
  c = fma2(c, t, both(0.243087605f));
  const float2 z = mul2(mul2(m, m), both(-0.721347520f));
  // |v| erfc(z) / 2
  const float2 tail = mul2(mul2(mul2(both(0.5f), m), mul2(c, t)), make_float2(ex2_approx(z.x), ex2_approx(z.y)));
  return make_float2(v.x > 0.f ? v.x - tail.x : v.x == v.x ? -tail.x : v.x, v.y > 0.f ? v.y - tail.y : v.y == v.y ? -tail.y : v.y);
}

template <int ACT>
__device__ __forceinline__ float activate(float v) {
  if (ACT == KDA_ACT_SILU) return v * fast_sigmoid(v);
  if (ACT == KDA_ACT_SIGMOID) return fast_sigmoid(v);
  if (ACT == KDA_ACT_RELU) return v < 0.f ? 0.f : v;
  return v;
}
template <int ACT, int C>
__device__ __forceinline__ void activate_all(float (&v)[C]) {
  static_assert(C % 2 == 0, "");
#pragma unroll
  for (int j = 0; j < C; j += 2) {
    if (ACT == KDA_ACT_GELU) {
      const float2 g = gelu2(make_float2(v[j], v[j + 1]));
      v[j] = g.x, v[j + 1] = g.y;
    } else {
      v[j] = activate<ACT>(v[j]), v[j + 1] = activate<ACT>(v[j + 1]);
    }
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
  // Tokens m .. m + C - 1 (those below M). The choices are made once for the C
  // values, and all reads are issued before anything is stored (y may be the
  // residual, so no load passes a store): 32 reads one by one had made the epilogue
  // of 8192 x 4096 outputs 5 times the products' time.
  // SCALED: the tokens' scales have been multiplied in already.
  template <bool SCALED = false, int C>
  __device__ __forceinline__ void operator()(float (&v)[C], long long m) const {
    const int live = n < p.N ? static_cast<int>(p.M - m < C ? p.M - m : C) : 0;
    if (live <= 0) return;
    float res[C];
    if (p.residual) {
      const Y* r = static_cast<const Y*>(p.residual) + m * p.ld_residual + n;
#pragma unroll
      for (int j = 0; j < C; ++j) res[j] = load_f(r + (j < live ? j : 0) * p.ld_residual);
    } else {
#pragma unroll
      for (int j = 0; j < C; ++j) res[j] = 0.f;
    }
    if (SCALED) {
#pragma unroll
      for (int j = 0; j < C; ++j) v[j] *= ws;
    } else if (p.x_scale) {
#pragma unroll
      for (int j = 0; j < C; ++j) v[j] *= p.x_scale[m + (j < live ? j : 0)] * ws;
    }
#pragma unroll
    for (int j = 0; j < C; ++j) v[j] += bias;
    switch (p.activation) {
      case KDA_ACT_SILU: activate_all<KDA_ACT_SILU>(v); break;
      case KDA_ACT_GELU: activate_all<KDA_ACT_GELU>(v); break;
      case KDA_ACT_SIGMOID: activate_all<KDA_ACT_SIGMOID>(v); break;
      case KDA_ACT_RELU: activate_all<KDA_ACT_RELU>(v); break;
      default: break;
    }
    Y* y = static_cast<Y*>(p.y) + m * p.ldy + n;
    if (live == C) {
#pragma unroll
      for (int j = 0; j < C; ++j) store_f(y + j * p.ldy, v[j] + res[j]);
    } else {
#pragma unroll
      for (int j = 0; j < C; ++j)
        if (j < live) store_f(y + j * p.ldy, v[j] + res[j]);
    }
  }
};

// 16 columns of this warp's 32 lanes of tensor memory.
__device__ __forceinline__ void tmem_load(uint32_t addr, float (&v)[16]) {
  uint32_t r[16];
  tc05::ld16_wait(addr, r);
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]);
}

}  // namespace linear
}  // namespace kda
