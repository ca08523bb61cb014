// Element types of the layer operators' tensors (bf16, fp32, e4m3), converted to
// and from fp32 one value at a time; reductions that keep NaN.
#pragma once

#include <cuda_fp8.h>

#include "kda_common.cuh"

namespace kda {

__device__ __forceinline__ float load_f(const float* p) { return *p; }
__device__ __forceinline__ float load_f(const __nv_bfloat16* p) { return __bfloat162float(*p); }

__device__ __forceinline__ void store_f(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_f(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Two fp32 values to two e4m3 bytes (lo in the low byte), round to nearest even,
// saturating at +-448; NaN stays NaN.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void store_f(__nv_fp8_storage_t* p, float v) {
  *p = static_cast<__nv_fp8_storage_t>(pack_e4m3x2(v, 0.f) & 0xffu);
}

// max(a, b), NaN when either is NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

}  // namespace kda
