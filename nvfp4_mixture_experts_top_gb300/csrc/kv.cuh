// kv.cuh -- helpers shared by the kernels of the 8-bit key/value cache.
#pragma once

#include "common.cuh"

namespace nvfp4moe {
namespace kv {

__host__ __device__ constexpr int log2_page(int S) { return S == 16 ? 4 : (S == 32 ? 5 : (S == 64 ? 6 : 7)); }

// Four fp32 values -> four E4M3 codes (the first in the low byte), round to
// nearest even, saturating at 448; NaN stays NaN.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// Two E4M3 codes -> f16x2 (exact: every E4M3 value is an f16 value).
__device__ __forceinline__ uint32_t decode2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}

__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Four codes times a power of two, rounded once to E4M3 again (the fp32
// product of an E4M3 value and 2^n is exact down to 2^-149, far below half of
// E4M3's smallest step).
__device__ __forceinline__ uint32_t rescale_codes(uint32_t w, float f) {
  const float2 a = f16x2_to_f32(decode2((uint16_t)w)), b = f16x2_to_f32(decode2((uint16_t)(w >> 16)));
  return encode4(a.x * f, a.y * f, b.x * f, b.y * f);
}

// TMA load of a 3-D box by one elected lane of a converged warp.
__device__ __forceinline__ void ew_tma_load_3d(void* smem_dst, const void* tmap, uint64_t* bar, int32_t x, int32_t y,
                                               int32_t z) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(smem_u32(smem_dst)),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

}  // namespace kv
}  // namespace nvfp4moe
