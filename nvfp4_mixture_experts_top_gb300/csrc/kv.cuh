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

// Four f16 values -> four E5M2 codes, and the f16 values of two of them (a code is
// the high byte of its value).
__device__ __forceinline__ uint32_t encode_e5m2(__half2 ab, __half2 cd) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e5m2x2.f16x2 lo, %1;\n\t"
      "cvt.rn.satfinite.e5m2x2.f16x2 hi, %2;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "r"(*reinterpret_cast<const uint32_t*>(&ab)), "r"(*reinterpret_cast<const uint32_t*>(&cd)));
  return r;
}
__device__ __forceinline__ __half2 e5m2_pair(uint32_t w, int pair) {
  const uint32_t h = __byte_perm(w, 0, pair ? 0x3424 : 0x1404);
  return *reinterpret_cast<const __half2*>(&h);
}

// Four E4M3 codes -> two f16x2 (exact: every E4M3 value is an f16 value), of the
// low and the high two codes.
__device__ __forceinline__ void decode4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Four codes times a power of two, rounded once to E4M3 again (the fp32
// product of an E4M3 value and 2^n is exact down to 2^-149, far below half of
// E4M3's smallest step).
__device__ __forceinline__ uint32_t rescale_codes(uint32_t w, float f) {
  uint32_t lo, hi;
  decode4(w, lo, hi);
  const float2 a = f16x2_to_f32(lo), b = f16x2_to_f32(hi);
  return encode4(a.x * f, a.y * f, b.x * f, b.y * f);
}

// TMA load of a 3-D box, issued by the calling thread.
__device__ __forceinline__ void tma_load_3d(void* smem_dst, const void* tmap, uint64_t* bar, int32_t x, int32_t y,
                                            int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(smem_dst)),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// Byte offset of 16-byte chunk c of row r in rows of D bytes, as the TMA's swizzle
// of D bytes (128 or 64) places it.
template <int D>
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
  return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ (r >> 1 & 3)) << 4);
}

// Instruction descriptor, kind::f8f6f4 with E4M3 inputs and fp32 accumulate;
// both operands K-major, or both MN-major (transposed).
__host__ __device__ constexpr uint32_t idesc_e4m3(uint32_t M, uint32_t N, bool mn_major) {
  return (1u << 4)                            // D format: F32
         | (mn_major ? (3u << 15) : 0u)       // A and B are MN-major
         | ((N >> 3) << 17)
         | ((M >> 4) << 24);
}

// D[tmem] (+)= A[smem] * B[smem], E4M3 operands, fp32 accumulation (M = 128, K = 32).
__device__ __forceinline__ void ew_mma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Warp-collective TMEM loads and stores: 32 lanes x 16 (8) consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

}  // namespace kv
}  // namespace nvfp4moe
