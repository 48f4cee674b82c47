// block_norm.cu -- the norms around a block, its gate and the residual
// addition in one pass:
//   u = a * rsqrt(mean(a^2) + eps) * w_post
//   y = x + alpha * gate * u,   h = y * rsqrt(mean(y^2) + eps) * w_pre
#include "common.cuh"
#include "kernels.h"

namespace nvfp4moe {
namespace {

struct NormParams {
  const __nv_bfloat16* x;
  const void* a;
  const __nv_bfloat16 *gate, *w_post, *w_pre;
  __nv_bfloat16 *y, *h;
  int64_t ld_x, ld_a, gate_ld_t, gate_ld_c;
  float alpha, eps;
  int T, H;
};

__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// Sum over the CTA, the same value and order for every thread.
__device__ __forceinline__ float block_sum(float v, float* part) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0f;
  for (int w = 0; w < warps; ++w) v += part[w];
  return v;
}

// One CTA per row, the row in registers: NI vectors of eight elements per thread.
template <typename A, int NI>
__global__ void __launch_bounds__(1024) block_norm_kernel(const NormParams p) {
  __shared__ float part[2][32];
  pdl_wait();
  pdl_trigger();
  const int64_t t = blockIdx.x;
  const int nv = p.H / 8;
  float y[NI][8];
  const bool has_a = p.a != nullptr;
  float sum = 0.0f;
#pragma unroll
  for (int k = 0; k < NI; ++k) {
    const int i = k * blockDim.x + threadIdx.x;
#pragma unroll
    for (int c = 0; c < 8; ++c) y[k][c] = 0.0f;
    if (i < nv && has_a) {
      if constexpr (sizeof(A) == 4) {
        const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p.a) + t * p.ld_a) + 2 * i;
        const float4 u = s[0], v = s[1];
        y[k][0] = u.x, y[k][1] = u.y, y[k][2] = u.z, y[k][3] = u.w;
        y[k][4] = v.x, y[k][5] = v.y, y[k][6] = v.z, y[k][7] = v.w;
      } else {
        unpack8(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.a) + t * p.ld_a)[i], y[k]);
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) sum += y[k][c] * y[k][c];
    }
  }
  float r = p.alpha;
  if (has_a && p.w_post != nullptr) r *= rsqrtf(block_sum(sum, part[0]) / (float)p.H + p.eps);
  float g1 = 1.0f;
  if (p.gate != nullptr && p.gate_ld_c == 0) g1 = __bfloat162float(p.gate[t * p.gate_ld_t]);
  sum = 0.0f;
#pragma unroll
  for (int k = 0; k < NI; ++k) {
    const int i = k * blockDim.x + threadIdx.x;
    if (i >= nv) continue;
    float v[8];
    if (has_a) {
#pragma unroll
      for (int c = 0; c < 8; ++c) y[k][c] *= r;
      if (p.w_post != nullptr) {
        unpack8(reinterpret_cast<const uint4*>(p.w_post)[i], v);
#pragma unroll
        for (int c = 0; c < 8; ++c) y[k][c] *= v[c];
      }
      if (p.gate != nullptr) {
        if (p.gate_ld_c) {
          unpack8(reinterpret_cast<const uint4*>(p.gate + t * p.gate_ld_t)[i], v);
#pragma unroll
          for (int c = 0; c < 8; ++c) y[k][c] *= v[c];
        } else {
#pragma unroll
          for (int c = 0; c < 8; ++c) y[k][c] *= g1;
        }
      }
    }
    unpack8(reinterpret_cast<const uint4*>(p.x + t * p.ld_x)[i], v);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      y[k][c] += v[c];
      sum += y[k][c] * y[k][c];
    }
    if (has_a) reinterpret_cast<uint4*>(p.y + t * p.H)[i] = pack8(y[k]);
  }
  if (p.w_pre == nullptr) return;
  r = rsqrtf(block_sum(sum, part[1]) / (float)p.H + p.eps);
#pragma unroll
  for (int k = 0; k < NI; ++k) {
    const int i = k * blockDim.x + threadIdx.x;
    if (i >= nv) continue;
    float v[8];
    unpack8(reinterpret_cast<const uint4*>(p.w_pre)[i], v);
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] *= y[k][c] * r;
    reinterpret_cast<uint4*>(p.h + t * p.H)[i] = pack8(v);
  }
}

template <typename A>
cudaError_t launch(const NormParams& p, cudaStream_t st) {
  const int nv = p.H / 8;
  if (nv <= 1024) return launch_pdl(block_norm_kernel<A, 1>, p.T, (nv + 31) / 32 * 32, 0, st, p);
  return launch_pdl(block_norm_kernel<A, 2>, p.T, ((nv + 1) / 2 + 31) / 32 * 32, 0, st, p);
}

}  // namespace

cudaError_t launch_block_norm(const void* x, int64_t ld_x, const void* a, int a_dtype, int64_t ld_a, const void* gate,
                              int64_t gate_ld_t, int64_t gate_ld_c, const void* w_post, const void* w_pre, float alpha,
                              float eps, int T, int H, void* y, void* h, cudaStream_t st) {
  using bf = __nv_bfloat16;
  NormParams p = {static_cast<const bf*>(x), a, static_cast<const bf*>(gate), static_cast<const bf*>(w_post),
                  static_cast<const bf*>(w_pre), static_cast<bf*>(y), static_cast<bf*>(h), ld_x, ld_a, gate_ld_t,
                  gate_ld_c, alpha, eps, T, H};
  return a_dtype == NVFP4_DT_F32 ? launch<float>(p, st) : launch<bf>(p, st);
}

}  // namespace nvfp4moe
