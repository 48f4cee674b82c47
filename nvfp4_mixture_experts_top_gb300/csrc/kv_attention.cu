// kv_attention.cu -- attention over the paged 8-bit key/value cache.
#include "common.cuh"
#include "kernels.h"
#include "kv.cuh"

namespace nvfp4moe {
namespace {

struct AttnParams {
  const __nv_bfloat16* q;
  const uint8_t *k_codes, *k_exps, *v_codes, *v_exps;
  const int32_t *table, *kv_lens, *query_start;
  __nv_bfloat16* out;
  float* lse;
  int32_t* dev_status;
  int64_t ld_q, ld_table, num_pages;
  int M, T, B, Hq, Hkv, shift;
  float scale;
};

// One warp per query token and head, one key at a time: the running maximum,
// sum and output of a softmax in registers, D / 32 elements per lane.
template <int D>
__global__ void __launch_bounds__(256) kv_attention_kernel(const AttnParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  const int64_t item = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 5;
  const int t = (int)(item / p.Hq), h = (int)(item % p.Hq);
  if (t >= p.T || t < p.query_start[0] || t >= p.query_start[p.B]) return;
  if (lane == 0 && (p.query_start[0] < 0 || p.query_start[p.B] > p.T)) report_status(p.dev_status, NVFP4_E_BAD_PAGE);
  int lo = 0, hi = p.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.query_start[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int S = 1 << p.shift;
  int64_t kv = p.kv_lens[lo];
  if (kv < 0 || kv > (int64_t)p.M * S) {
    if (lane == 0) report_status(p.dev_status, NVFP4_E_BAD_PAGE);
    kv = kv < 0 ? 0 : (int64_t)p.M * S;
  }
  const int64_t keys = kv - p.query_start[lo + 1] + t + 1;
  const int head = h / (p.Hq / p.Hkv);
  float q[E], o[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    q[i] = __bfloat162float(p.q[t * p.ld_q + h * D + lane * E + i]) * p.scale;
    o[i] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int64_t j = 0; j < keys; ++j) {
    const int page = p.table[lo * p.ld_table + (j >> p.shift)];
    if (page < 0 || page >= p.num_pages) {
      if (lane == 0) report_status(p.dev_status, NVFP4_E_BAD_PAGE);
      continue;
    }
    const int64_t block = (int64_t)page * p.Hkv + head;
    const int64_t at = (block * S + (j & (S - 1))) * D + lane * E;
    const float ks = exp2_int(p.k_exps[block] - 127), vs = exp2_int(p.v_exps[block] - 127);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) s += q[i] * (f32_from_e4m3(p.k_codes[at + i]) * ks);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    const float m1 = fmaxf(m, s);
    if (m1 == -INFINITY && s == -INFINITY) continue;  // (a NaN goes on)
    const float f = expf(m - m1), w = expf(s - m1);
    m = m1;
    l = l * f + w;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = o[i] * f + w * (f32_from_e4m3(p.v_codes[at + i]) * vs);
  }
#pragma unroll
  for (int i = 0; i < E; ++i)
    p.out[((int64_t)t * p.Hq + h) * D + lane * E + i] = __float2bfloat16(l == 0.0f ? 0.0f : o[i] / l);
  if (p.lse != nullptr && lane == 0) p.lse[(int64_t)t * p.Hq + h] = l == 0.0f ? -INFINITY : m + logf(l);
}

}  // namespace

size_t kv_attention_ws_bytes(int T, int B, int Hq, int Hkv, int D) {
  (void)T, (void)B, (void)Hq, (void)Hkv, (void)D;
  return 256;
}

cudaError_t launch_kv_attention(const KvAttention& a, cudaStream_t st) {
  AttnParams p = {static_cast<const __nv_bfloat16*>(a.q), a.k_codes, a.k_exps, a.v_codes, a.v_exps, a.table,
                  a.kv_lens, a.query_start, static_cast<__nv_bfloat16*>(a.out), a.lse, a.dev_status, a.ld_q,
                  a.ld_table, a.num_pages, a.M, a.T, a.B, a.Hq, a.Hkv, kv::log2_page(a.page_size), a.scale};
  const unsigned grid = (unsigned)(((int64_t)a.T * a.Hq * 32 + 255) / 256);
  return a.D == 128 ? launch_pdl(kv_attention_kernel<128>, grid, 256, 0, st, p)
                    : launch_pdl(kv_attention_kernel<64>, grid, 256, 0, st, p);
}

}  // namespace nvfp4moe
