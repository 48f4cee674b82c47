// kv_cache.cu -- the paged 8-bit key/value cache: the step's page and slot
// bookkeeping (kv_plan) and the quantising writer (kv_append).
#include "common.cuh"
#include "kernels.h"
#include "kv.cuh"

namespace nvfp4moe {
namespace {

// ---------------------------------------------------------------------------
// kv_plan
//
// Two exclusive prefix sums over the requests -- new tokens, and pages needed
// -- then every new page and every new token on its own.  A few kilobytes of
// integers: the time is one launch plus a short chain of dependent loads, so
// every CTA repeats the prefix sums (8 bytes of lengths per request, from L2)
// rather than waiting for another one to do it.
// ---------------------------------------------------------------------------

constexpr int kPlanThreads = 512;

struct PlanParams {
  const int32_t *ctx, *add;
  int32_t* table;
  const int32_t *free_pages, *free_count;
  int32_t *query_start, *kv_lens, *slot_map, *free_left, *dev_status;
  int64_t ld_table;
  int B, M, num_free, T, shift;  // page size = 1 << shift
};

// Lengths of request b as they count: a negative one, or more new tokens than
// the call has, brings no token (and is reported).
__device__ __forceinline__ bool plan_lengths(const PlanParams& p, int b, int& c, int& n) {
  c = p.ctx[b];
  n = p.add[b];
  const bool ok = c >= 0 && n >= 0 && n <= p.T && c <= INT32_MAX - n;
  if (!ok) {
    c = c > 0 ? c : 0;
    n = 0;
  }
  return ok;
}

__device__ __forceinline__ int pages_of(int64_t tokens, int shift) {
  return (int)((tokens + (1 << shift) - 1) >> shift);
}

__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const PlanParams p) {
  extern __shared__ int32_t sm[];  // start[B + 1], first[B] (-1: the request does not fit)
  int32_t* start = sm;
  int32_t* first = sm + p.B + 1;
  __shared__ int64_t sums[2][kPlanThreads / 32];
  __shared__ int32_t s_taken[kPlanThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_trigger();

  // each thread sums a contiguous range of requests, then the ranges' offsets
  const int per = (p.B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  int64_t tok = 0, pg = 0;
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    int c, n;
    bad |= !plan_lengths(p, b, c, n);
    tok += n;
    pg += pages_of((int64_t)c + n, p.shift) - pages_of(c, p.shift);
  }
  int64_t t_in = tok, p_in = pg;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t a = __shfl_up_sync(0xFFFFFFFFu, t_in, d), b = __shfl_up_sync(0xFFFFFFFFu, p_in, d);
    if (lane >= d) {
      t_in += a;
      p_in += b;
    }
  }
  if (lane == 31) {
    sums[0][warp] = t_in;
    sums[1][warp] = p_in;
  }
  __syncthreads();
  int64_t t_off = t_in - tok, p_off = p_in - pg;
  for (int w = 0; w < warp; ++w) {
    t_off += sums[0][w];
    p_off += sums[1][w];
  }
  int n_free = p.free_count[0];
  n_free = n_free < 0 ? 0 : (n_free > p.num_free ? p.num_free : n_free);
  const bool lead = blockIdx.x == 0;
  int taken = 0;
  bool full = false;
  for (int b = b0; b < b1; ++b) {
    int c, n;
    plan_lengths(p, b, c, n);
    const int want = pages_of((int64_t)c + n, p.shift), need = want - pages_of(c, p.shift);
    const bool fits = (need == 0 || p_off + need <= n_free) && want <= p.M;
    start[b] = (int32_t)(t_off < INT32_MAX ? t_off : INT32_MAX);
    first[b] = fits ? (int32_t)(need ? p_off : 0) : -1;
    if (lead) {
      p.query_start[b] = start[b];
      p.kv_lens[b] = fits ? c + n : c;
    }
    taken += fits ? need : 0;
    full |= !fits;
    t_off += n;
    p_off += need;
  }
  if (tid == kPlanThreads - 1) start[p.B] = (int32_t)(t_off < INT32_MAX ? t_off : INT32_MAX);
  if (lead) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) taken += __shfl_xor_sync(0xFFFFFFFFu, taken, d);
    if (lane == 0) s_taken[warp] = taken;
    if (bad) report_status(p.dev_status, NVFP4_E_BAD_PAGE);
    if (full) report_status(p.dev_status, NVFP4_E_CACHE_FULL);
  }
  __syncthreads();
  if (lead && tid == 0) {
    int all = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) all += s_taken[w];
    p.free_left[0] = n_free - all;
    p.query_start[p.B] = start[p.B];
    if (start[p.B] > p.T) report_status(p.dev_status, NVFP4_E_BAD_PAGE);
  }

  // new pages: a warp per request, lanes over its pages
  for (int b = blockIdx.x * (kPlanThreads / 32) + warp; b < p.B; b += gridDim.x * (kPlanThreads / 32)) {
    if (first[b] < 0) continue;
    int c, n;
    plan_lengths(p, b, c, n);
    const int held = pages_of(c, p.shift), want = pages_of((int64_t)c + n, p.shift);
    for (int j = held + lane; j < want; j += 32)
      p.table[b * p.ld_table + j] = p.free_pages[n_free - 1 - (first[b] + j - held)];
  }
  // slots: a thread per token
  const int total = start[p.B];
  for (int64_t t = (int64_t)blockIdx.x * kPlanThreads + tid; t < p.T; t += (int64_t)gridDim.x * kPlanThreads) {
    int slot = -1;
    if (t < total) {
      int lo = 0, hi = p.B;  // the last request that starts at or before t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= t) lo = mid;
        else hi = mid;
      }
      if (first[lo] >= 0) {
        const int c = p.ctx[lo];
        const int pos = c + (int)(t - start[lo]);
        const int held = pages_of(c, p.shift), j = pos >> p.shift;
        const int page =
            j < held ? p.table[lo * p.ld_table + j] : p.free_pages[n_free - 1 - (first[lo] + j - held)];
        slot = page < 0 ? -1 : (int)(((int64_t)page << p.shift) + (pos & ((1 << p.shift) - 1)));
      }
    }
    p.slot_map[t] = slot;
  }
}

// ---------------------------------------------------------------------------
// kv_append
//
// One team (a warp, or a CTA of eight) per run of consecutive slots, head and
// cache half: the run's amax, the block's exponent, then the codes.
// ---------------------------------------------------------------------------

constexpr int kAppendThreads = 256;

struct AppendParams {
  const void *k, *v;
  int64_t ld_k, ld_v;
  const int32_t* slots;
  uint8_t *k_codes, *k_exps, *v_codes, *v_exps;
  int32_t* dev_status;
  int64_t num_slots;
  int T, Hkv, shift;
};

template <typename X>
__device__ __forceinline__ void load8(const X* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// The block exponent of a largest magnitude: the smallest e in [-127, 127]
// with amax <= 448 * 2^e; 448 = 1.75 * 2^8, so e is the fp32 exponent less 8,
// one more where the significand is above 1.75.
__device__ __forceinline__ int block_exponent(float amax) {
  const uint32_t u = __float_as_uint(fminf(amax, 3.402823466e38f));
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e < -127 ? -127 : e;  // zeros and subnormals too
}

template <typename X, int D>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendParams p) {
  constexpr int LPR = D / 8;        // lanes of a row, eight elements each
  constexpr int RPW = 32 / LPR;     // rows of a warp's access
  const int lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  // one warp per (token, head, half); tokens inside a run leave at once
  const int64_t item = ((int64_t)blockIdx.x * kAppendThreads + threadIdx.x) >> 5;
  if (item >= (int64_t)p.T * p.Hkv * 2) return;
  const int half = (int)(item & 1), head = (int)((item >> 1) % p.Hkv), t = (int)((item >> 1) / p.Hkv);
  const int32_t slot = p.slots[t];
  const int S = 1 << p.shift;
  if (slot < 0) return;
  if (slot >= p.num_slots) {
    if (lane == 0) report_status(p.dev_status, NVFP4_E_BAD_PAGE);
    return;
  }
  const int o = slot & (S - 1);
  if (o > 0 && t > 0 && p.slots[t - 1] == slot - 1) return;
  int n = 1;
  while (o + n < S && t + n < p.T && p.slots[t + n] == slot + n) ++n;

  const X* x = static_cast<const X*>(half ? p.v : p.k) + (int64_t)t * (half ? p.ld_v : p.ld_k) + head * D;
  const int64_t ld = half ? p.ld_v : p.ld_k;
  const int64_t block = (int64_t)(slot >> p.shift) * p.Hkv + head;
  uint8_t* codes = (half ? p.v_codes : p.k_codes) + block * S * D;
  uint8_t* exps = (half ? p.v_exps : p.k_exps) + block;
  const int r0 = lane / LPR, c0 = (lane % LPR) * 8;

  float amax = 0.0f;
  for (int r = r0; r < n; r += RPW) {
    float v[8];
    load8<X>(x + r * ld + c0, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
  int e = block_exponent(amax);
  if (o > 0) {
    const int e0 = (int)*exps - 127;
    if (e > e0) {
      const float f = exp2_int(e0 - e < -127 ? -127 : e0 - e);
      for (int r = r0; r < o; r += RPW) {
        uint2* w = reinterpret_cast<uint2*>(codes + r * D + c0);
        const uint2 was = *w;
        *w = make_uint2(kv::rescale_codes(was.x, f), kv::rescale_codes(was.y, f));
      }
    } else {
      e = e0;
    }
  }
  const float f = exp2_int(-e);
  for (int r = r0; r < n; r += RPW) {
    float v[8];
    load8<X>(x + r * ld + c0, v);
    *reinterpret_cast<uint2*>(codes + (int64_t)(o + r) * D + c0) =
        make_uint2(kv::encode4(v[0] * f, v[1] * f, v[2] * f, v[3] * f),
                   kv::encode4(v[4] * f, v[5] * f, v[6] * f, v[7] * f));
  }
  __syncwarp();  // every lane has read the old exponent
  if (lane == 0) *exps = (uint8_t)(e + 127);
}

}  // namespace

cudaError_t launch_kv_plan(const int32_t* ctx, const int32_t* add, int B, int page_size, int32_t* table,
                           int64_t ld_table, int M, const int32_t* free_pages, int num_free,
                           const int32_t* free_count, int T, int32_t* query_start, int32_t* kv_lens,
                           int32_t* slot_map, int32_t* free_left, int32_t* dev_status, cudaStream_t st) {
  PlanParams p = {ctx, add, table, free_pages, free_count, query_start, kv_lens, slot_map, free_left, dev_status,
                  ld_table, B, M, num_free, T, kv::log2_page(page_size)};
  const int smem = (2 * B + 1) * (int)sizeof(int32_t);
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kv_plan_kernel),
                                            (2 * kMaxKvRequests + 1) * (int)sizeof(int32_t));
  if (e != cudaSuccess) return e;
  int64_t grid = ((int64_t)T + kPlanThreads - 1) / kPlanThreads;
  grid = grid < 1 ? 1 : (grid > num_sms() ? num_sms() : grid);
  return launch_pdl(kv_plan_kernel, (int)grid, kPlanThreads, smem, st, p);
}

cudaError_t launch_kv_append(const void* k, const void* v, int x_dtype, int64_t ld_k, int64_t ld_v,
                             const int32_t* slots, int T, int Hkv, int D, int64_t num_pages, int page_size,
                             uint8_t* k_codes, uint8_t* k_exps, uint8_t* v_codes, uint8_t* v_exps,
                             int32_t* dev_status, cudaStream_t st) {
  AppendParams p = {k, v, ld_k, ld_v, slots, k_codes, k_exps, v_codes, v_exps, dev_status, num_pages * page_size,
                    T, Hkv, kv::log2_page(page_size)};
  const int64_t warps = (int64_t)T * Hkv * 2;
  const unsigned grid = (unsigned)((warps * 32 + kAppendThreads - 1) / kAppendThreads);
  if (x_dtype == NVFP4_DT_BF16)
    return D == 128 ? launch_pdl(kv_append_kernel<__nv_bfloat16, 128>, grid, kAppendThreads, 0, st, p)
                    : launch_pdl(kv_append_kernel<__nv_bfloat16, 64>, grid, kAppendThreads, 0, st, p);
  return D == 128 ? launch_pdl(kv_append_kernel<float, 128>, grid, kAppendThreads, 0, st, p)
                  : launch_pdl(kv_append_kernel<float, 64>, grid, kAppendThreads, 0, st, p);
}

}  // namespace nvfp4moe
