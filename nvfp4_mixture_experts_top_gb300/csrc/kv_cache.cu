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
// A CTA per chunk of tokens, head and half of the cache: it finds the runs of
// consecutive slots in a page that start there, and of each run the largest magnitude,
// the block's exponent, then the codes.  A run of up to kShortRun rows is one warp's,
// a longer one the whole CTA's, with its rows in registers in between.
// ---------------------------------------------------------------------------

constexpr int kAppendThreads = 256;  // 512 for pages of 128 rows of 128
constexpr int kShortRun = 8;
constexpr int kRunWords = 5;         // 32 tokens each: a chunk and 127 rows after its last token

struct AppendParams {
  const void *k, *v;
  int64_t ld_k, ld_v;
  const int32_t* slots;
  uint8_t *k_codes, *k_exps, *v_codes, *v_exps;
  int32_t* dev_status;
  int64_t num_slots;
  int T, Hkv, shift, chunk_shift;
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

// Where a run goes.
template <typename X, int D>
struct Run {
  const X* x;
  int64_t ld;
  uint8_t *codes, *exps;
  int o, e0;  // its first row in the page; the block's exponent if it holds rows before
  __device__ __forceinline__ Run(const AppendParams& p, int t, int32_t slot, int head, int half) {
    const int S = 1 << p.shift;
    ld = half ? p.ld_v : p.ld_k;
    x = static_cast<const X*>(half ? p.v : p.k) + (int64_t)t * ld + head * D;
    const int64_t block = (int64_t)(slot >> p.shift) * p.Hkv + head;
    codes = (half ? p.v_codes : p.k_codes) + block * S * D;
    exps = (half ? p.v_exps : p.k_exps) + block;
    o = slot & (S - 1);
    e0 = o > 0 ? (int)*exps - 127 : -127;
  }
  // the block's exponent after the run; rescales the rows before it (rows r0, r0 + step, ...)
  __device__ __forceinline__ int settle(float amax, int r0, int step, int c0) const {
    const int e = block_exponent(amax);
    if (e <= e0 || o == 0) return max(e, e0);
    const float f = exp2_int(e0 - e < -127 ? -127 : e0 - e);
#pragma unroll 4
    for (int r = r0; r < o; r += step) {
      uint2* w = reinterpret_cast<uint2*>(codes + r * D + c0);
      const uint2 was = *w;
      *w = make_uint2(kv::rescale_codes(was.x, f), kv::rescale_codes(was.y, f));
    }
    return e;
  }
  __device__ __forceinline__ void put(int r, int c0, const float (&v)[8], float f) const {
    *reinterpret_cast<uint2*>(codes + (o + r) * D + c0) =
        make_uint2(kv::encode4(v[0] * f, v[1] * f, v[2] * f, v[3] * f),
                   kv::encode4(v[4] * f, v[5] * f, v[6] * f, v[7] * f));
  }
};

template <typename X, int D>
__global__ void __launch_bounds__(512) kv_append_kernel(const AppendParams p) {
  constexpr int LPR = D / 8;  // lanes of a row, eight elements each
  __shared__ float tops[16];
  __shared__ int32_t slot_of[32];
  __shared__ uint32_t starts_s, goes_on[kRunWords + 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
  const int half = blockIdx.x & 1, head = (int)(blockIdx.x >> 1) % p.Hkv;
  const int first = (int)((blockIdx.x >> 1) / p.Hkv) << p.chunk_shift;
  const int c0 = (lane % LPR) * 8;
  pdl_wait();
  pdl_trigger();
  // the tokens that start a run and those that go on with one, a word per warp
  if (warp <= kRunWords) {
    const int tl = first + warp * 32 + lane;
    const bool there = warp < kRunWords && tl < p.T;
    const int32_t slot = there ? p.slots[tl] : -1, before = there && tl > 0 ? p.slots[tl - 1] : -1;
    const bool goes = slot >= 0 && (slot & ((1 << p.shift) - 1)) != 0 && before == slot - 1;
    const uint32_t on = __ballot_sync(0xFFFFFFFFu, goes);
    if (lane == 0) goes_on[warp] = on;
    if (warp == 0) {
      const bool begins = slot >= 0 && !goes && lane < 1 << p.chunk_shift, bad = begins && slot >= p.num_slots;
      if (bad) report_status(p.dev_status, NVFP4_E_BAD_PAGE);
      const uint32_t starts = __ballot_sync(0xFFFFFFFFu, begins && !bad);
      if (lane == 0) starts_s = starts;
      slot_of[lane] = slot;
    }
  }
  __syncthreads();
  const uint32_t starts = starts_s;
  auto length = [&](int i) {
    int at = i + 1;
    for (;;) {
      const int c = __ffs(~(goes_on[at >> 5] >> (at & 31))) - 1;  // (ones end with the word at the latest)
      if (c >= 0) at += min(c, 32 - (at & 31));
      else at += 32;
      if ((at & 31) != 0 || !(goes_on[at >> 5] & 1)) return at - i;
    }
  };

  int turn = 0;
  for (uint32_t todo = starts; todo; todo &= todo - 1) {
    const int i = __ffs(todo) - 1;
    const int32_t slot = slot_of[i];
    if (turn++ % warps != warp) continue;
    const int n = length(i);
    if (n > kShortRun) continue;
    constexpr int RPW = 32 / LPR, M = kShortRun / RPW;
    const Run<X, D> run(p, first + i, slot, head, half);
    const int r0 = lane / LPR;
    float v[M][8], amax = 0.0f;
#pragma unroll
    for (int k = 0; k < M; ++k) {
      if (r0 + k * RPW < n) {
        load8<X>(run.x + (r0 + k * RPW) * run.ld + c0, v[k]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] = 0.0f;
      }
    }
#pragma unroll
    for (int k = 0; k < M; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[k][j]));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
    const int e = run.settle(amax, r0, RPW, c0);
    const float f = exp2_int(-e);
#pragma unroll
    for (int k = 0; k < M; ++k)
      if (r0 + k * RPW < n) run.put(r0 + k * RPW, c0, v[k], f);
    __syncwarp();  // every lane has read the old exponent
    if (lane == 0) *run.exps = (uint8_t)(e + 127);
  }

  for (uint32_t todo = starts; todo; todo &= todo - 1) {
    const int i = __ffs(todo) - 1;
    const int32_t slot = slot_of[i];
    const int n = length(i);
    if (n <= kShortRun) continue;
    constexpr int M = 4, W = sizeof(X) / 2;
    const int RPC = blockDim.x / LPR;  // (at least a quarter of a page)
    const Run<X, D> run(p, first + i, slot, head, half);
    const int r0 = tid / LPR;
    uint4 w[M][W];
#pragma unroll
    for (int k = 0; k < M; ++k)
#pragma unroll
      for (int j = 0; j < W; ++j)
        w[k][j] = r0 + k * RPC < n ? reinterpret_cast<const uint4*>(run.x + (r0 + k * RPC) * run.ld + c0)[j]
                                   : make_uint4(0, 0, 0, 0);
    float amax = 0.0f;
#pragma unroll
    for (int k = 0; k < M; ++k) {
      float v[8];
      load8<X>(reinterpret_cast<const X*>(w[k]), v);
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
    if (lane == 0) tops[warp] = amax;
    __syncthreads();  // (every thread has read the old exponent)
#pragma unroll
    for (int k = 0; k < 16; ++k) amax = fmaxf(amax, k < warps ? tops[k] : 0.0f);
    const int e = run.settle(amax, r0, RPC, c0);
    const float f = exp2_int(-e);
#pragma unroll
    for (int k = 0; k < M; ++k) {
      float v[8];
      load8<X>(reinterpret_cast<const X*>(w[k]), v);
      if (r0 + k * RPC < n) run.put(r0 + k * RPC, c0, v, f);
    }
    if (tid == 0) *run.exps = (uint8_t)(e + 127);
    __syncthreads();  // (tops is read)
  }
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
                    T, Hkv, kv::log2_page(page_size), 0};
  // 32 tokens per CTA where that fills the GPU, else 8, one per warp
  p.chunk_shift = ((int64_t)T >> 5) * Hkv * 2 >= num_sms() ? 5 : 3;
  const int64_t chunks = ((int64_t)T + (1 << p.chunk_shift) - 1) >> p.chunk_shift;
  const unsigned grid = (unsigned)(chunks * Hkv * 2);
  const int threads = page_size * D > 8192 ? 512 : kAppendThreads;  // four rows of a page per thread
  if (x_dtype == NVFP4_DT_BF16)
    return D == 128 ? launch_pdl(kv_append_kernel<__nv_bfloat16, 128>, grid, threads, 0, st, p)
                    : launch_pdl(kv_append_kernel<__nv_bfloat16, 64>, grid, threads, 0, st, p);
  return D == 128 ? launch_pdl(kv_append_kernel<float, 128>, grid, threads, 0, st, p)
                  : launch_pdl(kv_append_kernel<float, 64>, grid, threads, 0, st, p);
}

}  // namespace nvfp4moe
