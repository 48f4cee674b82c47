// kv_attention.cu -- attention over the paged 8-bit key/value cache:
//   s_j = scale * q . k_j,   out = sum_j softmax(s)_j v_j,   lse = ln sum_j exp s_j
// for few query rows per request and K/V head (single tokens, drafted tokens).
//
// Bound: every cached byte of a request is read once for all query heads of a
// K/V head; 2 * D bytes and 4 * D * rows flops per key leave HBM as the limit
// up to some tens of rows.  So the kernel is built to keep loads in flight:
//  - the work is cut into units of 128 keys of one (request, K/V head, row
//    tile), and the CTAs that fit on the GPU take equal ranges of all units,
//    whatever the lengths.  A CTA that ends inside a sequence leaves a partial
//    result, and a small second kernel joins them in order (no atomics: the
//    result repeats bit for bit);
//  - one warp of a CTA does nothing but page lookups and copies: it fills a
//    ring of 32-key tiles by TMA and runs ahead of the arithmetic across the
//    ends of sequences; the other warps take tiles in turn, each with its own
//    running maximum, sum and output;
//  - arithmetic is mma.sync m16n8k16 on f16 with fp32 accumulation: every E4M3
//    value is an f16 value, and a query row is carried as f16 with its own
//    power of two.  Keys (and the head dimension of V) are the 16-row side and
//    query rows the 8-column side, so 8 rows cost half of what 16 do.  tcgen05
//    would need the operands converted through shared or tensor memory for
//    less than a tenth of its rate.
// Softmax statistics and outputs are fp32.  Weights are rounded to f16 after a
// shift by 2^12 (so that they keep 11 bits down to 2^-26 of the largest).
#include <cuda.h>

#include "common.cuh"
#include "kernels.h"
#include "kv.cuh"
#include "tmap.h"

namespace nvfp4moe {
namespace {

constexpr int kTile = 32;                 // keys of a warp's step
constexpr int kWholeKeys = 512;           // sequences up to this long are not split
constexpr float kBoost = 12.0f;           // log2 of the weights' shift
constexpr int kFarExp = -60;              // value blocks further below the largest one count as this far

// The sequence -- request, K/V head, row tile -- that a CTA's range starts in,
// for the join: units of it before the range, units of it in all, its first
// output row (token * group + head in group), K/V head and rows.
struct Cut {
  int32_t before, span, row, head, rows, pad[3];
};

struct Params {
  const __nv_bfloat16* q;
  const uint8_t *k_exps, *v_exps;
  const int32_t *table, *kv_lens, *query_start;
  __nv_bfloat16* out;
  float* lse;
  int32_t* dev_status;
  float* part;      // [CTA][2][rows][D] partial outputs
  float* part_lse;  // [CTA][2][rows] their log2-sums
  Cut* cut;         // [CTA]
  int64_t* total;   // units of the whole call
  int64_t ld_q, ld_table, num_pages;
  int M, T, B, Hq, Hkv, shift;
  float scale;
};

// A request as the kernel sees it: lengths cut to what the table, q and out hold.
struct Request {
  int q0, n, kv;
  bool bad;
};
__device__ __forceinline__ Request get_request(const Params& p, int b) {
  Request r;
  const int a = p.query_start[b], e = p.query_start[b + 1], kv = p.kv_lens[b];
  r.q0 = min(max(a, 0), p.T);
  const int q1 = min(max(e, r.q0), p.T);
  r.n = q1 - r.q0;
  const int64_t cap = (int64_t)p.M << p.shift;
  r.kv = kv < 0 ? 0 : (kv > cap ? (int)cap : kv);
  r.bad = r.q0 != a || q1 != e || r.kv != kv;
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// D += A B, A [16 x 16] f16 (row), B [16 x 8] f16 (column), fp32 accumulators.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transpose of an 8 x 8 matrix of 16-bit elements held two to a lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Byte offset of 16-byte chunk c of key row r in a tile's [32][D] codes, as the
// TMA's 128-byte (D = 64: 64-byte) swizzle places it.
template <int D>
__device__ __forceinline__ uint32_t tile_offset(int r, int c) {
  return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ (r >> 1 & 3)) << 4);
}
// Key of row i (0..7) of an eight-key MMA block.  Any order of the keys gives
// the same sums as long as K and V agree; with this one both access patterns of
// the swizzled tile are free of bank conflicts: K (lane (g, t) reads the row of
// key g, chunks t and t + 4) and V (rows of keys 2t and 2t + 1, chunk g).
template <int D>
__device__ __forceinline__ int key_of(int i) {
  return D == 128 ? i ^ ((i & 1) << 2) : (i & 4) | ((i & 1) << 1) | ((i >> 1 ^ i) & 1);
}

template <int D, int NT>
struct Geo {
  static constexpr int ROWS = 8 * NT;
  // warps that compute: with the copying one, two CTAs give each of an SM's
  // four schedulers four warps of 128 registers (three of 168)
  static constexpr int WARPS = D * NT > 128 ? 5 : 7;
  static constexpr int THREADS = (WARPS + 1) * 32;
  static constexpr int CTAS = 2;                       // of an SM
  static constexpr int UNIT = WARPS * kTile;           // keys of a work unit
  static constexpr int TILE_BYTES = kTile * D;         // codes of K or of V
  static constexpr int SLOT_BYTES = 2 * TILE_BYTES;
  static constexpr int JOIN_BYTES = WARPS * ROWS * D * 4;
  static constexpr int SLOTS = (111 * 1024 + D * 8 - JOIN_BYTES) / SLOT_BYTES;
  static constexpr int RING_BYTES = SLOTS * SLOT_BYTES;
  static constexpr int SMEM_BYTES = RING_BYTES + JOIN_BYTES;
  // "full" barriers are a ring of their own, a whole number of laps of the
  // warps: the use of a barrier before a warp's next tile is then a tile of the
  // same warp, so the phase it waits for is never two ahead.  (With a barrier
  // per slot it could be: copies finish out of order.)
  static constexpr int FULLS = (SLOTS + WARPS - 1) / WARPS * WARPS;
  static_assert(WARPS < SLOTS && FULLS <= 32, "ring sizes");
};

// The pieces of sequences that a CTA's range of the work consists of, in order.
template <int D, int NT>
struct Pieces {
  int b;          // request
  int64_t off;    // of the range in the request's work
  int64_t pos, hi;
  bool split;
  // the current piece
  Request rq;
  int hk, row0, rows, nrows, span, u0, take;
  int limit;      // keys that the last row of the tile sees
  int t0, t1;     // its tiles

  __device__ __forceinline__ static int units(int kv) {
    return kv > Geo<D, NT>::UNIT ? (kv + Geo<D, NT>::UNIT - 1) / Geo<D, NT>::UNIT : 1;
  }
  __device__ __forceinline__ static int64_t row_tiles(int n, int group) {
    return ((int64_t)n * group + Geo<D, NT>::ROWS - 1) / Geo<D, NT>::ROWS;
  }
  __device__ __forceinline__ bool next(const Params& p, int group) {
    while (pos < hi && b < p.B) {
      rq = get_request(p, b);
      const int tiles = (int)row_tiles(rq.n, group);
      span = split ? units(rq.kv) : 1;
      if (off >= (int64_t)tiles * p.Hkv * span) {
        ++b;
        off = 0;
        continue;
      }
      const int seq = (int)(off / span);
      u0 = (int)(off - (int64_t)seq * span);
      take = (int)min((int64_t)(span - u0), hi - pos);
      hk = seq / tiles;
      row0 = (seq - hk * tiles) * Geo<D, NT>::ROWS;
      rows = rq.n * group;
      nrows = min(Geo<D, NT>::ROWS, rows - row0);
      limit = min(rq.kv, rq.kv - rq.n + (row0 + nrows - 1) / group + 1);
      const int end = limit > 0 ? (limit + kTile - 1) / kTile : 0;
      t0 = split ? u0 * Geo<D, NT>::WARPS : 0;
      t1 = split ? min((u0 + take) * Geo<D, NT>::WARPS, end) : end;
      pos += take;
      off += take;
      return true;
    }
    return false;
  }
};

template <int D, int NT>
__global__ void __launch_bounds__((Geo<D, NT>::THREADS), (Geo<D, NT>::CTAS))
    kv_attention_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const Params p) {
  using G = Geo<D, NT>;
  using P = Pieces<D, NT>;
  constexpr int ROWS = G::ROWS, WARPS = G::WARPS, SLOTS = G::SLOTS, FULLS = G::FULLS, ALL = WARPS + 1;
  constexpr int NQ = D / 16;   // MMA steps over the head dimension
  constexpr int NV = D / 16;   // 16-row blocks of V^T
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(8) uint64_t full_bar[FULLS], empty_bar[SLOTS];
  __shared__ uint2 head[SLOTS];  // exponent bytes of a slot's two halves; bit h: half h has no page
  __shared__ int64_t s_sum[2][ALL], s_off;
  __shared__ int s_long[ALL], s_b;
  __shared__ float s_m[WARPS][ROWS], s_l[WARPS][ROWS];
  __shared__ int s_u[WARPS];
  __shared__ volatile int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3, kg = key_of<D>(g);
  const int group = p.Hq / p.Hkv;
  if (tid == 0) {
    for (int i = 0; i < FULLS; ++i) mbar_init(&full_bar[i], 1);
    for (int i = 0; i < SLOTS; ++i) mbar_init(&empty_bar[i], 1);
    abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  pdl_wait();
  pdl_trigger();

  // ---- the CTA's range of the work: units if some sequence is longer than
  // kWholeKeys, else whole sequences (nothing to join then)
  P it;
  {
    const int per = (p.B + G::THREADS - 1) / G::THREADS;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    int64_t seqs = 0, units = 0;
    int longest = 0;
    for (int b = b0; b < b1; ++b) {
      const Request r = get_request(p, b);
      const int64_t n = P::row_tiles(r.n, group) * p.Hkv;
      seqs += n;
      units += n * P::units(r.kv);
      if (n) longest = max(longest, r.kv);
      if (blockIdx.x == 0 && r.bad) report_status(p.dev_status, NVFP4_E_BAD_PAGE);
    }
    int64_t in_s = seqs, in_u = units;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t a = __shfl_up_sync(0xFFFFFFFFu, in_s, d), c = __shfl_up_sync(0xFFFFFFFFu, in_u, d);
      if (lane >= d) {
        in_s += a;
        in_u += c;
      }
      longest = max(longest, __shfl_xor_sync(0xFFFFFFFFu, longest, d));
    }
    if (lane == 31) {
      s_sum[0][warp] = in_s;
      s_sum[1][warp] = in_u;
      s_long[warp] = longest;
    }
    __syncthreads();
    for (int w = 0; w < ALL; ++w) longest = max(longest, s_long[w]);
    it.split = longest > kWholeKeys;
    int64_t total = 0, before = it.split ? in_u - units : in_s - seqs;
    for (int w = 0; w < ALL; ++w) {
      const int64_t x = s_sum[it.split ? 1 : 0][w];
      total += x;
      if (w < warp) before += x;
    }
    it.pos = total * blockIdx.x / gridDim.x;
    it.hi = total * (blockIdx.x + 1) / gridDim.x;
    if (it.pos < it.hi && before <= it.pos && it.pos < before + (it.split ? units : seqs)) {
      for (int b = b0; b < b1; ++b) {
        const Request r = get_request(p, b);
        const int64_t w = P::row_tiles(r.n, group) * p.Hkv * (it.split ? P::units(r.kv) : 1);
        if (it.pos < before + w) {
          s_b = b;
          s_off = it.pos - before;
          break;
        }
        before += w;
      }
    }
    __syncthreads();
    if (blockIdx.x == 0 && tid == 0) *p.total = total;
    if (it.pos >= it.hi) {
      if (tid == 0) p.cut[blockIdx.x].before = 0;
      return;
    }
    it.b = s_b;
    it.off = s_off;
  }

  if (warp == WARPS) {
    // ------------------------------------------------------------ copies
    const int S = 1 << p.shift;
    int slot = 0, full = 0;
    uint32_t phase = 1, full_phase = 0, issued = 0, issued_par = 0;
    bool ok = true;
    while (ok && it.next(p, group)) {
      const int32_t* table = p.table + it.b * p.ld_table;
      int page_a = -1, page_b = -1;  // of 32 tiles, one per lane (two pages where they hold 16 keys)
      uint32_t exps = 0;
      for (int tile = it.t0; tile < it.t1; ++tile) {
        const int j = (tile - it.t0) & 31;
        if (j == 0) {
          page_a = page_b = -1;
          exps = 0;
          if (tile + lane < it.t1) {
            const int key = (tile + lane) * kTile;
            page_a = table[key >> p.shift];
            page_b = p.shift == 4 && key + 16 < it.limit ? table[(key >> p.shift) + 1] : page_a;
            if (page_a < 0 || page_a >= p.num_pages) page_a = -1;
            if (page_b < 0 || page_b >= p.num_pages) page_b = -1;
            if (page_a < 0 || page_b < 0) report_status(p.dev_status, NVFP4_E_BAD_PAGE);
            if (page_a >= 0) {
              const int64_t at = (int64_t)page_a * p.Hkv + it.hk;
              exps = p.k_exps[at] | (uint32_t)p.v_exps[at] << 8;
            }
            if (page_b >= 0) {
              const int64_t at = (int64_t)page_b * p.Hkv + it.hk;
              exps |= (uint32_t)p.k_exps[at] << 16 | (uint32_t)p.v_exps[at] << 24;
            }
          }
        }
        const int pa = __shfl_sync(0xFFFFFFFFu, page_a, j), pb = __shfl_sync(0xFFFFFFFFu, page_b, j);
        if (!warp_wait(&empty_bar[slot], phase, &abort_flag, p.dev_status)) {
          ok = false;
          break;
        }
        const int key0 = tile * kTile;
        uint8_t* dst = smem + slot * G::SLOT_BYTES;
        const int pages = p.shift == 4 ? 2 : 1;  // boxes of a tile
        const uint32_t bytes = p.shift == 4 ? (uint32_t)G::SLOT_BYTES / 2 : (uint32_t)G::SLOT_BYTES;
        const uint32_t ex = __shfl_sync(0xFFFFFFFFu, exps, j);
        if (lane == 0) head[slot] = make_uint2(ex, (pa < 0 ? 1u : 0u) | (pb < 0 ? 2u : 0u));
        __syncwarp();
        ew_arrive_expect_tx(&full_bar[full], (pa >= 0 ? bytes : 0) + (pages == 2 && pb >= 0 ? bytes : 0));
        if (pa >= 0) {
          const int block = pa * p.Hkv + it.hk, row = key0 & (S - 1);
          kv::ew_tma_load_3d(dst, &tm_k, &full_bar[full], 0, row, block);
          kv::ew_tma_load_3d(dst + G::TILE_BYTES, &tm_v, &full_bar[full], 0, row, block);
        }
        if (pages == 2 && pb >= 0) {
          const int block = pb * p.Hkv + it.hk;
          kv::ew_tma_load_3d(dst + G::TILE_BYTES / 2, &tm_k, &full_bar[full], 0, 0, block);
          kv::ew_tma_load_3d(dst + G::TILE_BYTES * 3 / 2, &tm_v, &full_bar[full], 0, 0, block);
        }
        issued |= 1u << full;
        issued_par = (issued_par & ~(1u << full)) | (full_phase << full);
        if (++full == FULLS) {
          full = 0;
          full_phase ^= 1;
        }
        if (++slot == SLOTS) {
          slot = 0;
          phase ^= 1;
        }
      }
    }
    if (!ok) {  // given up: wait for the copies in flight before the CTA's memory goes
      for (int i = 0; i < FULLS; ++i)
        if (issued >> i & 1) mbar_wait(&full_bar[i], issued_par >> i & 1);
    }
    return;
  }

  // -------------------------------------------------------------- arithmetic
  int slot = warp, full = warp;  // of this warp's next tile
  uint32_t full_phase = 0;
  int turn = warp;              // tiles of the CTA until this warp's next one
  bool first = true, ok = true;
  while (it.next(p, group)) {
    if (first && tid == 0)
      p.cut[blockIdx.x] = {it.split ? it.u0 : 0, it.span, it.rq.q0 * group + it.row0, it.hk, it.nrows, {0, 0, 0}};

    // query rows: lane (g, t) holds row g's elements for its keys' chunks, as
    // f16 times the row's power of two
    uint32_t qf[NT][NQ][2];
    float qs[NT][2];     // log2 logit per accumulator unit, rows 2t and 2t + 1
    int lim[NT][2];      // keys that the row sees
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = it.row0 + n * 8 + g;
      float v[D / 4], amax = 0.0f;
      const __nv_bfloat16* src =
          p.q + (int64_t)(it.rq.q0 + r / group) * p.ld_q + (int64_t)(it.hk * group + r % group) * D + 16 * t;
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        uint4 w[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if (r < it.rows) {
          w[0] = *reinterpret_cast<const uint4*>(src + 64 * h);
          w[1] = *reinterpret_cast<const uint4*>(src + 64 * h + 8);
        }
        const uint32_t x[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[h * 16 + 2 * i] = __uint_as_float(x[i] << 16);
          v[h * 16 + 2 * i + 1] = __uint_as_float(x[i] & 0xFFFF0000u);
        }
      }
#pragma unroll
      for (int i = 0; i < D / 4; ++i) amax = fmaxf(amax, fabsf(v[i]));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
      const int e = amax == 0.0f ? 0 : min(14 - floor_log2(amax), 126);
      const float f = exp2_int(e);
#pragma unroll
      for (int k = 0; k < NQ; ++k) {
        qf[n][k][0] = pack_f16(v[4 * k] * f, v[4 * k + 1] * f);
        qf[n][k][1] = pack_f16(v[4 * k + 2] * f, v[4 * k + 3] * f);
      }
      const float rs = p.scale * 1.4426950408889634f * exp2_int(-e);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        qs[n][c] = __shfl_sync(0xFFFFFFFFu, rs, (2 * t + c) * 4);
        const int rr = it.row0 + n * 8 + 2 * t + c;
        lim[n][c] = rr < it.rows ? min(it.rq.kv, it.rq.kv - it.rq.n + rr / group + 1) : 0;
      }
    }
    const int all_see = it.rq.kv - it.rq.n + it.row0 / group + 1;  // keys below this are seen by every row

    float o[NT][NV][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < NV; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.0f;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.0f;
    }
    int unit_exp = -127;  // outputs are held in units of 2^unit_exp, the largest value exponent so far

    int tile = it.t0 + turn;
    for (; tile < it.t1; tile += WARPS) {
      ok = ok && warp_wait(&full_bar[full], full_phase, &abort_flag, p.dev_status);
      const uint2 hd = head[slot];
      const uint8_t* kt = smem + slot * G::SLOT_BYTES;
      const uint8_t* vt = kt + G::TILE_BYTES;
      const int key0 = tile * kTile;
      const bool ragged = key0 + kTile > it.limit || hd.y;

      // S^T = K Q^T, two blocks of 16 keys
      float s[NT][2][4];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
        for (int n = 0; n < NT; ++n) s[n][kb][0] = s[n][kb][1] = s[n][kb][2] = s[n][kb][3] = 0.0f;
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          const uint4 ka = *reinterpret_cast<const uint4*>(kt + tile_offset<D>(kb * 16 + kg, h * 4 + t));
          const uint4 kc = *reinterpret_cast<const uint4*>(kt + tile_offset<D>(kb * 16 + kg + 8, h * 4 + t));
          const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wc[4] = {kc.x, kc.y, kc.z, kc.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a0 = kv::decode2((uint16_t)wa[i]), a2 = kv::decode2((uint16_t)(wa[i] >> 16));
            const uint32_t a1 = kv::decode2((uint16_t)wc[i]), a3 = kv::decode2((uint16_t)(wc[i] >> 16));
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma16816(s[n][kb], a0, a1, a2, a3, qf[n][h * 4 + i][0], qf[n][h * 4 + i][1]);
          }
        }
      }
      // logits in log2 units; keys that a row does not see are -inf
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        const float ks = exp2_int((int)(hd.x >> (16 * kb) & 255) - 127);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[n][kb][c] = s[n][kb][c] * qs[n][c & 1] * ks;
      }
      if (key0 + kTile > all_see || hd.y) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (key0 + kb * 16 + kg + (c >> 1) * 8 >= lim[n][c & 1] || (hd.y >> kb & 1)) s[n][kb][c] = -INFINITY;
      }
      // value exponents of the two blocks relative to the largest so far
      const int va = hd.y & 1 ? -127 : (int)(hd.x >> 8 & 255) - 127, vb = hd.y & 2 ? -127 : (int)(hd.x >> 24) - 127;
      const int ue = max(unit_exp, max(va, vb));
      const float vs[2] = {exp2_int(max(va - ue, kFarExp)), exp2_int(max(vb - ue, kFarExp))};
      const float us = exp2_int(max(unit_exp - ue, -127));
      unit_exp = ue;
      uint32_t pf[NT][2][2];  // weights as the MMA's 16 x 8 operand
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float f[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float mx = fmaxf(fmaxf(s[n][0][c], s[n][0][c + 2]), fmaxf(s[n][1][c], s[n][1][c + 2]));
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
          const float m1 = fmaxf(m[n][c], mx), ms = m1 == -INFINITY ? 0.0f : m1;
          f[c] = ex2(m[n][c] - ms);
          m[n][c] = m1;
          float sum = 0.0f;
#pragma unroll
          for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int d = 0; d < 4; d += 2) {
              const float w = ex2(s[n][kb][c + d] - ms + kBoost);
              sum += w;
              s[n][kb][c + d] = w * vs[kb];
            }
          l[n][c] = l[n][c] * f[c] + sum;
          f[c] *= us;
        }
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          pf[n][kb][0] = transpose8x8(pack_f16(s[n][kb][0], s[n][kb][1]));
          pf[n][kb][1] = transpose8x8(pack_f16(s[n][kb][2], s[n][kb][3]));
        }
        if (__any_sync(0xFFFFFFFFu, f[0] != 1.0f || f[1] != 1.0f)) {
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            o[n][i][0] *= f[0];
            o[n][i][1] *= f[1];
            o[n][i][2] *= f[0];
            o[n][i][3] *= f[1];
          }
        }
      }
      // O^T += V^T P^T: lane (g, t) reads D / 8 elements of keys 2t, 2t+1, 2t+8, 2t+9
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        constexpr int NW = D / 32;  // 4-byte words of a lane's elements of a key
        uint32_t w[4][NW];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = kb * 16 + key_of<D>(2 * t + (i & 1)) + (i >> 1) * 8;
          if constexpr (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(vt + tile_offset<D>(r, g));
            w[i][0] = x.x, w[i][1] = x.y, w[i][2] = x.z, w[i][3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(vt + tile_offset<D>(r, g >> 1) + (g & 1) * 8);
            w[i][0] = x.x, w[i][1] = x.y;
          }
          // rows past the sequence hold anything, and 0 * NaN would spread
          if (ragged && (key0 + r >= it.limit || (hd.y >> kb & 1))) {
#pragma unroll
            for (int k = 0; k < NW; ++k) w[i][k] = 0;
          }
        }
#pragma unroll
        for (int i = 0; i < NW; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // elements 2h, 2h + 1 of word i: (key 2t, key 2t + 1) pairs of each
            const uint32_t x = __byte_perm(w[0][i], w[1][i], h ? 0x7362 : 0x5140);
            const uint32_t y = __byte_perm(w[2][i], w[3][i], h ? 0x7362 : 0x5140);
            const uint32_t a0 = kv::decode2((uint16_t)x), a1 = kv::decode2((uint16_t)(x >> 16));
            const uint32_t a2 = kv::decode2((uint16_t)y), a3 = kv::decode2((uint16_t)(y >> 16));
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816(o[n][2 * i + h], a0, a1, a2, a3, pf[n][kb][0], pf[n][kb][1]);
          }
      }
      __syncwarp();  // every lane has read the slot
      if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&empty_bar[slot])) : "memory");
      slot += WARPS;
      if (slot >= SLOTS) slot -= SLOTS;
      full += WARPS;
      if (full >= FULLS) {
        full = warp;
        full_phase ^= 1;
      }
    }
    turn = tile - max(it.t1, it.t0);

    // ---- join the warps: lane (g, t) holds D / 8 consecutive elements, from
    // g * D / 8, of rows 2t and 2t + 1
    float* join = reinterpret_cast<float*>(smem + G::RING_BYTES);
    constexpr int EL = D / 8;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float sum = l[n][c];
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 4);
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 8);
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 16);
        const int r = n * 8 + 2 * t + c;
        if (g == 0) {
          s_m[warp][r] = m[n][c];
          s_l[warp][r] = sum;
        }
        // four elements at a time, permuted within the row so that the lanes of
        // an access and the threads that read it spread over the banks
#pragma unroll
        for (int i = 0; i < EL / 4; ++i)
          *reinterpret_cast<float4*>(join + (warp * ROWS + r) * D + (((g * EL / 4 + i) ^ g ^ (t << 1)) << 2)) =
              make_float4(o[n][2 * i][c], o[n][2 * i][c + 2], o[n][2 * i + 1][c], o[n][2 * i + 1][c + 2]);
      }
    if (lane == 0) s_u[warp] = unit_exp;
    asm volatile("bar.sync 1, %0;" ::"n"(WARPS * 32) : "memory");
    const bool whole = it.take == it.span;
    const int64_t part = (int64_t)blockIdx.x * 2 + (first ? 0 : 1);
    int umax = s_u[0];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) umax = max(umax, s_u[w]);
    constexpr int TPR = D / 4;  // threads of a row, four elements each
    for (int r = tid / TPR; r < it.nrows; r += WARPS * 32 / TPR) {
      const int d4 = tid % TPR, d = d4 * 4, at4 = (d4 ^ (d4 / (EL / 4)) ^ (r & 6)) << 2;
      float mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) mx = fmaxf(mx, s_m[w][r]);
      const float ms = mx == -INFINITY ? 0.0f : mx;
      float sum = 0.0f;
      float4 acc = make_float4(0, 0, 0, 0);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float f = ex2(s_m[w][r] - ms), fu = f * exp2_int(max(s_u[w] - umax, -127));
        sum += s_l[w][r] * f;
        const float4 x = *reinterpret_cast<const float4*>(join + (w * ROWS + r) * D + at4);
        acc.x += x.x * fu, acc.y += x.y * fu, acc.z += x.z * fu, acc.w += x.w * fu;
      }
      const bool none = sum == 0.0f;
      const float inv = none ? 0.0f : 1.0f / sum, us = exp2_int(umax);
      acc = none ? make_float4(0, 0, 0, 0)
                 : make_float4(acc.x * inv * us, acc.y * inv * us, acc.z * inv * us, acc.w * inv * us);
      const float lse2 = none ? -INFINITY : mx + (log2f(sum) - kBoost);
      if (whole) {
        const int rr = it.row0 + r;
        const int64_t at = (int64_t)(it.rq.q0 + rr / group) * p.Hq + it.hk * group + rr % group;
        const __nv_bfloat162 lo2 = __floats2bfloat162_rn(acc.x, acc.y), hi2 = __floats2bfloat162_rn(acc.z, acc.w);
        *reinterpret_cast<uint2*>(p.out + at * D + d) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo2), *reinterpret_cast<const uint32_t*>(&hi2));
        if (p.lse != nullptr && d == 0) p.lse[at] = lse2 * 0.6931471805599453f;
      } else {
        *reinterpret_cast<float4*>(p.part + (part * ROWS + r) * D + d) = acc;
        if (d == 0) p.part_lse[part * ROWS + r] = lse2;
      }
    }
    asm volatile("bar.sync 1, %0;" ::"n"(WARPS * 32) : "memory");  // the join buffer is free again
    first = false;
  }
}

// Joins the partial results of a sequence, a CTA per row: CTA (c - 1, r) takes
// row r of the sequence that the range of CTA c starts in, if no range before c
// starts inside it.  Its four warps take parts in turn.
template <int D, int NT>
__global__ void __launch_bounds__(128) kv_attention_join_kernel(const Params p, int ctas) {
  constexpr int ROWS = Geo<D, NT>::ROWS;
  constexpr int E = D / 32;
  __shared__ float s_acc[4][D], s_top[4], s_sum[4];
  pdl_wait();
  pdl_trigger();
  const int c = blockIdx.x + 1, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = blockIdx.y;
  const Cut cut = p.cut[c];
  if (cut.before == 0 || r >= cut.rows) return;
  const int64_t W = *p.total;
  // unit u belongs to the last CTA whose range starts at or before it
  auto owner = [&](int64_t u) { return (int)(((u + 1) * ctas - 1) / W); };
  const int64_t a = W * c / ctas - cut.before, e = a + cut.span;
  const int c0 = owner(a);
  if (owner(a + cut.before - 1) != c0) return;
  // a part per CTA, or with fewer units than CTAs a part per unit; a CTA's
  // first piece is its part 0, its last one its part 1
  const int n = W >= ctas ? owner(e - 1) - c0 + 1 : cut.span;
  const int first = c0 * 2 + (W * c0 / ctas >= a ? 0 : 1);
  auto row_of = [&](int k) {
    const int part = k == 0 ? first : (W >= ctas ? c0 + k : owner(a + k)) * 2;
    return (int64_t)part * ROWS + r;
  };
  float top = -INFINITY, sum = 0.0f, acc[E] = {};
  for (int k0 = warp; k0 < n; k0 += 128) {  // lane i: part k0 + 4 i
    const int m = min(32, (n - k0 + 3) / 4);
    const int64_t row = row_of(min(k0 + 4 * lane, n - 1));
    const float z = lane < m ? p.part_lse[row] : -INFINITY;
    float mx = z;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
    const float t1 = fmaxf(top, mx), ms = t1 == -INFINITY ? 0.0f : t1, f = ex2(top - ms), w = ex2(z - ms);
    top = t1;
    sum = sum * f + w;
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] *= f;
#pragma unroll 8
    for (int k = 0; k < m; ++k) {
      const float wk = __shfl_sync(0xFFFFFFFFu, w, k);
      const float* src = p.part + __shfl_sync(0xFFFFFFFFu, row, k) * D + lane * E;
      float x[E];
      if constexpr (E == 4) {
        const float4 y = *reinterpret_cast<const float4*>(src);
        x[0] = y.x, x[1] = y.y, x[2] = y.z, x[3] = y.w;
      } else {
        const float2 y = *reinterpret_cast<const float2*>(src);
        x[0] = y.x, x[1] = y.y;
      }
#pragma unroll
      for (int i = 0; i < E; ++i) acc[i] += wk * x[i];
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
  if (lane == 0) {
    s_top[warp] = top;
    s_sum[warp] = sum;
  }
#pragma unroll
  for (int i = 0; i < E; ++i) s_acc[warp][lane * E + i] = acc[i];
  __syncthreads();
  const float mx = fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3])), ms = mx == -INFINITY ? 0.0f : mx;
  float total = 0.0f, out = 0.0f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float f = ex2(s_top[w] - ms);
    total += s_sum[w] * f;
    if (tid < D) out += s_acc[w][tid] * f;
  }
  const int group = p.Hq / p.Hkv, rr = cut.row + r;
  const int64_t at = (int64_t)(rr / group) * p.Hq + cut.head * group + rr % group;
  if (tid < D) p.out[at * D + tid] = __float2bfloat16(total == 0.0f ? 0.0f : out / total);
  if (p.lse != nullptr && tid == 0)
    p.lse[at] = total == 0.0f ? -INFINITY : (mx + log2f(total)) * 0.6931471805599453f;
}

template <int D, int NT>
size_t carve(Params* p, void* base) {
  using G = Geo<D, NT>;
  const size_t ctas = (size_t)num_sms() * G::CTAS;
  uint8_t* b = static_cast<uint8_t*>(base);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    uint8_t* at = b ? b + off : nullptr;
    off += (bytes + 255) & ~(size_t)255;
    return at;
  };
  uint8_t* total = take(sizeof(int64_t));
  uint8_t* cut = take(ctas * sizeof(Cut));
  uint8_t* lse = take(ctas * 2 * G::ROWS * sizeof(float));
  uint8_t* part = take(ctas * 2 * G::ROWS * D * sizeof(float));
  if (p != nullptr) {
    p->total = reinterpret_cast<int64_t*>(total);
    p->cut = reinterpret_cast<Cut*>(cut);
    p->part_lse = reinterpret_cast<float*>(lse);
    p->part = reinterpret_cast<float*>(part);
  }
  return off;
}

template <int D, int NT>
cudaError_t launch(const KvAttention& a, cudaStream_t st) {
  using G = Geo<D, NT>;
  Params p = {static_cast<const __nv_bfloat16*>(a.q), a.k_exps, a.v_exps, a.table, a.kv_lens,
              a.query_start, static_cast<__nv_bfloat16*>(a.out), a.lse, a.dev_status, nullptr, nullptr, nullptr,
              nullptr, a.ld_q, a.ld_table, a.num_pages, a.M, a.T, a.B, a.Hq, a.Hkv, kv::log2_page(a.page_size),
              a.scale};
  carve<D, NT>(&p, a.workspace);
  CUtensorMap tm_k, tm_v;
  const uint32_t box = a.page_size < kTile ? a.page_size : kTile;
  const uint64_t blocks = (uint64_t)a.num_pages * a.Hkv;
  if (make_tmap_3d_u8(&tm_k, a.k_codes, D, a.page_size, blocks, box, D) != cudaSuccess ||
      make_tmap_3d_u8(&tm_v, a.v_codes, D, a.page_size, blocks, box, D) != cudaSuccess)
    return cudaErrorInvalidValue;
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kv_attention_kernel<D, NT>), G::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  const int ctas = num_sms() * G::CTAS;
  e = launch_pdl(kv_attention_kernel<D, NT>, ctas, G::THREADS, G::SMEM_BYTES, st, tm_k, tm_v, p);
  // a table that holds no sequence long enough to be split needs no join
  if (e != cudaSuccess || (int64_t)a.M * a.page_size <= kWholeKeys) return e;
  return launch_pdl(kv_attention_join_kernel<D, NT>, dim3(ctas - 1, G::ROWS), 128, 0, st, p, ctas);
}

}  // namespace

size_t kv_attention_ws_bytes(int T, int B, int Hq, int Hkv, int D) {
  (void)T, (void)B, (void)Hq, (void)Hkv;
  return D == 128 ? carve<128, 2>(nullptr, nullptr) : carve<64, 2>(nullptr, nullptr);
}

// Eight query rows per K/V head and request, or tiles of sixteen.
cudaError_t launch_kv_attention(const KvAttention& a, cudaStream_t st) {
  const bool few = (int64_t)a.max_query_len * (a.Hq / a.Hkv) <= 8;
  if (a.D == 128) return few ? launch<128, 1>(a, st) : launch<128, 2>(a, st);
  return few ? launch<64, 1>(a, st) : launch<64, 2>(a, st);
}

}  // namespace nvfp4moe
