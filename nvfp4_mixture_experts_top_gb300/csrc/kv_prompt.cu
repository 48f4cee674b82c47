// kv_prompt.cu -- attention over the paged 8-bit key/value cache for many query rows
// per request and K/V head (prompt chunks): a tile of 128 rows against tiles of 128
// keys, S = Q K^T and O += P V on tcgen05 with the cached codes as they are.
//
// A row is a lane: its maximum, sum and reference are a thread's own.
//   S = Q K^T   K's codes as they are (kind::f8f6f4), the query row as the sum of two
//               E4M3 values times its power of two, 2^-e (q1 + q2): exact for what
//               bf16 holds down to 2^-9 of the row's largest element, within 2^-17
//   O += P V    f16: four warps widen each V tile once for all 128 rows (exact, times
//               its block's power of two); weights have 11 bits.  Splitting weights
//               into three 8-bit terms instead took 4.75 instructions per weight next
//               to 0.5, and half as long again on the tensor cores: 934 us for three
//               chunks of 1.5-2.1K tokens after 0.5-4K.
// A tile is 512 + 512 cycles of products at D = 128, next to 512 of exponentials (a
// quarter per cycle and scheduler); S and V's f16 form are double buffered so that
// all run at a time.
//
// Roles, ring, division of the work and join as in kv_attention.cu, and warps 6-9 that
// widen V; one CTA per SM.
#include "kv_attention.cuh"

namespace nvfp4moe {
namespace {

using namespace kv;

constexpr int kRows = 128;

constexpr int kPromptThreads = 320;
constexpr float kRowSlack = 5.0f;   // log2 by which a logit may pass the row's reference
constexpr float kRowBoost = 10.5f;  // log2 of the weights' shift: 2^(10.5 + 5) is in f16's range

template <int D>
struct Geo {
  static constexpr int QOFF = 0;                            // [2 terms][128][D] E4M3
  static constexpr int POFF = QOFF + 2 * kRows * D;         // [2 halves of the keys][128 rows][64] f16
  static constexpr int VOFF = POFF + kRows * kTile * 2;     // [2 buffers][D / 64][128 keys][64] f16
  static constexpr int ROFF = VOFF + 2 * kTile * D * 2;
  static constexpr int SUBS = D == 128 ? 6 : 10;  // K in the even slots, V in the odd ones
  static constexpr int SMEM_BYTES = ROFF + SUBS * kTile * D;
  static constexpr int OCOL = 2 * kTile;                    // TMEM: two S, then O
  static constexpr int COLS = 512;
};

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }

template <int D>
__global__ void __launch_bounds__(kPromptThreads, 1)
    kv_prompt_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const Params p) {
  using G = Geo<D>;
  constexpr int SUBS = G::SUBS;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(8) uint64_t full[SUBS], empty[SUBS], s_full[2], s_empty[2], v_full[2], v_empty[2], q_full, p_full, pv_done,
      drained;
  __shared__ Heads heads;
  __shared__ RangeScratch<kPromptThreads> scratch;
  __shared__ uint32_t tmem_s;
  __shared__ volatile int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = p.Hq / p.Hkv;
  if (tid == 0) {
    for (int i = 0; i < SUBS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kHeads; ++i) mbar_init(&heads.full[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 4);
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    mbar_init(&q_full, 4);
    mbar_init(&p_full, 4);
    mbar_init(&pv_done, 1);
    mbar_init(&drained, 1);
    abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  if (warp == 5) {
    tmem_alloc(&tmem_s, G::COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_trigger();  // after this CTA's TMEM allocation
  const uint32_t tmem = tmem_s;
  Pieces<kRows> it;
  range_of_cta<kPromptThreads, kRows>(p, group, it, scratch);

  bool ok = true;
  int gc = 0;  // tiles of the CTA so far, the same count in every role
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    // (after a failure the softmax warps go on without waiting)
    if (ok) ok = warp_wait(bar, parity, &abort_flag, p.dev_status);
    return ok;
  };
  if (warp == 4) {
    copy_tiles<D, SUBS, kRows>(p, group, it, &tm_k, &tm_v, smem + G::ROFF, full, empty, heads, &abort_flag);
  } else if (warp == 5) {
    // ------------------------------------------------------------ products
    constexpr uint32_t idesc_s = idesc_e4m3(kRows, kTile, false);
    // kind::f16 with F16 operands and fp32 accumulation, V MN-major (bit 16)
    constexpr uint32_t idesc_o = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((kRows >> 4) << 24);
    constexpr uint32_t layout = D == 128 ? 2 : 4;  // swizzle of rows of D bytes
    const uint32_t base = smem_u32(smem), ring = base + G::ROFF;
    int sub = 0;
    uint32_t phase = 0, q_phase = 0;
    bool issued = false;
    auto advance = [&] {
      if (++sub == SUBS) {
        sub = 0;
        phase ^= 1;
      }
    };
    auto product_s = [&](int n) {  // S of tile n of the CTA: K's slot is the current one
      if (!wait(&full[sub], phase) || !wait(&s_empty[n & 1], ((n >> 1) & 1) ^ 1)) return;
      tc_fence_after();
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int k = 0; k < D / 32; ++k)
          ew_mma_e4m3(tmem + (n & 1) * kTile, smem_desc(base + G::QOFF + t * kRows * D + k * 32, 16, 8 * D, layout),
                      smem_desc(ring + sub * kTile * D + k * 32, 16, 8 * D, layout), idesc_s, t > 0 || k > 0);
      ew_commit(&empty[sub]);
      ew_commit(&s_full[n & 1]);
      issued = true;
    };
    while (ok && it.next(p, group)) {
      const int nt = it.nt;
      if (nt == 0) continue;
      if (!wait(&q_full, q_phase)) break;
      q_phase ^= 1;
      product_s(gc);
      for (int i = 0; i < nt && ok; ++i, ++gc) {
        advance();
        advance();  // (V's slot is the widening warps')
        if (i + 1 < nt) product_s(gc + 1);
        if (!wait(&v_full[gc & 1], (gc >> 1) & 1) || !wait(&p_full, gc & 1)) break;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          ew_mma_bf16_ss(tmem + G::OCOL,
                         smem_desc(base + G::POFF + (k >> 2) * (kRows * 128) + (k & 3) * 32, 16, 1024, 2),
                         smem_desc(base + G::VOFF + (gc & 1) * (kTile * D * 2) + k * 2048, kTile * 128, 1024, 2), idesc_o,
                         i > 0 || k > 0);
        ew_commit(&v_empty[gc & 1]);
        ew_commit(&pv_done);
      }
    }
    if (!ok && issued) {  // given up: no product may outlive the operands and the TMEM
      ew_commit(&drained);
      mbar_wait(&drained, 0);
    }
  } else if (warp > 5) {
    // ------------------------------------------------------------ V to f16
    const int th = tid - 6 * 32;
    int sub = 1, unit = -127;
    uint32_t phase = 0;
    while (it.next(p, group)) {
      unit = -127;
      for (int i = 0; i < it.nt; ++i, ++gc) {
        const int key0 = (it.t0 + i) * kTile, hd = gc & (kHeads - 1);
        wait(&full[sub], phase);
        wait(&heads.full[hd], gc / kHeads & 1);
        wait(&v_empty[gc & 1], ((gc >> 1) & 1) ^ 1);
        const int2 vr = heads.vrange[hd];
        unit = max(unit, vr.y);
        const bool plain = vr.x == unit && key0 + kTile <= it.limit;
        const uint8_t* src = smem + G::ROFF + sub * kTile * D;
        uint8_t* dst = smem + G::VOFF + (gc & 1) * (kTile * D * 2);
#pragma unroll 2
        for (int n = 0; n < D / 16; ++n) {
          constexpr int CPR = D / 16;  // chunks of 16 elements of a row
          const int r = (n * 128 + th) / CPR, c = (n * 128 + th) % CPR;
          const uint4 w = *reinterpret_cast<const uint4*>(src + swizzled<D>(r, c));
          uint32_t h[8];
          decode4(w.x, h[0], h[1]);
          decode4(w.y, h[2], h[3]);
          decode4(w.z, h[4], h[5]);
          decode4(w.w, h[6], h[7]);
          if (!plain) {
            // rows past the sequence hold anything, and 0 * NaN would spread: zeros instead
            const int ve = heads.vexp[hd][r >> p.shift];
            const bool there = key0 + r < it.limit && ve != kNoPage;
            const __half2 f = __float2half2_rn(there ? exp2_int(max(ve - unit, kFarExp)) : 0.0f);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const __half2 y = __hmul2(as_half2(h[k]), f);
              h[k] = there ? *reinterpret_cast<const uint32_t*>(&y) : 0u;
            }
          }
          uint8_t* row = dst + (c >> 2) * (kTile * 128);
          *reinterpret_cast<uint4*>(row + swizzled<128>(r, (c & 3) * 2)) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(row + swizzled<128>(r, (c & 3) * 2 + 1)) = make_uint4(h[4], h[5], h[6], h[7]);
        }
        fence_proxy_async_smem();
        asm volatile("bar.sync 2, 128;" ::: "memory");
        if (warp == 6) {
          ew_arrive(&empty[sub]);
          ew_arrive(&v_full[gc & 1]);
        }
        sub += 2;
        if (sub >= SUBS) {
          sub -= SUBS;
          phase ^= 1;
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax, a row per thread
    const uint32_t lane_tmem = tmem + ((uint32_t)(warp * 32) << 16);
    bool first = true;
    while (it.next(p, group)) {
      const int nt = it.nt, rr = it.row0 + tid, tok = rr / group;
      const bool live = tid < it.nrows;
      const int64_t at = (int64_t)(it.rq.q0 + tok) * p.Hq + it.hk * group + rr - tok * group;
      if (first && tid == 0)
        p.cut[blockIdx.x] = {it.u0, it.span, it.rq.q0 * group + it.row0, it.hk, it.nrows, {0, 0, 0}};
      // keys that the row sees; that all of the tile's rows see
      const int lim = live ? min(it.rq.kv, it.rq.kv - it.rq.n + tok + 1) : 0;
      const int all_see = it.rq.kv - it.rq.n + it.row0 / group + 1;
      // the row as 2^-e (q1 + q2), in the sign of the scale; not finite: a row of NaN
      float qs = 0.0f;
      if (nt > 0) {
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (int64_t)(it.rq.q0 + tok) * p.ld_q +
                                                          (int64_t)(it.hk * group + rr - tok * group) * D);
        float amax = 0.0f;
        if (live) {
#pragma unroll 4
          for (int i = 0; i < D / 8; ++i) {
            const uint4 w = src[i];
            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(x[k] << 16)), fabsf(__uint_as_float(x[k] & 0xFFFF0000u))));
          }
        }
        const int e = amax == 0.0f ? 0 : min(7 - floor_log2(amax), 126);
        float f = exp2_int(e);
        if (p.scale < 0.0f) f = -f;
        if (!(amax <= 3.402823466e38f)) f = __int_as_float(0x7FFFFFFF);
        // (a zero scale stays apart from a key that is not seen: -inf * qs)
        qs = fmaxf(fabsf(p.scale) * 1.4426950408889634f * exp2_int(-e), 1.175494351e-38f);
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          uint32_t hi[4] = {}, lo[4] = {};
          if (live) {
            const uint4 v[2] = {src[2 * c], src[2 * c + 1]};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t a = i & 1 ? v[i >> 1].z : v[i >> 1].x, b = i & 1 ? v[i >> 1].w : v[i >> 1].y;
              const float x0 = __uint_as_float(a << 16) * f, x1 = __uint_as_float(a & 0xFFFF0000u) * f;
              const float x2 = __uint_as_float(b << 16) * f, x3 = __uint_as_float(b & 0xFFFF0000u) * f;
              hi[i] = encode4(x0, x1, x2, x3);
              uint32_t d0, d1;
              decode4(hi[i], d0, d1);
              const float2 y0 = f16x2_to_f32(d0), y1 = f16x2_to_f32(d1);
              lo[i] = encode4(x0 - y0.x, x1 - y0.y, x2 - y1.x, x3 - y1.y);
            }
          }
          *reinterpret_cast<uint4*>(smem + G::QOFF + swizzled<D>(tid, c)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(smem + G::QOFF + kRows * D + swizzled<D>(tid, c)) =
              make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        ew_arrive(&q_full);
      }

      float m = -INFINITY, ref = 0.0f, l = 0.0f;  // reference (0 while there is none), sum
      int unit = -127;  // outputs are in units of 2^unit, the largest value exponent so far
      for (int i = 0; i < nt; ++i, ++gc) {
        const int key0 = (it.t0 + i) * kTile, buf = gc & 1, hd = gc & (kHeads - 1);
        wait(&s_full[buf], (gc >> 1) & 1);
        tc_fence_after();
        wait(&heads.full[hd], gc / kHeads & 1);
        const int2 vr = heads.vrange[hd];
        // the row's logits, 32 keys at a time, twice: for the maximum, then for the
        // weights.  Loops stay rolled: unrolled, the roles' code outgrew the
        // instruction cache, and half of all issue slots were lost to it.
        const uint32_t s_tmem = lane_tmem + buf * kTile;
        const int seen = lim - key0;
        const bool odd = key0 + kTile > all_see || vr.x == kNoPage;
        auto hide = [&](uint32_t (&x)[32], int k) {  // keys that the row does not see are -inf
          const bool gone0 = heads.vexp[hd][k >> p.shift] == kNoPage;
          const bool gone1 = heads.vexp[hd][(k + 16) >> p.shift] == kNoPage;
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (k + j >= seen || (j < 16 ? gone0 : gone1)) x[j] = 0xFF800000u;
        };
        // log2 units per unit of S
        auto factor = [&](int k) {
          return fminf(fmaxf(qs * heads.kscale[hd][k >> p.shift], 1.175494351e-38f), 3.402823466e38f);
        };
        float top = -INFINITY;
#pragma unroll 1
        for (int k = 0; k < kTile; k += 32) {
          uint32_t x[32];
          tmem_ld_32x32b_x32(s_tmem + k, x);
          const float c0 = factor(k), c1 = factor(k + 16);
          tmem_ld_wait();
          if (odd) hide(x, k);
          float mx[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            mx[j] = fmaxf(fmaxf(__uint_as_float(x[4 * j]), __uint_as_float(x[4 * j + 1])),
                          fmaxf(__uint_as_float(x[4 * j + 2]), __uint_as_float(x[4 * j + 3])));
          top = fmaxf(top, fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c0,
                                 fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])) * c1));
        }
        const int unit1 = max(unit, vr.y);
        if (__any_sync(0xFFFFFFFFu, top > ref + kRowSlack || (m == -INFINITY && top != -INFINITY)) || unit1 != unit) {
          // the references move to the maxima, sums and outputs with them
          const float m1 = fmaxf(m, top), r1 = m1 == -INFINITY ? 0.0f : m1, f = ex2(m - r1);
          l *= f;
          m = m1;
          ref = r1;
          if (i > 0) {
            const float fo = f * exp2_int(max(unit - unit1, -127));
            wait(&pv_done, (gc & 1) ^ 1);
            tc_fence_after();
#pragma unroll 1
            for (int o = 0; o < D; o += 32) {
              uint32_t y[32];
              tmem_ld_32x32b_x32(lane_tmem + G::OCOL + o, y);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 32; ++j) y[j] = __float_as_uint(__uint_as_float(y[j]) * fo);
              tmem_st_32x32b_x32(lane_tmem + G::OCOL + o, y);
            }
            tmem_st_wait();
            tc_fence_before();
          }
          unit = unit1;
        }
        const float up = kRowBoost - ref;
        float sum[4] = {};
        wait(&pv_done, (gc & 1) ^ 1);  // the last product has read P
#pragma unroll 1
        for (int k = 0; k < kTile; k += 32) {
          uint32_t x[32];
          tmem_ld_32x32b_x32(s_tmem + k, x);
          const float c0 = factor(k), c1 = factor(k + 16);
          tmem_ld_wait();
          if (odd) hide(x, k);
          uint8_t* dst = smem + G::POFF + (k >> 6) * (kRows * 128);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int n = 8 * q + 2 * j;
              const float a = ex2(fmaf(__uint_as_float(x[n]), q < 2 ? c0 : c1, up));
              const float b = ex2(fmaf(__uint_as_float(x[n + 1]), q < 2 ? c0 : c1, up));
              sum[j] += a + b;
              const __half2 h = __floats2half2_rn(a, b);
              w[j] = *reinterpret_cast<const uint32_t*>(&h);
            }
            *reinterpret_cast<uint4*>(dst + swizzled<128>(tid, (k >> 3 & 4) + q)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        tc_fence_before();
        __syncwarp();
        ew_arrive(&s_empty[buf]);
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        fence_proxy_async_smem();
        __syncwarp();
        ew_arrive(&p_full);
      }

      // ---- the piece's result
      const bool whole = it.take == it.span, none = l == 0.0f;
      const int64_t part = ((int64_t)blockIdx.x * 2 + (first ? 0 : 1)) * kRows + tid;
      const float inv = none ? 0.0f : reciprocal(l), us = exp2_int(unit);
      const float lse2 = none ? -INFINITY : ref + (lg2(l) - kRowBoost);
      if (live) {
        if (!whole) p.part_lse[part] = lse2;
        else if (p.lse != nullptr) p.lse[at] = lse2 * 0.6931471805599453f;
      }
      if (nt > 0) {
        wait(&pv_done, (gc & 1) ^ 1);
        tc_fence_after();
      }
#pragma unroll 1
      for (int o = 0; o < D; o += 32) {
        uint32_t x[32];
        if (nt > 0) {
          tmem_ld_32x32b_x32(lane_tmem + G::OCOL + o, x);
          tmem_ld_wait();
        }
        float y[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) y[j] = none ? 0.0f : __uint_as_float(x[j]) * inv * us;
        if (!live) continue;
        if (whole) {
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * j], y[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t*>(&b);
          }
          uint4* dst = reinterpret_cast<uint4*>(p.out + at * D + o);
#pragma unroll
          for (int j = 0; j < 4; ++j) dst[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        } else {
          float4* dst = reinterpret_cast<float4*>(p.part + part * D + o);
#pragma unroll
          for (int j = 0; j < 8; ++j) dst[j] = make_float4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
        }
      }
      tc_fence_before();
      first = false;
    }
    if (first && tid == 0) p.cut[blockIdx.x].before = 0;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, G::COLS);
  }
}

template <int D>
cudaError_t launch_prompt(const KvAttention& a, cudaStream_t st) {
  return launch<D, kRows>(kv_prompt_kernel<D>, 1, kPromptThreads, Geo<D>::SMEM_BYTES, a, st);
}

}  // namespace

size_t kv_prompt_ws_bytes(int D) {
  return D == 128 ? carve<128, kRows>(nullptr, nullptr, num_sms()) : carve<64, kRows>(nullptr, nullptr, num_sms());
}

cudaError_t launch_kv_prompt(const KvAttention& a, cudaStream_t st) {
  return a.D == 128 ? launch_prompt<128>(a, st) : launch_prompt<64>(a, st);
}

}  // namespace nvfp4moe
