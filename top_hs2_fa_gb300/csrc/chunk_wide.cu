// chunk_wide.cu — attention of query chunks on tcgen05: units of up to 128 rows.
//
// Bound by the tensor pipe: 4 D flops per (row, key) against 4 D / rows bytes of K and V. A
// unit's rows are a KV head's query heads of consecutive tokens, token-major, so that a chunk
// of 128 / G tokens fills the 128 rows of an MMA whatever G is, and one K/V tile serves all
// the heads that share it. Persistent CTAs (one per SM) walk equal ranges of the units' key
// tiles (chunk_plan.cuh); the pipeline runs on across units.
//   warp 0      TMA producer of Q (two buffers, one per unit) and the K tiles
//   warp 10     TMA producer of the V tiles
//   warp 1      issues S_j = Q K_j^T into one of two TMEM buffers
//   warp 11     issues O += P_j V_j with P_j read from tensor memory; two issuers, so that one's
//               waits overlap the other's instructions
//   warps 2-9   softmax, two threads per row (warps w and w + 4 share a lane quadrant, each has
//               64 of the tile's 128 columns, i.e. one page): row max over both halves, p =
//               2^(x c - m) with the reference m moving only when it is exceeded by 2^8, P
//               rounded to bf16 over the tile's own S columns, the normaliser summed in fp32
//               from the unrounded weights
// FP8 / FP4 caches come as expanded bf16 pages: their page factors scale the logits (c) and the
// weights (2^lv) per half-tile, at no cost per element.
// TMEM: S0 [0,128), S1 [128,256), O [256,384) and [384,512) in turn, so that a unit's output is
// read while the next one accumulates. Every wait is bounded.
#include <cuda.h>

#include "chunk_plan.cuh"
#include "tc.cuh"

namespace hs2 {

namespace {

constexpr int kWRows = 128;
constexpr int kWThreads = 384;
constexpr int kWVWarp = 10, kWPVWarp = 11;
constexpr uint32_t kWTmem = 512;
constexpr float kWRescale = 8.f;
constexpr int kWStages = 2;  // K slots and V slots

template <int D>
struct WideSmem {
  static constexpr uint32_t kTile = 128 * D * 2;
  uint8_t q[2][kTile];
  uint8_t k[kWStages][kTile];
  uint8_t v[kWStages][kTile];
  float xch[2][kWRows];
  uint64_t q_full[2], q_empty[2], k_full[kWStages], k_empty[kWStages], v_full[kWStages], v_empty[kWStages], s_full[2],
      p_full[2], p_empty[2], o_empty[2];
  uint64_t x_full[4], x_empty[4];
  uint64_t all;  // a meeting of the softmax threads
  uint32_t tmem_base;
  int abort, last;
};

template <typename S>
HS2_DEVI bool stopped(S& sm) { return *(volatile int*)&sm.abort != 0; }
template <typename S>
HS2_DEVI void stop(S& sm, int32_t* dev_err) {
  flag_error(dev_err, HS2_DEV_TIMEOUT);
  atomicExch(&sm.abort, 1);
}

HS2_DEVI float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

}  // namespace

template <int D, bool EXP>
__global__ void __launch_bounds__(kWThreads, 1)
    chunk_wide_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const ChunkArgs a, const ChunkPlan p,
                      const float2* params) {
  using Sm = WideSmem<D>;
  constexpr uint32_t kTile = Sm::kTile;
  constexpr int NB = D / 64;  // 64-column blocks of a row
  extern __shared__ __align__(1024) uint8_t dsmem[];
  Sm& sm = *reinterpret_cast<Sm*>(dsmem + ((1024 - (tc::smem_u32(dsmem) & 1023)) & 1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(&sm.q_full[s], 1);
      tc::mbar_init(&sm.q_empty[s], 1);
      tc::mbar_init(&sm.s_full[s], 1);
      tc::mbar_init(&sm.p_full[s], 256);
      tc::mbar_init(&sm.p_empty[s], 1);
      tc::mbar_init(&sm.o_empty[s], 256);
    }
    for (int s = 0; s < kWStages; ++s) {
      tc::mbar_init(&sm.k_full[s], 1);
      tc::mbar_init(&sm.k_empty[s], 1);
      tc::mbar_init(&sm.v_full[s], 1);
      tc::mbar_init(&sm.v_empty[s], 1);
    }
    for (int q = 0; q < 4; ++q) {
      tc::mbar_init(&sm.x_full[q], 64);
      tc::mbar_init(&sm.x_empty[q], 64);
    }
    tc::mbar_init(&sm.all, 256);
    sm.abort = 0;
    tc::fence_mbar_init();
  }
  if (warp == 1) tc::tmem_alloc(&sm.tmem_base, kWTmem);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  griddep_wait();
  const uint32_t tS = sm.tmem_base, tO = tS + 256;
  const ChunkRange rg = chunk_range(p, blockIdx.x);
  const int per = p.head[1];

  if (warp == 0 || warp == kWVWarp) {
    // ------------------------------------------------------------------ TMA producers
    if (lane == 0) {
      const bool is_k = warp == 0;
      uint64_t* full = is_k ? sm.k_full : sm.v_full;
      uint64_t* empty = is_k ? sm.k_empty : sm.v_empty;
      const CUtensorMap* tm = is_k ? &tm_k : &tm_v;
      const int oob = (EXP ? p.max_exp_pages : a.num_pages) * a.Hkv * kPage;  // the row past the pool: zeros
      int issued = 0, seg = 0, q_issued = 0;
      bool ok = true;
      for (int at = rg.begin, un = rg.first_unit; ok && at < rg.end; ++un, ++seg) {
        const ChunkUnit u = load_unit(p, un);
        const int j0 = at - u.prefix, j1 = min(u.ntiles, rg.end - u.prefix);
        at = u.prefix + j1;
        if (is_k) {
          const int qb = seg & 1;
          if (!tc::mbar_wait(&sm.q_empty[qb], ((seg >> 1) & 1) ^ 1)) { ok = false; break; }
          tc::mbar_arrive_expect_tx(&sm.q_full[qb], kTile);
          for (int c = 0; c < NB; ++c)
            tc::tma_load_3d(sm.q[qb] + c * 16384, &tm_q, 64 * c, u.g * a.G, u.row, &sm.q_full[qb]);
          q_issued = seg + 1;
        }
        const int32_t* bt = a.bt + (size_t)u.b * a.max_pages;
        for (int j = j0; j < j1; ++j) {
          const int st = issued % kWStages;
          if (stopped(sm) || !tc::mbar_wait(&empty[st], ((issued / kWStages) & 1) ^ 1)) { ok = false; break; }
          int rows[2];
          for (int h = 0; h < 2; ++h) {
            const int lp = u.page0 + 2 * j + h;
            rows[h] = oob;
            if (lp < u.npages) {
              if (EXP) {
                rows[h] = ((u.slot_page + lp) * a.Hkv + u.g) * kPage;
              } else {
                const int phys = bt[lp];
                if (phys < 0 || phys >= a.num_pages) flag_error(a.dev_err, HS2_DEV_BAD_PAGE);
                else rows[h] = (phys * a.Hkv + u.g) * kPage;
              }
            }
          }
          tc::mbar_arrive_expect_tx(&full[st], kTile);
          uint8_t* dst = is_k ? sm.k[st] : sm.v[st];
          for (int h = 0; h < 2; ++h)
            for (int c = 0; c < NB; ++c) tc::tma_load_2d(dst + c * 16384 + h * 8192, tm, 64 * c, rows[h], &full[st]);
          ++issued;
        }
      }
      if (!ok) stop(sm, a.dev_err);
      for (int i = max(0, issued - kWStages); i < issued; ++i) (void)tc::mbar_wait(&full[i % kWStages], (i / kWStages) & 1);
      for (int i = max(0, q_issued - 2); i < q_issued; ++i) (void)tc::mbar_wait(&sm.q_full[i & 1], (i >> 1) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ S = Q K^T
    constexpr uint32_t idS = tc::idesc_bf16_f32(128, 128);
    const uint32_t el = tc::elect_one();
    int it = 0, seg = 0;
    bool ok = true;
    for (int at = rg.begin, un = rg.first_unit; ok && at < rg.end; ++un, ++seg) {
      const int2 pt = *reinterpret_cast<const int2*>(p.units + 12 * (size_t)un + 6);  // ntiles, prefix
      const int end = min(rg.end, pt.y + pt.x);
      const int qb = seg & 1;
      const uint64_t qd = tc::sdesc_sw128(tc::smem_u32(sm.q[qb]));
      ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.q_full[qb], (seg >> 1) & 1));
      for (; ok && at < end; ++at, ++it) {
        const int st = it & 1, kv = it % kWStages;
        // S_j's buffer holds P_{j-2} until its P.V is done
        ok = __all_sync(0xffffffffu, (it < 2 || tc::mbar_wait(&sm.p_empty[st], ((it - 2) >> 1) & 1)) &&
                                         tc::mbar_wait(&sm.k_full[kv], (it / kWStages) & 1));
        if (!ok) break;
        tc::tc_fence_after();
        const uint64_t kd = tc::sdesc_sw128(tc::smem_u32(sm.k[kv]));
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = ((ks >> 2) * 16384u + (ks & 3) * 32u) >> 4;
          tc::mma_f16_warp(tS + st * 128, qd + off, kd + off, idS, ks > 0 ? 1u : 0u, el);
        }
        tc::mma_commit_warp(&sm.s_full[st], el);
        tc::mma_commit_warp(&sm.k_empty[kv], el);
      }
      if (ok) tc::mma_commit_warp(&sm.q_empty[qb], el);
    }
    if (!ok && lane == 0) stop(sm, a.dev_err);
    if (it > 0) (void)tc::mbar_wait(&sm.s_full[(it - 1) & 1], ((it - 1) >> 1) & 1);
  } else if (warp == kWPVWarp) {
    // ------------------------------------------------------------------ O += P V
    constexpr uint32_t idO = tc::idesc_bf16_f32_bmn(128, D);
    const uint32_t el = tc::elect_one();
    int it = 0, seg = 0;
    bool ok = true;
    for (int at = rg.begin, un = rg.first_unit; ok && at < rg.end; ++un, ++seg) {
      const int2 pt = *reinterpret_cast<const int2*>(p.units + 12 * (size_t)un + 6);
      const int end = min(rg.end, pt.y + pt.x);
      const uint32_t o = tO + (seg & 1) * 128;
      ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.o_empty[seg & 1], ((seg >> 1) & 1) ^ 1));
      for (int j = 0; ok && at < end; ++at, ++it, ++j) {
        const int st = it & 1, kv = it % kWStages;
        ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.v_full[kv], (it / kWStages) & 1) &&
                                         tc::mbar_wait(&sm.p_full[st], (it >> 1) & 1));
        if (!ok) break;
        tc::tc_fence_after();
        const uint64_t vd = tc::sdesc_sw128_mn(tc::smem_u32(sm.v[kv]), 16384u, 1024u);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          tc::mma_f16_ts_warp(o, tS + st * 128 + ks * 8, vd + ks * 128, idO, (j > 0 || ks > 0) ? 1u : 0u, el);
        tc::mma_commit_warp(&sm.v_empty[kv], el);
        tc::mma_commit_warp(&sm.p_empty[st], el);
      }
    }
    if (!ok && lane == 0) stop(sm, a.dev_err);
    if (it > 0) (void)tc::mbar_wait(&sm.p_empty[(it - 1) & 1], ((it - 1) >> 1) & 1);
  } else {
    // ------------------------------------------------------------------ softmax warps
    const int qd = warp & 3;
    const int half = (warp - 2) >> 2;
    const int r = qd * 32 + lane;
    const uint32_t lane_off = (uint32_t)(qd * 32) << 16;
    int rounds = 0;  // of swap
    auto swap = [&](float v, float& other) -> bool {
      if (rounds > 0 && !__all_sync(0xffffffffu, tc::mbar_wait(&sm.x_empty[qd], (rounds - 1) & 1))) return false;
      sm.xch[half][r] = v;
      tc::mbar_arrive(&sm.x_full[qd]);
      if (!__all_sync(0xffffffffu, tc::mbar_wait(&sm.x_full[qd], rounds & 1))) return false;
      other = sm.xch[half ^ 1][r];
      tc::mbar_arrive(&sm.x_empty[qd]);
      ++rounds;
      return true;
    };
    int meetings = 0;
    auto meet = [&]() -> bool {  // bounded, unlike a hardware barrier
      tc::mbar_arrive(&sm.all);
      return __all_sync(0xffffffffu, tc::mbar_wait(&sm.all, meetings++ & 1));
    };
    bool ok = true;
    int it = 0, seg = 0;
    const int tr = r / a.G;  // the row's token of the unit
    for (int at = rg.begin, un = rg.first_unit; ok && at < rg.end; ++un, ++seg) {
      const ChunkUnit u = load_unit(p, un);
      const int j0 = at - u.prefix, j1 = min(u.ntiles, rg.end - u.prefix);
      at = u.prefix + j1;
      const int pos = u.pos0 + tr, pos_last = u.pos0 + u.ntok - 1;
      const uint32_t o = tO + (seg & 1) * 128;
      const int32_t* bt = a.bt + (size_t)u.b * a.max_pages;
      float m_used = -INFINITY, l = 0.f;
      // this half's page of tile j: (factor of the logits or -1 where it is not there, log2 of V's)
      auto page_params = [&](int j) -> float2 {
        const int lp = u.page0 + 2 * j + half;
        if (lp >= u.npages) return make_float2(-1.f, 0.f);
        if (EXP) return params[(size_t)(u.slot_page + lp) * a.Hkv + u.g];
        const int phys = bt[lp];
        return make_float2(phys >= 0 && phys < a.num_pages ? 1.f : -1.f, 0.f);
      };
      float2 pp = page_params(j0);
      for (int j = j0; j < j1; ++j, ++it) {
        const int sb = it & 1;
        const float2 par = pp;
        if (j + 1 < j1) pp = page_params(j + 1);
        if (!__all_sync(0xffffffffu, !stopped(sm) && tc::mbar_wait(&sm.s_full[sb], (it >> 1) & 1))) { ok = false; break; }
        tc::tc_fence_after();
        float x[64];
        {
          uint32_t raw[2][32];
#pragma unroll
          for (int c = 0; c < 2; ++c) tc::tmem_ld32_async(tS + lane_off + sb * 128 + half * 64 + c * 32, raw[c]);
          tc::tmem_wait_ld(raw[1]);
          tc::tmem_regs_ready(raw[0]);
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e) x[c * 32 + e] = __uint_as_float(raw[c][e]);
        }
        const int kb = (u.page0 + 2 * j + half) * kPage;  // this half's first key
        if (par.x < 0.f) {
#pragma unroll
          for (int e = 0; e < 64; ++e) x[e] = -INFINITY;
        } else if (kb + 63 > u.pos0 || (a.w > 0 && kb <= pos_last - a.w)) {
          const int hi = pos - kb, lo = a.w > 0 ? hi - a.w : -1;
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (e > hi || e <= lo) x[e] = -INFINITY;
        }
        const float c = par.x * a.scale_log2;
        float mt = fmaxf(x[0], x[1]);
#pragma unroll
        for (int e = 2; e < 64; e += 2) mt = max3(mt, x[e], x[e + 1]);
        mt *= fabsf(c);
        float mo;
        if (!swap(mt, mo)) { ok = false; break; }
        const float m_new = max3(m_used, mt, mo);
        const bool need = m_new > m_used + kWRescale || (m_used == -INFINITY && m_new > -INFINITY);
        const float alpha = (need && m_used > -INFINITY) ? tc::ex2(m_used - m_new) : 1.f;
        if (need) m_used = m_new;
        l *= alpha;
        if (j > j0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          if (!__all_sync(0xffffffffu, tc::mbar_wait(&sm.p_empty[(it - 1) & 1], ((it - 1) >> 1) & 1))) { ok = false; break; }
          tc::tc_fence_after();
#pragma unroll 1
          for (int k = 0; k < D / 64; ++k) {  // this half's share of the D columns
            float ov[32];
            const uint32_t col = half * (D / 2) + k * 32;
            tc::tmem_ld32(o + lane_off + col, ov);
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] *= alpha;
            tc::tmem_st32(o + lane_off + col, ov);
          }
        }
        // p = 2^(x c - m) (a row with nothing visible yet: all zero), times the page's V factor
        const float shift = m_used == -INFINITY ? 0.f : par.y - m_used;
        float sum0 = 0.f, sum1 = 0.f;
        uint32_t w[32];
#pragma unroll
        for (int e = 0; e < 64; e += 2) {
          const float p0 = tc::ex2(fmaf(x[e], c, shift)), p1 = tc::ex2(fmaf(x[e + 1], c, shift));
          sum0 += p0;
          sum1 += p1;
          w[e >> 1] = pack_bf16(p0, p1);
        }
        if (par.x < 0.f) {  // no page: c is negative and -inf * c is not a weight
#pragma unroll
          for (int e = 0; e < 32; ++e) w[e] = 0u;
          sum0 = sum1 = 0.f;
        }
        l += EXP ? (sum0 + sum1) * tc::ex2(-par.y) : sum0 + sum1;
        tc::tmem_st32u(tS + lane_off + sb * 128 + half * 32, w);
        if (!EXP && kb < u.t && kb + kPage > u.t) {
          // the sequence ends inside this page: what lies behind it in the pool may be anything,
          // and 0 times a NaN is a NaN
          if (!__all_sync(0xffffffffu, tc::mbar_wait(&sm.v_full[it % kWStages], (it / kWStages) & 1))) { ok = false; break; }
          uint8_t* v = sm.v[it % kWStages] + half * 8192;
          const int dead = kb + kPage - u.t;
          for (int e = qd * 32 + lane; e < dead * 8 * NB; e += 128) {
            const int blk = e / (dead * 8), z = e % (dead * 8);
            *reinterpret_cast<uint4*>(v + blk * 16384 + (u.t - kb) * 128 + 16 * z) = make_uint4(0, 0, 0, 0);
          }
          tc::fence_async_smem();
        }
        tc::tc_fence_before();
        tc::mbar_arrive(&sm.p_full[sb]);
      }
      if (!ok) break;
      // ---- the unit's (or this part's) output
      if (!__all_sync(0xffffffffu, !stopped(sm) && tc::mbar_wait(&sm.p_empty[(it - 1) & 1], ((it - 1) >> 1) & 1))) { ok = false; break; }
      float lo;
      if (!swap(l, lo)) { ok = false; break; }
      tc::tc_fence_after();
      const bool whole = j0 == 0 && j1 == u.ntiles;
      const bool live = tr < u.ntok;
      const int head = u.g * a.G + r % a.G;
      const size_t row = (size_t)(u.row + tr) * a.Hq + head;
      const float lsum = half ? lo + l : l + lo;
      // normalised values of 32 columns to o
      auto store = [&](const float (&ov)[32], float f, int col) {
        if (a.o_bf16) {
          uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.o) + row * D + col);
#pragma unroll
          for (int e = 0; e < 32; e += 8)
            dst[e / 8] = make_uint4(pack_bf16(ov[e] * f, ov[e + 1] * f), pack_bf16(ov[e + 2] * f, ov[e + 3] * f),
                                    pack_bf16(ov[e + 4] * f, ov[e + 5] * f), pack_bf16(ov[e + 6] * f, ov[e + 7] * f));
        } else {
          float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.o) + row * D + col);
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            dst[e / 4] = make_float4(ov[e] * f, ov[e + 1] * f, ov[e + 2] * f, ov[e + 3] * f);
        }
      };
      const float b2 = sink_b2(a.sink, head);
      auto finish = [&](float M, float L, float& f) {  // the output's factor; the row's lse
        const float M2 = fmaxf(M, b2), sc = exp2_rel(M, M2);
        const float den = L * sc + exp2_rel(b2, M2);
        f = den > 0.f ? sc / den : 0.f;
        if (a.lse && half == 0 && live) a.lse[row] = den > 0.f ? (M2 + log2f(den)) / kLog2e : -INFINITY;
      };
      if (whole) {
        float f;
        finish(m_used, lsum, f);
#pragma unroll 1
        for (int k = 0; k < D / 64; ++k) {
          float ov[32];
          tc::tmem_ld32(o + lane_off + half * (D / 2) + k * 32, ov);
          if (live) store(ov, f, half * (D / 2) + k * 32);
        }
        tc::tc_fence_before();
        tc::mbar_arrive(&sm.o_empty[seg & 1]);
      } else {
        const int slot = part_slot(u, per, blockIdx.x);
        float4* po = reinterpret_cast<float4*>(p.part_o) + (size_t)slot * (D / 4) * kWRows;
        if (half == 0) reinterpret_cast<float2*>(p.part_ml)[(size_t)slot * kWRows + r] = make_float2(m_used, lsum);
#pragma unroll 1
        for (int k = 0; k < D / 64; ++k) {
          float ov[32];
          tc::tmem_ld32(o + lane_off + half * (D / 2) + k * 32, ov);
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            po[(half * (D / 8) + k * 8 + e / 4) * kWRows + r] = make_float4(ov[e], ov[e + 1], ov[e + 2], ov[e + 3]);
        }
        tc::tc_fence_before();
        tc::mbar_arrive(&sm.o_empty[seg & 1]);
        // the last CTA to leave its part merges them all, in CTA order
        const int c0 = u.prefix / per, c1 = (u.prefix + u.ntiles - 1) / per;
        __threadfence();
        if (!meet()) { ok = false; break; }
        if (threadIdx.x == 64) sm.last = atomicAdd(&p.arrive[un], 1) == c1 - c0;
        if (!meet()) { ok = false; break; }
        if (*(volatile int*)&sm.last) {
          __threadfence();
          auto slot_of = [&](int c) { return part_slot(u, per, c); };
          float M = -INFINITY, L = 0.f;
          for (int c = c0; c <= c1; ++c)
            M = fmaxf(M, __ldcg(reinterpret_cast<const float2*>(p.part_ml) + (size_t)slot_of(c) * kWRows + r).x);
          for (int c = c0; c <= c1; ++c) {
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + (size_t)slot_of(c) * kWRows + r);
            L += exp2_rel(ml.x, M) * ml.y;
          }
          float f;
          finish(M, L, f);
#pragma unroll 1
          for (int k = 0; k < D / 64; ++k) {
            float ov[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] = 0.f;
            for (int c = c0; c <= c1; ++c) {
              const size_t sl = slot_of(c);
              const float g = exp2_rel(__ldcg(reinterpret_cast<const float2*>(p.part_ml) + sl * kWRows + r).x, M);
              const float4* src = reinterpret_cast<const float4*>(p.part_o) + sl * (D / 4) * kWRows;
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 v = __ldcg(src + (half * (D / 8) + k * 8 + e / 4) * kWRows + r);
                ov[e] += g * v.x, ov[e + 1] += g * v.y, ov[e + 2] += g * v.z, ov[e + 3] += g * v.w;
              }
            }
            if (live) store(ov, f, half * (D / 2) + k * 32);
          }
        }
        if (!meet()) { ok = false; break; }  // sm.last is rewritten by the next part
      }
    }
    if (!ok && !stopped(sm)) stop(sm, a.dev_err);
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) tc::tmem_dealloc(sm.tmem_base, kWTmem);
}

template <int D>
static cudaError_t launch_wide(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const ChunkArgs& a,
                               const ChunkPlan& p, const float2* params, cudaStream_t s) {
  const size_t sm = sizeof(WideSmem<D>) + 1024;
  auto kern = params ? chunk_wide_kernel<D, true> : chunk_wide_kernel<D, false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(p.ctas), dim3(kWThreads), sm, s, tq, tk, tv, a, p, params);
}

cudaError_t launch_chunk_wide(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const ChunkArgs& a,
                              const ChunkPlan& p, const float2* params, int d, cudaStream_t s) {
  return d == 128 ? launch_wide<128>(tq, tk, tv, a, p, params, s) : launch_wide<64>(tq, tk, tv, a, p, params, s);
}

}  // namespace hs2
