// chunk_wide.cu — attention of query chunks on tcgen05: units of up to 256 rows.
//
// Bound by the tensor pipe: 4 D flops per (row, key) against 4 D / rows bytes of K and V. A
// unit's rows are a KV head's query heads of consecutive tokens, token-major, so that a chunk
// of 128 / G tokens fills the 128 rows of an MMA whatever G is, and one K/V tile serves all
// the heads that share it. A unit is two such halves, a and b, that take turns on the tensor
// pipe: while one half's softmax runs, the other's products do (one half with two S buffers left
// the pipe waiting for the softmax of the only tile: 1.02 ms against 0.70 for 2048 tokens over
// 32768 FP4 keys). That call takes 0.665 ms now, 1.60 PFLOP/s or 0.84 of the burst rate, its
// expansion and merge included. Persistent CTAs (one per SM) walk equal ranges of the units' key tiles
// (chunk_plan.cuh).
//   warp 0      TMA producer of Q and the K tiles; warp 1 of the V tiles
//   warps 2, 3  issue half a's and half b's MMAs: O += P_j V_j with P_j read from tensor memory,
//               then S_{j+1} = Q K^T over it
//   warps 4-7, 8-11  softmax of half a, b: a thread has a whole row. p = 2^(x c - m) with the
//               reference m moving only when it is exceeded by 2^8, P rounded to bf16 over the
//               tile's own S columns (an MMA's operands have one type, and V is bf16: a weight
//               is off by at most 2^-8 of itself), the normaliser summed in fp32 from unrounded weights
// FP8 / FP4 caches come as expanded bf16 pages: their page factors scale the logits (c) and the
// weights (2^lv) per page, at no cost per element.
// TMEM: S of a [0,128), of b [128,256), O of a [256,384), of b [384,512). Every wait is bounded.
#include <cuda.h>

#include "chunk_plan.cuh"
#include "f32x2.cuh"
#include "rows_m.cuh"
#include "tc.cuh"

namespace hs2 {

namespace {

constexpr int kWStages = 2;  // K slots and V slots

template <int D>
struct WideSmem {
  static constexpr uint32_t kTile = 128 * D * 2;
  uint8_t q[2][kTile];  // by half
  uint8_t k[kWStages][kTile];
  uint8_t v[kWStages][kTile];
  uint64_t q_full, q_empty, k_full[kWStages], k_empty[kWStages], v_full[kWStages], v_empty[kWStages];
  // by half
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint32_t tmem_base;
  int abort;
};

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
    tc::mbar_init(&sm.q_full, 1);
    tc::mbar_init(&sm.q_empty, 2);  // the last S of either half
    for (int s = 0; s < kWStages; ++s) {
      tc::mbar_init(&sm.k_full[s], 1);
      tc::mbar_init(&sm.k_empty[s], 2);  // S, P.V of either half
      tc::mbar_init(&sm.v_full[s], 1);
      tc::mbar_init(&sm.v_empty[s], 2);
    }
    for (int h = 0; h < 2; ++h) {
      tc::mbar_init(&sm.s_full[h], 1);
      tc::mbar_init(&sm.p_full[h], 128);
      tc::mbar_init(&sm.pv_done[h], 1);
    }
    sm.abort = 0;
    tc::fence_mbar_init();
  }
  griddep_wait();
  const ChunkRange rg = chunk_range(p, blockIdx.x);
  if (rg.begin >= rg.end) return;  // nothing for this CTA (the whole block leaves)
  if (warp == 1) tc::tmem_alloc(&sm.tmem_base, kWTmem);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tS = sm.tmem_base, tO = tS + 256;
  const int per = p.head[1];
  const int half_tok = kWRows >> a.log2G;  // tokens of a half

  if (warp < 2) {
    // ------------------------------------------------------------------ TMA producers
    wide_regs_down<kWRegsMisc>();
    if (lane == 0) {
      const bool is_k = warp == 0;
      uint64_t* full = is_k ? sm.k_full : sm.v_full;
      uint64_t* empty = is_k ? sm.k_empty : sm.v_empty;
      const CUtensorMap* tm = is_k ? &tm_k : &tm_v;
      const int oob = (EXP ? p.max_exp_pages : a.num_pages) * a.Hkv * kPage;  // the row past the pool: zeros
      int issued = 0, seg = 0;
      bool ok = true;
      for (int at = rg.begin, un = rg.first_unit; ok && at < rg.end; ++un, ++seg) {
        const ChunkUnit u = load_unit(p, un);
        const int j0 = at - u.prefix, j1 = min(u.ntiles, rg.end - u.prefix);
        at = u.prefix + j1;
        if (is_k) {
          if (!tc::mbar_wait(&sm.q_empty, (seg & 1) ^ 1)) { ok = false; break; }
          const int halves = u.ntok > half_tok ? 2 : 1;
          tc::mbar_arrive_expect_tx(&sm.q_full, halves * kTile);
          for (int h = 0; h < halves; ++h)
            for (int c = 0; c < NB; ++c)
              tc::tma_load_3d(sm.q[h] + c * 16384, &tm_q, 64 * c, u.g * a.G, u.row + h * half_tok, &sm.q_full);
        }
        const int32_t* bt = a.bt + (size_t)u.b * a.max_pages;
        for (int j = j0; j < j1; ++j) {
          const int st = issued % kWStages;
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
          if (stopped(sm) || !tc::mbar_wait(&empty[st], ((issued / kWStages) & 1) ^ 1)) { ok = false; break; }
          tc::mbar_arrive_expect_tx(&full[st], kTile);
          uint8_t* dst = is_k ? sm.k[st] : sm.v[st];
          for (int h = 0; h < 2; ++h)
            for (int c = 0; c < NB; ++c) tc::tma_load_2d(dst + c * 16384 + h * 8192, tm, 64 * c, rows[h], &full[st]);
          ++issued;
        }
      }
      if (!ok) stop(sm, a.dev_err);
      for (int i = max(0, issued - kWStages); i < issued; ++i) (void)tc::mbar_wait(&full[i % kWStages], (i / kWStages) & 1);
      if (is_k && seg > 0) (void)tc::mbar_wait(&sm.q_full, (seg - 1) & 1);
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------------ MMA issuers
    wide_regs_down<kWRegsMisc>();
    constexpr uint32_t idS = tc::idesc_bf16_f32(128, 128), idO = tc::idesc_bf16_f32_bmn(128, D);
    const int h = warp - 2;
    const uint32_t el = tc::elect_one();
    const uint32_t s = tS + h * 128, o = tO + h * 128;
    const uint64_t qd = tc::sdesc_sw128(tc::smem_u32(sm.q[h]));
    int it = 0, seg = 0, mine = 0;  // tiles and units of the CTA, and the tiles of this half
    bool ok = true;
    auto all = [&](bool v) { return __all_sync(0xffffffffu, v); };
    for (int at = rg.begin, un = rg.first_unit; ok && at < rg.end; ++un, ++seg) {
      const ChunkUnit u = load_unit(p, un);
      const int end = min(rg.end, u.prefix + u.ntiles);
      const bool here = h == 0 || u.ntok > half_tok;
      ok = all(tc::mbar_wait(&sm.q_full, seg & 1));
      // S of tile i of the CTA
      auto scores = [&](int i) -> bool {
        const int kv = i % kWStages;
        if (!all(tc::mbar_wait(&sm.k_full[kv], (i / kWStages) & 1))) return false;
        if (here) {
          tc::tc_fence_after();
          const uint64_t kd = tc::sdesc_sw128(tc::smem_u32(sm.k[kv]));
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t off = ((ks >> 2) * 16384u + (ks & 3) * 32u) >> 4;
            tc::mma_f16_warp(s, qd + off, kd + off, idS, ks > 0 ? 1u : 0u, el);
          }
          tc::mma_commit_warp(&sm.s_full[h], el);
          tc::mma_commit_warp(&sm.k_empty[kv], el);
        } else if (el) {
          tc::mbar_arrive(&sm.k_empty[kv]);
        }
        return true;
      };
      ok = ok && scores(it);
      // (the first P of a unit comes from the threads that have read the last unit out of O)
      for (int j = 0; ok && at < end; ++at, ++it, ++j) {
        const int kv = it % kWStages;
        ok = all(tc::mbar_wait(&sm.v_full[kv], (it / kWStages) & 1) &&
                 (!here || tc::mbar_wait(&sm.p_full[h], mine & 1)));
        if (!ok) break;
        if (here) {
          tc::tc_fence_after();
          const uint64_t vd = tc::sdesc_sw128_mn(tc::smem_u32(sm.v[kv]), 16384u, 1024u);
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            tc::mma_f16_ts_warp(o, s + ks * 8, vd + ks * 128, idO, (j > 0 || ks > 0) ? 1u : 0u, el);
          tc::mma_commit_warp(&sm.v_empty[kv], el);
          tc::mma_commit_warp(&sm.pv_done[h], el);
          ++mine;
        } else if (el) {
          tc::mbar_arrive(&sm.v_empty[kv]);
        }
        if (at + 1 < end) ok = scores(it + 1);
      }
      if (ok) {
        if (here) tc::mma_commit_warp(&sm.q_empty, el);
        else if (el) tc::mbar_arrive(&sm.q_empty);
      }
    }
    if (!ok && lane == 0) stop(sm, a.dev_err);
    if (mine > 0) (void)tc::mbar_wait(&sm.pv_done[h], (mine - 1) & 1);
    if (!ok) (void)tc::mbar_wait(&sm.s_full[h], mine & 1, 1000000ull);  // an S whose P never came
  } else {
    // ------------------------------------------------------------------ softmax warps
    wide_regs_up<kWRegsSoftmax>();
    const int h = (warp - 4) >> 2;
    const int qd = warp & 3, r = qd * 32 + lane;
    const uint32_t lane_off = (uint32_t)(qd * 32) << 16;
    const uint32_t s = tS + h * 128 + lane_off, o = tO + h * 128 + lane_off;
    bool ok = true;
    int it = 0, mine = 0;  // tiles of the CTA, and of them this half's
    const int tr = h * half_tok + (r >> a.log2G);  // the row's token of the unit
    for (int at = rg.begin, un = rg.first_unit; ok && at < rg.end; ++un) {
      const ChunkUnit u = load_unit(p, un);
      const int j0 = at - u.prefix, j1 = min(u.ntiles, rg.end - u.prefix);
      at = u.prefix + j1;
      if (h == 1 && u.ntok <= half_tok) {  // no second half
        it += j1 - j0;
        continue;
      }
      const int pos = u.pos0 + tr, pos_first = u.pos0 + h * half_tok, pos_last = u.pos0 + u.ntok - 1;
      const int32_t* bt = a.bt + (size_t)u.b * a.max_pages;
      float m_used = -INFINITY, l = 0.f;
      // page `lp` of the sequence: (factor of the logits or -1 where it is not there, log2 of V's);
      // of a bf16 cache the raw table entry, looked at a tile later when it has arrived
      auto page_params = [&](int lp) -> float2 {
        if (lp >= u.npages) return make_float2(EXP ? -1.f : __int_as_float(-1), 0.f);
        if (EXP) return params[(size_t)(u.slot_page + lp) * a.Hkv + u.g];
        return make_float2(__int_as_float(bt[lp]), 0.f);
      };
      float2 n0 = page_params(u.page0 + 2 * j0), n1 = page_params(u.page0 + 2 * j0 + 1);
      for (int j = j0; j < j1; ++j, ++it, ++mine) {
        float2 par[2] = {n0, n1};
        if (!EXP)
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int phys = __float_as_int(par[q].x);
            par[q].x = phys >= 0 && phys < a.num_pages ? 1.f : -1.f;
          }
        if (j + 1 < j1) n0 = page_params(u.page0 + 2 * j + 2), n1 = page_params(u.page0 + 2 * j + 3);
        if (!__all_sync(0xffffffffu, !stopped(sm) && tc::mbar_wait(&sm.s_full[h], mine & 1))) { ok = false; break; }
        tc::tc_fence_after();
        float x[128];
        {
          uint32_t raw[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tc::tmem_ld32_async(s + c * 32, raw[c]);
          tc::tmem_wait_ld(raw[3]);
#pragma unroll
          for (int c = 0; c < 3; ++c) tc::tmem_regs_ready(raw[c]);
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e) x[c * 32 + e] = __uint_as_float(raw[c][e]);
        }
        const int kb = (u.page0 + 2 * j) * kPage;  // the tile's first key
        if (kb + 127 > pos_first || (a.w > 0 && kb <= pos_last - a.w) || par[0].x < 0.f || par[1].x < 0.f) {
          const int hi = pos - kb, lo = a.w > 0 ? hi - a.w : -1;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            // a bit per key, one test each (two comparisons each: 37 us against 33 for chunks of 333 to
            // 1200 tokens with a window of 128, where every tile is masked)
            const uint32_t seen = par[q >> 1].x < 0.f ? 0u : bits_upto(hi - 32 * q) & ~bits_upto(lo - 32 * q);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(seen & (1u << e))) x[32 * q + e] = -INFINITY;
          }
        }
        // a page that is not there has no weights: any positive factor will do
        const float c0 = fabsf(par[0].x) * a.scale_log2, c1 = fabsf(par[1].x) * a.scale_log2;
        float t[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          t[q] = fmaxf(x[32 * q], x[32 * q + 1]);
#pragma unroll
          for (int e = 2; e < 32; e += 2) t[q] = max3(t[q], x[32 * q + e], x[32 * q + e + 1]);
        }
        const float m_new = max3(m_used, fmaxf(t[0], t[1]) * c0, fmaxf(t[2], t[3]) * c1);
        const bool need = m_new > m_used + kWRescale || (m_used == -INFINITY && m_new > -INFINITY);
        const float alpha = (need && m_used > -INFINITY) ? tc::ex2(m_used - m_new) : 1.f;
        if (need) m_used = m_new;
        l *= alpha;
        if (j > j0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          if (!__all_sync(0xffffffffu, tc::mbar_wait(&sm.pv_done[h], (mine - 1) & 1))) { ok = false; break; }
          tc::tc_fence_after();
#pragma unroll 1
          for (int k = 0; k < D / 32; ++k) {
            float ov[32];
            tc::tmem_ld32(o + k * 32, ov);
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] *= alpha;
            tc::tmem_st32(o + k * 32, ov);
          }
        }
        // p = 2^(x c - m) (a row with nothing visible yet: all zero), times the page's V factor
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float c = q ? c1 : c0;
          const float shift = m_used == -INFINITY ? 0.f : par[q].y - m_used;
          F2 sum{0.f, 0.f};
          uint32_t w[32];
#pragma unroll
          for (int e = 0; e < 64; e += 2) {
            F2 y = fma2({x[64 * q + e], x[64 * q + e + 1]}, {c, c}, {shift, shift});
            y.x = tc::ex2(y.x), y.y = tc::ex2(y.y);
            sum = add2(sum, y);
            w[e >> 1] = pack_bf16(y.x, y.y);
          }
          l += EXP ? (sum.x + sum.y) * tc::ex2(-par[q].y) : sum.x + sum.y;
          tc::tmem_st32u(s + q * 32, w);
        }
        if (!EXP && kb < u.t && kb + 128 > u.t) {
          // the sequence ends inside this tile: what lies behind it in the pool may be anything,
          // and 0 times a NaN is a NaN. Either half clears it before its own P.V
          if (!__all_sync(0xffffffffu, tc::mbar_wait(&sm.v_full[it % kWStages], (it / kWStages) & 1))) { ok = false; break; }
          const int from = u.t - kb, dead = 128 - from;
          for (int e = r; e < dead * 8 * NB; e += 128) {
            const int blk = e / (dead * 8), z = e % (dead * 8);
            *reinterpret_cast<uint4*>(sm.v[it % kWStages] + blk * 16384 + from * 128 + 16 * z) = make_uint4(0, 0, 0, 0);
          }
          tc::fence_async_smem();
        }
        tc::tc_fence_before();
        tc::mbar_arrive(&sm.p_full[h]);
      }
      if (!ok) break;
      // ---- the unit's (or this part's) output
      if (!__all_sync(0xffffffffu, !stopped(sm) && tc::mbar_wait(&sm.pv_done[h], (mine - 1) & 1))) { ok = false; break; }
      tc::tc_fence_after();
      const bool whole = j0 == 0 && j1 == u.ntiles;
      const bool live = tr < u.ntok;
      const int head = u.g * a.G + (r & (a.G - 1));
      const size_t row = (size_t)(u.row + tr) * a.Hq + head;
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
        f = chunk_factor(sc, den);
        if (a.lse && live) a.lse[row] = chunk_lse(den, M2);
      };
      if (whole) {
        float f;
        finish(m_used, l, f);
#pragma unroll 1
        for (int k = 0; k < D / 32; ++k) {
          float ov[32];
          tc::tmem_ld32(o + k * 32, ov);
          if (live) store(ov, f, k * 32);
        }
        tc::tc_fence_before();
      } else {
        const size_t at_p = (size_t)part_slot(u, per, blockIdx.x) * 2 * kWRows + h * kWRows + r;
        reinterpret_cast<float2*>(p.part_ml)[at_p] = make_float2(m_used, l);
        float* po = p.part_o + at_p * D;
#pragma unroll 1
        for (int k = 0; k < D / 32; ++k) {
          float ov[32];
          tc::tmem_ld32(o + k * 32, ov);
          if (live)
#pragma unroll
            for (int e = 0; e < 32; e += 8) store8(po + k * 32 + e, ov + e);
        }
        tc::tc_fence_before();
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
