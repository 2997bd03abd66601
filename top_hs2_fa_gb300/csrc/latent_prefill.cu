// latent_prefill.cu — latent attention over expanded keys and values (expanded form) on tcgen05.
//
// x = scale (q_n . k + q_r . r), o = softmax(x) v per head: 192 channels of K (128 of the head's, 64 that
// the heads share) and 128 of V, causal over packed sequences. Bound by the tensor pipe, 2 (192 + 128)
// flops per (row, key); a head's keys are read once per 256 rows. The scheme is chunk_wide.cu's: a
// unit is 256 tokens of a head, two halves of 128 rows that take turns on the tensor pipe, a softmax
// thread per row, P as bf16 (a weight is off by at most 2^-8 of itself) over its tile's S. Q takes
// 96 KB, so K comes in blocks of 64 channels through a ring of four (a tile is three, and a block of the next
// tile is asked for as soon as both halves are done with one), V in a ring of two tiles.
//   warp 0      TMA producer of Q and the K blocks; warp 1 of the V tiles
//   warps 2, 3  issue half a's and half b's MMAs: O += P_j V_j with P_j read from tensor memory,
//               then S_{j+1} = Q K^T over it
//   warps 4-7, 8-11  softmax of half a, b
// TMEM: S of a [0,128), of b [128,256), O of a [256,384), of b [384,512). Every wait is bounded.
#include <cuda.h>

#include "chunk_plan.cuh"
#include "f32x2.cuh"
#include "rows_m.cuh"
#include "tc.cuh"

namespace hs2 {

namespace {

constexpr int kPBlocks = (kLatentNope + kLatentRot) / 64;  // of a row of Q or K
constexpr int kPKRing = 4, kPVRing = 2;
constexpr uint32_t kPBlock = 16384;                // 128 rows of 64 channels
constexpr uint32_t kPVTile = 2 * kPBlock;

struct PrefillSmem {
  uint8_t q[2][kPBlocks * kPBlock];  // by half
  uint8_t k[kPKRing][kPBlock];
  uint8_t v[kPVRing][kPVTile];
  uint64_t q_full, q_empty, k_full[kPKRing], k_empty[kPKRing], v_full[kPVRing], v_empty[kPVRing];
  // by half
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint32_t tmem_base;
  int abort;
};

}  // namespace

__global__ void __launch_bounds__(kWThreads, 1)
    latent_prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_r, const __grid_constant__ CUtensorMap tm_v, const ChunkArgs a,
                          const ChunkPlan p) {
  constexpr int D = kLatentValue;
  extern __shared__ __align__(1024) uint8_t dsmem[];
  PrefillSmem& sm = *reinterpret_cast<PrefillSmem*>(dsmem + ((1024 - (tc::smem_u32(dsmem) & 1023)) & 1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    tc::mbar_init(&sm.q_full, 1);
    tc::mbar_init(&sm.q_empty, 2);  // the last S of either half
    for (int s = 0; s < kPKRing; ++s) {
      tc::mbar_init(&sm.k_full[s], 1);
      tc::mbar_init(&sm.k_empty[s], 2);  // S, P.V of either half
    }
    for (int s = 0; s < kPVRing; ++s) {
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

  if (warp == 0) {
    // ------------------------------------------------------------------ Q and K
    wide_regs_down<kWRegsMisc>();
    if (lane == 0) {
      int issued = 0, seg = 0;  // blocks
      bool ok = true;
      for (int at = rg.begin, un = rg.first_unit; ok && at < rg.end; ++un, ++seg) {
        const ChunkUnit u = load_unit(p, un);
        const int j0 = at - u.prefix, j1 = min(u.ntiles, rg.end - u.prefix);
        at = u.prefix + j1;
        if (!tc::mbar_wait(&sm.q_empty, (seg & 1) ^ 1)) { ok = false; break; }
        const int halves = u.ntok > kWRows ? 2 : 1;
        tc::mbar_arrive_expect_tx(&sm.q_full, halves * kPBlocks * kPBlock);
        for (int h = 0; h < halves; ++h)
          for (int c = 0; c < kPBlocks; ++c)
            tc::tma_load_3d(sm.q[h] + c * kPBlock, &tm_q, 64 * c, u.g, u.row + h * kWRows, &sm.q_full);
        for (int j = j0; ok && j < j1; ++j)
          for (int c = 0; c < kPBlocks; ++c, ++issued) {
            const int st = issued % kPKRing;
            if (stopped(sm) || !tc::mbar_wait(&sm.k_empty[st], ((issued / kPKRing) & 1) ^ 1)) { ok = false; break; }
            tc::mbar_arrive_expect_tx(&sm.k_full[st], kPBlock);
            const int row = u.slot_page + 128 * j;
            if (c < kPBlocks - 1) tc::tma_load_3d(sm.k[st], &tm_k, 64 * c, u.g, row, &sm.k_full[st]);
            else tc::tma_load_3d(sm.k[st], &tm_r, 0, 0, row, &sm.k_full[st]);
          }
      }
      if (!ok) stop(sm, a.dev_err);
      for (int i = max(0, issued - kPKRing); i < issued; ++i) (void)tc::mbar_wait(&sm.k_full[i % kPKRing], (i / kPKRing) & 1);
      if (seg > 0) (void)tc::mbar_wait(&sm.q_full, (seg - 1) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ V
    wide_regs_down<kWRegsMisc>();
    if (lane == 0) {
      int issued = 0;
      bool ok = true;
      for (int at = rg.begin, un = rg.first_unit; ok && at < rg.end; ++un) {
        const ChunkUnit u = load_unit(p, un);
        const int j0 = at - u.prefix, j1 = min(u.ntiles, rg.end - u.prefix);
        at = u.prefix + j1;
        for (int j = j0; j < j1; ++j, ++issued) {
          const int st = issued % kPVRing;
          if (stopped(sm) || !tc::mbar_wait(&sm.v_empty[st], ((issued / kPVRing) & 1) ^ 1)) { ok = false; break; }
          tc::mbar_arrive_expect_tx(&sm.v_full[st], kPVTile);
          for (int c = 0; c < 2; ++c)
            tc::tma_load_3d(sm.v[st] + c * kPBlock, &tm_v, 64 * c, u.g, u.slot_page + 128 * j, &sm.v_full[st]);
        }
      }
      if (!ok) stop(sm, a.dev_err);
      for (int i = max(0, issued - kPVRing); i < issued; ++i) (void)tc::mbar_wait(&sm.v_full[i % kPVRing], (i / kPVRing) & 1);
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
      const bool here = h == 0 || u.ntok > kWRows;
      ok = all(tc::mbar_wait(&sm.q_full, seg & 1));
      // S of tile i of the CTA, block by block
      auto scores = [&](int i) -> bool {
#pragma unroll
        for (int c = 0; c < kPBlocks; ++c) {
          const int n = i * kPBlocks + c, st = n % kPKRing;
          if (!all(tc::mbar_wait(&sm.k_full[st], (n / kPKRing) & 1))) return false;
          if (here) {
            tc::tc_fence_after();
            const uint64_t kd = tc::sdesc_sw128(tc::smem_u32(sm.k[st]));
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              tc::mma_f16_warp(s, qd + ((c * kPBlock + ks * 32u) >> 4), kd + ks * 2, idS, (c > 0 || ks > 0) ? 1u : 0u, el);
            tc::mma_commit_warp(&sm.k_empty[st], el);
          } else if (el) {
            tc::mbar_arrive(&sm.k_empty[st]);
          }
        }
        if (here) tc::mma_commit_warp(&sm.s_full[h], el);
        return true;
      };
      ok = ok && scores(it);
      // (the first P of a unit comes from the threads that have read the last unit out of O)
      for (int j = 0; ok && at < end; ++at, ++it, ++j) {
        const int st = it % kPVRing;
        ok = all(tc::mbar_wait(&sm.v_full[st], (it / kPVRing) & 1) && (!here || tc::mbar_wait(&sm.p_full[h], mine & 1)));
        if (!ok) break;
        if (here) {
          tc::tc_fence_after();
          const uint64_t vd = tc::sdesc_sw128_mn(tc::smem_u32(sm.v[st]), kPBlock, 1024u);
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            tc::mma_f16_ts_warp(o, s + ks * 8, vd + ks * 128, idO, (j > 0 || ks > 0) ? 1u : 0u, el);
          tc::mma_commit_warp(&sm.v_empty[st], el);
          tc::mma_commit_warp(&sm.pv_done[h], el);
          ++mine;
        } else if (el) {
          tc::mbar_arrive(&sm.v_empty[st]);
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
    const int tr = h * kWRows + r;  // the row's token of the unit
    for (int at = rg.begin, un = rg.first_unit; ok && at < rg.end; ++un) {
      const ChunkUnit u = load_unit(p, un);
      const int j0 = at - u.prefix, j1 = min(u.ntiles, rg.end - u.prefix);
      at = u.prefix + j1;
      if (h == 1 && u.ntok <= kWRows) {  // no second half
        it += j1 - j0;
        continue;
      }
      const int pos = u.pos0 + tr, pos_first = u.pos0 + h * kWRows;
      float m_used = -INFINITY, l = 0.f;
      for (int j = j0; j < j1; ++j, ++it, ++mine) {
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
        const int kb = 128 * j;  // the tile's first key
        if (kb + 127 > pos_first) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t seen = bits_upto(pos - kb - 32 * q);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(seen & (1u << e))) x[32 * q + e] = -INFINITY;
          }
        }
        const float c = a.scale_log2;
        float t[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          t[q] = fmaxf(x[32 * q], x[32 * q + 1]);
#pragma unroll
          for (int e = 2; e < 32; e += 2) t[q] = max3(t[q], x[32 * q + e], x[32 * q + e + 1]);
        }
        const float m_new = fmaxf(m_used, fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * c);
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
        // p = 2^(x c - m) (a row with nothing visible yet: all zero)
        const float shift = m_used == -INFINITY ? 0.f : -m_used;
#pragma unroll
        for (int q = 0; q < 4; q += 2) {
          F2 sum{0.f, 0.f};
          uint32_t w[32];
#pragma unroll
          for (int e = 0; e < 64; e += 2) {
            F2 y = fma2({x[32 * q + e], x[32 * q + e + 1]}, {c, c}, {shift, shift});
            y.x = tc::ex2(y.x), y.y = tc::ex2(y.y);
            sum = add2(sum, y);
            w[e >> 1] = pack_bf16(y.x, y.y);
          }
          l += sum.x + sum.y;
          tc::tmem_st32u(s + q * 16, w);
        }
        if (kb < u.t && kb + 128 > u.t) {
          // the sequence ends inside this tile: what lies behind it may be anything, and 0 times a NaN
          // is a NaN. Either half clears it before its own P.V
          const int st = it % kPVRing;
          if (!__all_sync(0xffffffffu, tc::mbar_wait(&sm.v_full[st], (it / kPVRing) & 1))) { ok = false; break; }
          const int from = u.t - kb, dead = 128 - from;
          for (int e = r; e < dead * 16; e += 128) {
            const int blk = e / (dead * 8), z = e % (dead * 8);
            *reinterpret_cast<uint4*>(sm.v[st] + blk * kPBlock + from * 128 + 16 * z) = make_uint4(0, 0, 0, 0);
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
      const bool live = tr < u.ntok;
      if (j0 == 0 && j1 == u.ntiles) {
        const size_t row = (size_t)(u.row + tr) * a.Hq + u.g;
        const float sc = exp2_rel(m_used, m_used), den = l * sc, f = chunk_factor(sc, den);
        if (a.lse && live) a.lse[row] = chunk_lse(den, m_used);
#pragma unroll 1
        for (int k = 0; k < D / 32; ++k) {
          float ov[32];
          tc::tmem_ld32(o + k * 32, ov);
          if (!live) continue;
          if (a.o_bf16) {
            uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.o) + row * D + k * 32);
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              dst[e / 8] = make_uint4(pack_bf16(ov[e] * f, ov[e + 1] * f), pack_bf16(ov[e + 2] * f, ov[e + 3] * f),
                                      pack_bf16(ov[e + 4] * f, ov[e + 5] * f), pack_bf16(ov[e + 6] * f, ov[e + 7] * f));
          } else {
            float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.o) + row * D + k * 32);
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              dst[e / 4] = make_float4(ov[e] * f, ov[e + 1] * f, ov[e + 2] * f, ov[e + 3] * f);
          }
        }
      } else {
        const size_t at_p = (size_t)part_slot(u, per, blockIdx.x) * 2 * kWRows + tr;
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
      }
      tc::tc_fence_before();
    }
    if (!ok && !stopped(sm)) stop(sm, a.dev_err);
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) tc::tmem_dealloc(sm.tmem_base, kWTmem);
}

cudaError_t launch_latent_prefill(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tr, const CUtensorMap& tv,
                                  const ChunkArgs& a, const ChunkPlan& p, cudaStream_t s) {
  constexpr size_t sm = sizeof(PrefillSmem) + 1024;
  static_assert(sm <= 227 * 1024, "shared memory of a CTA");
  cudaError_t e = cudaFuncSetAttribute(latent_prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm);
  if (e != cudaSuccess) return e;
  return launch_pdl(latent_prefill_kernel, dim3(p.ctas), dim3(kWThreads), sm, s, tq, tk, tr, tv, a, p);
}

}  // namespace hs2
