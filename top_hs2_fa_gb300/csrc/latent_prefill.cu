// latent_prefill.cu — latent attention over expanded keys and values (expanded form) on tcgen05.
//
// x = scale (q_n . k + q_r . r), o = softmax(x) v per head: 192 channels of K (128 of the head's, 64 that
// the heads share) and 128 of V, causal over packed sequences. Bound by the tensor pipe, 2 (192 + 128)
// flops per (row, key); a head's keys are read once per 256 rows. The scheme is chunk_wide.cu's: a
// unit is 256 tokens of a head, two halves of 128 rows that take turns on the tensor pipe, P as bf16 (a
// weight is off by at most 2^-8 of itself) over its tile's S. Q takes 96 KB of shared memory, a tile of
// K and V 80, and a half is done with one most of a tile's time after the other: K comes in blocks of 64
// channels through a ring of five, V 64 keys at a time through a ring of three, so that 1300 to 1500 cycles at
// least are left from the release of a piece to the next use of its place.
// A prompt of 16384 tokens of 16 heads: 843 to 867 us, 1.61 PFLOP/s, 0.84 of the burst rate; chunks of 333 to 1200
// tokens over up to 6100 keys, 32 heads, 349 to 357 us, 1.25 (their units whole by falling length; in equal
// ranges 923 to 937 and 404 to 411). A tile takes 3100 cycles (2560 at the tensor
// pipe's rate, which the MMAs' operands, 8 KB of shared memory in 64 cycles, allow barely), the end of a unit as
// much as two or three more.
//   warps 0, 1, 3   TMA producers of the K blocks, of V, of Q (each half as soon as its last S is done)
//   warp 2      issues all MMAs, the halves in turn: O_a += P_j V_j with P_j read from tensor memory, then
//               S_a of tile j + 1 over it, then b's. (A warp for each half let their instructions
//               mix, and both halves' softmaxes run at the same time: 5150 cycles a tile of 2560.)
//   warps 4-11, 12-19  softmax of half a, b: a row is two threads', 64 keys of the tile each. The reference
//               that they share moves only when it is exceeded by 2^8
// The 96 registers of the launch leave 72 bytes of spill stores a thread.
// TMEM: S of a [0,128), of b [128,256), O of a [256,384), of b [384,512). Every wait is bounded.
#include <cuda.h>

#include "chunk_plan.cuh"
#include "f32x2.cuh"
#include "keys_m.cuh"
#include "rows_m.cuh"
#include "tc.cuh"

namespace hs2 {

namespace {

constexpr int kPBlocks = (kLatentNope + kLatentRot) / 64;  // of a row of Q or K
constexpr int kPThreads = 640;
// Registers per thread: 128 * 56 + 512 * 104 of the 640 * 96 of the launch.
constexpr int kPRegsMisc = 56, kPRegsSoftmax = 104;
constexpr int kPKRing = 5, kPVRing = 3;
constexpr uint32_t kPBlock = 16384;                // 128 rows of 64 channels
constexpr uint32_t kPVHalf = 64 * kLatentValue * 2;  // 64 keys of V: two blocks of 64 channels

struct PrefillSmem {
  uint8_t q[2][kPBlocks * kPBlock];  // by half
  uint8_t k[kPKRing][kPBlock];
  uint8_t v[kPVRing][kPVHalf];
  uint64_t k_full[kPKRing], k_empty[kPKRing], v_full[kPVRing], v_empty[kPVRing];
  // by half
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], pv_done[2];
  float row[2][128];  // by half: what a row's two threads tell one another
  ChunkUnit own[kOwnUnits];
  ChunkRange own_range;
  uint32_t tmem_base;
  int abort;
};

// Barrier `id` of the 256 threads of a half: whether any of them passes true.
HS2_DEVI bool any_of_256(int id, bool v) {
  int r;
  asm volatile(
      "{.reg .pred p, q; setp.ne.b32 q, %1, 0;\n\tbar.red.or.pred p, %2, 256, q;\n\tselp.b32 %0, 1, 0, p;}"
      : "=r"(r)
      : "r"((int)v), "r"(id)
      : "memory");
  return r != 0;
}

}  // namespace

__global__ void __launch_bounds__(kPThreads, 1)
    latent_prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_r, const __grid_constant__ CUtensorMap tm_v, const ChunkArgs a,
                          const ChunkPlan p) {
  constexpr int D = kLatentValue;
  extern __shared__ __align__(1024) uint8_t dsmem[];
  PrefillSmem& sm = *reinterpret_cast<PrefillSmem*>(dsmem + ((1024 - (tc::smem_u32(dsmem) & 1023)) & 1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kPKRing; ++s) {
      tc::mbar_init(&sm.k_full[s], 1);
      tc::mbar_init(&sm.k_empty[s], 1);
    }
    for (int s = 0; s < kPVRing; ++s) {
      tc::mbar_init(&sm.v_full[s], 1);
      tc::mbar_init(&sm.v_empty[s], 1);
    }
    for (int h = 0; h < 2; ++h) {
      tc::mbar_init(&sm.q_full[h], 1);
      tc::mbar_init(&sm.q_empty[h], 1);
      tc::mbar_init(&sm.s_full[h], 1);
      tc::mbar_init(&sm.p_full[h], 256);
      tc::mbar_init(&sm.pv_done[h], 1);
    }
    sm.abort = 0;
    tc::fence_mbar_init();
  }
  griddep_wait();
  bool listed;
  const ChunkRange rg = plan_range<0>(a, p, blockIdx.x, sm.own, &sm.own_range, listed);
  if (rg.begin >= rg.end) return;  // nothing for this CTA (the whole block leaves)
  if (warp == 1) tc::tmem_alloc(&sm.tmem_base, kWTmem);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tS = sm.tmem_base, tO = tS + 256;

  if (warp == 0) {
    // ------------------------------------------------------------------ K
    wide_regs_down<kPRegsMisc>();
    if (lane == 0) {
      int issued = 0;  // blocks
      bool ok = true;
      for (int at = rg.begin, un = rg.first_unit; ok && at < rg.end; ++un) {
        const ChunkUnit u = load_unit(p, listed, sm.own, un);
        const int j0 = at - u.prefix, j1 = min(u.ntiles, rg.end - u.prefix);
        at = u.prefix + j1;
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
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ V
    wide_regs_down<kPRegsMisc>();
    if (lane == 0) {
      int issued = 0;
      bool ok = true;
      for (int at = rg.begin, un = rg.first_unit; ok && at < rg.end; ++un) {
        const ChunkUnit u = load_unit(p, listed, sm.own, un);
        const int j0 = at - u.prefix, j1 = min(u.ntiles, rg.end - u.prefix);
        at = u.prefix + j1;
        for (int j = 2 * j0; j < 2 * j1; ++j, ++issued) {
          const int st = issued % kPVRing;
          if (stopped(sm) || !tc::mbar_wait(&sm.v_empty[st], ((issued / kPVRing) & 1) ^ 1)) { ok = false; break; }
          tc::mbar_arrive_expect_tx(&sm.v_full[st], kPVHalf);
          for (int c = 0; c < 2; ++c)
            tc::tma_load_3d(sm.v[st] + c * (kPVHalf / 2), &tm_v, 64 * c, u.g, u.slot_page + 64 * j, &sm.v_full[st]);
        }
      }
      if (!ok) stop(sm, a.dev_err);
      for (int i = max(0, issued - kPVRing); i < issued; ++i) (void)tc::mbar_wait(&sm.v_full[i % kPVRing], (i / kPVRing) & 1);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------------ MMA issuer
    wide_regs_down<kPRegsMisc>();
    constexpr uint32_t idS = tc::idesc_bf16_f32(128, 128), idO = tc::idesc_bf16_f32_bmn(128, D);
    const uint32_t el = tc::elect_one();
    int seg[2] = {0, 0}, mine[2] = {0, 0};  // units with either half, and its tiles
    bool ok = true;
    auto all = [&](bool v) { return __all_sync(0xffffffffu, v); };
    const uint64_t q0 = tc::sdesc_sw128(tc::smem_u32(sm.q[0])), k0 = tc::sdesc_sw128(tc::smem_u32(sm.k[0]));
    const uint64_t v0 = tc::sdesc_sw128_mn(tc::smem_u32(sm.v[0]), kPVHalf / 2, 1024u);
    constexpr uint32_t kBlk = kPBlock >> 4, kVh = kPVHalf >> 4;
    // the places of the rings, and the phases that they are in
    int ks = 0, kp = 0, vs = 0, vp = 0;
    int next = fetch_unit(p, listed, sm.own, rg.first_unit, true);
    for (int at = rg.begin, un = rg.first_unit; ok && at < rg.end; ++un) {
      const ChunkUnit u = spread_unit(next);
      const int end = min(rg.end, u.prefix + u.ntiles);
      next = fetch_unit(p, listed, sm.own, un + 1, end < rg.end);
      const bool both = u.ntok > kWRows;
      // S of half h of the tile at the K ring's place
      auto scores = [&](int h, bool last) -> bool {
        int st = ks, ph = kp;
#pragma unroll
        for (int c = 0; c < kPBlocks; ++c) {
          if (h == 0) {
            if (!all(tc::mbar_wait(&sm.k_full[st], ph))) return false;
            tc::tc_fence_after();
          }
          tc::mma4_f16_warp<2, 2>(tS + h * 128, q0 + h * (kPBlocks * kBlk) + c * kBlk, k0 + st * kBlk, idS, c > 0 ? 1u : 0u, el);
          if (h == 1 || !both) tc::mma_commit_warp(&sm.k_empty[st], el);
          if (++st == kPKRing) st = 0, ph ^= 1;
        }
        tc::mma_commit_warp(&sm.s_full[h], el);
        if (last) tc::mma_commit_warp(&sm.q_empty[h], el);
        return true;
      };
      auto k_next = [&]() {
        ks += kPBlocks;
        if (ks >= kPKRing) ks -= kPKRing, kp ^= 1;
      };
      ok = all(tc::mbar_wait(&sm.q_full[0], seg[0]++ & 1)) && scores(0, at + 1 == end);
      if (ok && both) {
        ok = all(tc::mbar_wait(&sm.q_full[1], seg[1]++ & 1));
        tc::tc_fence_after();
        if (ok) (void)scores(1, at + 1 == end);
      }
      k_next();
      // (the first P of a unit comes from the threads that have read the last unit out of O)
      for (int j = 0; ok && at < end; ++at, ++j) {
        const bool more = at + 1 < end, last = at + 2 == end;
        // O += P V, 64 keys at a time (the second 64 may still be on their way)
        auto products = [&](int h) -> bool {
          int st = vs, ph = vp;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (h == 0) {
              if (!all(tc::mbar_wait(&sm.v_full[st], ph))) return false;
              tc::tc_fence_after();
            }
            tc::mma4_f16_ts_warp<8, 128>(tO + h * 128, tS + h * 128 + c * 32, v0 + st * kVh, idO, (j > 0 || c > 0) ? 1u : 0u, el);
            if (h == 1 || !both) tc::mma_commit_warp(&sm.v_empty[st], el);
            if (++st == kPVRing) st = 0, ph ^= 1;
          }
          tc::mma_commit_warp(&sm.pv_done[h], el);
          return true;
        };
        ok = all(tc::mbar_wait(&sm.p_full[0], mine[0] & 1)) && products(0);
        if (!ok) break;
        ++mine[0];
        if (more && !(ok = scores(0, last))) break;
        if (both) {
          ok = all(tc::mbar_wait(&sm.p_full[1], mine[1] & 1));
          if (!ok) break;
          tc::tc_fence_after();
          (void)products(1);
          ++mine[1];
          if (more) (void)scores(1, last);
        }
        if (more) k_next();
        vs += 2;
        if (vs >= kPVRing) vs -= kPVRing, vp ^= 1;
      }
    }
    if (!ok && lane == 0) stop(sm, a.dev_err);
    for (int h = 0; h < 2; ++h) {
      if (mine[h] > 0) (void)tc::mbar_wait(&sm.pv_done[h], (mine[h] - 1) & 1);
      if (!ok) (void)tc::mbar_wait(&sm.s_full[h], mine[h] & 1, 1000000ull);  // an S whose P never came
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------------ Q, a half as soon as its last S is done
    wide_regs_down<kPRegsMisc>();
    if (lane == 0) {
      int na = 0, nb = 0;  // units with half a, b
      bool ok = true;
      auto load = [&](int h, int n, const ChunkUnit& u) {
        if (stopped(sm) || !tc::mbar_wait(&sm.q_empty[h], (n & 1) ^ 1)) return false;
        tc::mbar_arrive_expect_tx(&sm.q_full[h], kPBlocks * kPBlock);
        for (int c = 0; c < kPBlocks; ++c)
          tc::tma_load_3d(sm.q[h] + c * kPBlock, &tm_q, 64 * c, u.g, u.row + h * kWRows, &sm.q_full[h]);
        return true;
      };
      for (int at = rg.begin, un = rg.first_unit; ok && at < rg.end; ++un) {
        const ChunkUnit u = load_unit(p, listed, sm.own, un);
        at = min(rg.end, u.prefix + u.ntiles);
        ok = load(0, na, u);
        na += ok;
        if (ok && u.ntok > kWRows) {
          ok = load(1, nb, u);
          nb += ok;
        }
      }
      if (!ok) stop(sm, a.dev_err);
      if (na > 0) (void)tc::mbar_wait(&sm.q_full[0], (na - 1) & 1);
      if (nb > 0) (void)tc::mbar_wait(&sm.q_full[1], (nb - 1) & 1);
    }
  } else {
    // ------------------------------------------------------------------ softmax warps
    wide_regs_up<kPRegsSoftmax>();
    const int h = (warp - 4) >> 3, cg = ((warp - 4) >> 2) & 1, bar = 1 + h;
    const int qd = warp & 3, r = qd * 32 + lane;
    const uint32_t lane_off = (uint32_t)(qd * 32) << 16;
    const uint32_t s = tS + h * 128 + lane_off, o = tO + h * 128 + cg * 64 + lane_off;
    bool ok = true;
    int it = 0, mine = 0;  // tiles of the CTA, and of them this half's
    const int tr = h * kWRows + r;  // the row's token of the unit
    const float c = a.scale_log2;
    const bool wide_out = ((uintptr_t)a.o & 31) == 0;
    int next = fetch_unit(p, listed, sm.own, rg.first_unit, true);
    for (int at = rg.begin, un = rg.first_unit; ok && at < rg.end; ++un) {
      const ChunkUnit u = spread_unit(next);
      const int j0 = at - u.prefix, j1 = min(u.ntiles, rg.end - u.prefix);
      at = u.prefix + j1;
      next = fetch_unit(p, listed, sm.own, un + 1, at < rg.end);
      if (h == 1 && u.ntok <= kWRows) {  // no second half
        it += j1 - j0;
        continue;
      }
      const int pos = u.pos0 + tr, pos_first = u.pos0 + h * kWRows;
      float m_used = -INFINITY, l = 0.f;
      for (int j = j0; j < j1; ++j, ++it, ++mine) {
        ok = ok && tc::mbar_wait(&sm.s_full[h], mine & 1);
        __syncwarp();
        tc::tc_fence_after();
        float x[64];
        {
          uint32_t raw[2][32];
          tc::tmem_ld32_async(s + cg * 64, raw[0]);
          tc::tmem_ld32_async(s + cg * 64 + 32, raw[1]);
          tc::tmem_wait_ld(raw[1]);
          tc::tmem_regs_ready(raw[0]);
#pragma unroll
          for (int e = 0; e < 64; ++e) x[e] = __uint_as_float(raw[e >> 5][e & 31]);
        }
        const int kb = 128 * j;  // the tile's first key
        if (kb + 127 > pos_first) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t seen = bits_upto(pos - kb - cg * 64 - 32 * q);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(seen & (1u << e))) x[32 * q + e] = -INFINITY;
          }
        }
        float t[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          t[q] = fmaxf(x[16 * q], x[16 * q + 1]);
#pragma unroll
          for (int e = 2; e < 16; e += 2) t[q] = max3(t[q], x[16 * q + e], x[16 * q + e + 1]);
        }
        const float top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * c;
        // The two threads of a row share its reference, which moves when either's part exceeds it by 2^8 (or
        // is the first that the row sees). After this barrier the whole half has read its S: P may go over it.
        if (any_of_256(bar, top > m_used + kWRescale || (m_used == -INFINITY && top > -INFINITY) || !ok || stopped(sm))) {
          if (cg) sm.row[h][r] = top;
          if (any_of_256(bar, !ok || stopped(sm))) { ok = false; break; }
          if (!cg) sm.row[h][r] = max3(m_used, top, sm.row[h][r]);
          (void)any_of_256(bar, false);
          const float m_new = sm.row[h][r];
          const bool need = m_new > m_used + kWRescale || (m_used == -INFINITY && m_new > -INFINITY);
          const float alpha = need && m_used > -INFINITY ? tc::ex2(m_used - m_new) : 1.f;
          if (need) m_used = m_new;
          l *= alpha;
          if (j > j0 && __any_sync(0xffffffffu, alpha != 1.f)) {
            ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.pv_done[h], (mine - 1) & 1));
            tc::tc_fence_after();
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
              float ov[16];
              tmem_cols<16>(o + k * 16, ov);
#pragma unroll
              for (int e = 0; e < 16; ++e) ov[e] *= alpha;
              tmem_put<16>(o + k * 16, ov);
            }
          }
          (void)any_of_256(bar, false);  // the maxima have been read
        }
        // p = 2^(x c - m) (a row with nothing visible yet: all zero)
        const float shift = m_used == -INFINITY ? 0.f : -m_used;
        {
          F2 sum{0.f, 0.f};
          uint32_t w[32];
#pragma unroll
          for (int e = 0; e < 64; e += 2) {
            F2 y = fma2({x[e], x[e + 1]}, {c, c}, {shift, shift});
            y.x = tc::ex2(y.x), y.y = tc::ex2(y.y);
            sum = add2(sum, y);
            w[e >> 1] = pack_bf16(y.x, y.y);
          }
          l += sum.x + sum.y;
          tc::tmem_st32u(s + cg * 32, w);
        }
        if (kb < u.t && kb + 128 > u.t) {
          // the sequence ends inside this tile: what lies behind it may be anything, and 0 times a NaN
          // is a NaN. Either half clears it before its own P.V
          bool landed = true;
          for (int n = 2 * it; n < 2 * it + 2; ++n) landed = landed && tc::mbar_wait(&sm.v_full[n % kPVRing], (n / kPVRing) & 1);
          ok = ok && landed;
          for (int e = (u.t - kb) * 16 + cg * 128 + r; ok && e < 128 * 16; e += 256) {
            const int key = e >> 4, blk = (e >> 3) & 1;
            *reinterpret_cast<uint4*>(sm.v[(2 * it + (key >> 6)) % kPVRing] + blk * (kPVHalf / 2) + (key & 63) * 128 + (e & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          tc::fence_async_smem();
          __syncwarp();
        }
        tc::tc_fence_before();
        tc::mbar_arrive(&sm.p_full[h]);
      }
      if (any_of_256(bar, !ok)) {
        ok = false;
        break;
      }
      // ---- the unit's (or this part's) output
      if (cg) sm.row[h][r] = l;
      ok = tc::mbar_wait(&sm.pv_done[h], (mine - 1) & 1);
      if (any_of_256(bar, !ok || stopped(sm))) { ok = false; break; }
      tc::tc_fence_after();
      if (!cg) sm.row[h][r] = l += sm.row[h][r];
      (void)any_of_256(bar, false);
      l = sm.row[h][r];
      const bool live = tr < u.ntok;
      if (j0 == 0 && j1 == u.ntiles) {
        const size_t row = (size_t)(u.row + tr) * a.Hq + u.g;
        auto put8 = [&](float* d, const float* x) {  // o may start on 16 bytes
          if (wide_out) return store8(d, x);
          reinterpret_cast<float4*>(d)[0] = make_float4(x[0], x[1], x[2], x[3]);
          reinterpret_cast<float4*>(d)[1] = make_float4(x[4], x[5], x[6], x[7]);
        };
        const float sc = exp2_rel(m_used, m_used), den = l * sc, f = chunk_factor(sc, den);
        if (a.lse && live && cg == 0) a.lse[row] = chunk_lse(den, m_used);
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
          float ov[32];
          tc::tmem_ld32(o + k * 32, ov);
          if (!live) continue;
          const size_t to = row * D + cg * 64 + k * 32;
          if (a.o_bf16) {
            float w[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) w[e / 2] = __uint_as_float(pack_bf16(ov[e] * f, ov[e + 1] * f));
            float* dst = reinterpret_cast<float*>(reinterpret_cast<__nv_bfloat16*>(a.o) + to);
            put8(dst, w);
            put8(dst + 8, w + 8);
          } else {
            float* dst = reinterpret_cast<float*>(a.o) + to;
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] *= f;
#pragma unroll
            for (int e = 0; e < 32; e += 8) put8(dst + e, ov + e);
          }
        }
      } else {
        // the plan's ranges, read here (kept in a register 0.5 to 1 % slower, with its spill): listed units are whole
        const size_t at_p = (size_t)part_slot(u, p.head[1], blockIdx.x) * 2 * kWRows + tr;
        if (cg == 0) reinterpret_cast<float2*>(p.part_ml)[at_p] = make_float2(m_used, l);
        float* po = p.part_o + at_p * D + cg * 64;
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
          float ov[32];
          tc::tmem_ld32(o + k * 32, ov);
          if (live)
#pragma unroll
            for (int e = 0; e < 32; e += 8) store8(po + k * 32 + e, ov + e);
        }
      }
      tc::tc_fence_before();
      (void)any_of_256(bar, false);  // the sums have been read
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
  return launch_pdl(latent_prefill_kernel, dim3(p.ctas), dim3(kPThreads), sm, s, tq, tk, tr, tv, a, p);
}

}  // namespace hs2
