// latent_chunk.cu — latent attention in the latent space (absorbed form) over a paged bf16 cache, on tcgen05.
//
// A cache row [c (DC) | r (64)] is key and value of all heads at once: x = scale q . [c, r], o = sum p c.
// With Hq heads a key's 2 (DC + 64) bytes meet 2 Hq (2 DC + 64) flops a token: single tokens of up to 64
// heads are bound by the bytes, 128 heads stand at the balance of the two, chunks by the tensor pipe.
//
// The keys take the MMAs' M side, as in chunk_narrow.cu: S^T[128 keys][N rows] = K Q^T and
// O^T[DC][N] += C^T P^T, N = 16, 32 or 64 rows (tokens times heads), so that O of 512 channels
// fits tensor memory (4 x 64 columns; with the rows as M it would take all 512) and a tile is read
// once: the same shared-memory tile is S's K-major A operand and, MN-major, O's. Units of 128 rows
// (Hq = 128, or chunks) go to a pair of CTAs, 64 rows each, that walk the same tiles side by side: either loads them
// whole, by plain copies, and fetches one of the two pages two tiles ahead into L2, so that HBM is read once
// (without: single tokens of 128 heads 142 us; both pages by either CTA 128, the mixed batch 243). Nothing passes
// from one CTA to the other.
//   64 single tokens of 16 heads over 16K to 32K keys (1.81 GB): 286 to 290 us with the merge, 0.92 to 0.93
//     of the copy bandwidth.
//   32 single tokens of 128 heads over 4K to 16K keys: 128 us, 0.71 PFLOP/s; 12 sequences of 1 to 200 tokens of
//     32 heads 239 us, 0.79. A tile takes some 5500 cycles there, 3700 of them products (48 cycles an MMA of 64 rows,
//     whose 6 KB of operands come from shared memory); with 64 rows of 512 channels a tile fills what
//     Q leaves of it, so that the softmax between them is not hidden.
//   warp 0   producer: the tile in DC / 128 pieces of 128 channels (32 KB) and one of the 64 rotated ones,
//            each with a barrier, through rings of pieces: with 64 rows of 512 channels a tile fills the
//            ring, and a piece of the next one comes as soon as its channels' O is done
//   warps 1, 3   MMA issuers, of S (piece by piece as they land) and of O (piece by piece, each
//            committed to the ring)
//   warp 2   Q of the next unit by TMA
//   warps 4-7, 8-11 (64 rows: to 19)  softmax, a key a thread, 8 or 16 rows each (32 each: 4 % slower):
//            p = 2^(x c + nm) with a reference nm per row that moves only when a weight would exceed 2^14; P
//            rounds to bf16, C's type (a weight is off by at most 2^-8 of itself), and goes where the tile's
//            rotated channels were, which S alone needs; the normaliser is summed in fp32 from unrounded p
// Units, ranges and merging as in chunk_plan.cuh, the plan found here where a call has few keys or few rows. Every
// wait is bounded; the four warps of a softmax group leave their loop together (they meet at a hardware barrier).
#include <cuda.h>

#include "chunk_plan.cuh"
#include "f32x2.cuh"
#include "keys_m.cuh"
#include "tc.cuh"

namespace hs2 {

namespace {

// `bytes` bytes from `src` on into L2 (both multiples of 16).
HS2_DEVI void l2_prefetch(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
constexpr int kAhead = 2;  // tiles

constexpr uint32_t kPiece = 32768, kRotPiece = 16384;

template <int DC, int N>
struct LatentSmem {
  static constexpr int PIECES = DC / 128;  // of a tile
  static constexpr int BLOCKS = DC / 64 + 1;
  // what 227 KB hold beside Q (of 256 channels: less than three tiles' pieces, see below)
  static constexpr int RING = N == 64 ? 4 : 5;
  static constexpr int ROT = DC == 512 && N >= 32 ? 1 : 2;
  static constexpr int O_BUFS = N == 64 ? 1 : 2;  // by the parity of the unit
  static constexpr int GROUPS = N == 64 ? 4 : 2;  // of four softmax warps, N / GROUPS rows each
  static constexpr int THREADS = 128 * (1 + GROUPS);
  uint8_t piece[RING][kPiece];   // [two blocks of 64 channels][128 keys][128 bytes]
  uint8_t rot[ROT][kRotPiece];   // [128 keys][128 bytes]: r, then P ([key][row])
  uint8_t q[BLOCKS * N * 128];
  alignas(16) float nm[N], alpha[N], factor[N];
  alignas(16) float warp_m[GROUPS][4][N / GROUPS], sums[GROUPS][4][N / GROUPS];
  uint64_t full[RING], empty[RING], rot_full[ROT], rot_empty[ROT];
  uint64_t s_full[2], s_empty[2], p_ready[2], pv_done[2], o_empty[O_BUFS], q_full, q_empty;
  ChunkUnit own[line_seqs(false)];
  ChunkRange own_range;
  uint32_t tmem_base;
  int abort;
};

}  // namespace

// PAIR: CTAs 2i and 2i + 1 take rows [0, 64) and [64, 128) of the units of range i. The second walks a unit's tiles
// also where it has no such rows: going ahead to its next unit instead took longer (mixed batch 248 us against 239).
template <int DC, int N, bool PAIR>
__global__ void __launch_bounds__(LatentSmem<DC, N>::THREADS, 1)
    latent_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k, const ChunkArgs a,
                        const ChunkPlan p) {
  using Sm = LatentSmem<DC, N>;
  constexpr int PIECES = Sm::PIECES, BLOCKS = Sm::BLOCKS, RING = Sm::RING, ROT = Sm::ROT, OB = Sm::O_BUFS;
  constexpr int NG = Sm::GROUPS, C = N / NG;  // softmax groups; columns (rows of the unit) of a thread
  constexpr uint32_t kObuf = PIECES * N;   // tensor memory columns of an O
  static_assert(128 + OB * kObuf <= 512, "tensor memory");
  static_assert(RING < 3 * PIECES, "at most two tiles between their S and their O: two phases of p_ready");
  extern __shared__ __align__(1024) uint8_t dsmem[];
  Sm& sm = *reinterpret_cast<Sm*>(dsmem + ((1024 - (tc::smem_u32(dsmem) & 1023)) & 1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = PAIR ? blockIdx.x >> 1 : blockIdx.x, row0 = PAIR ? (blockIdx.x & 1) * N : 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < RING; ++s) {
      tc::mbar_init(&sm.full[s], 1);
      tc::mbar_init(&sm.empty[s], 1);
    }
    for (int s = 0; s < ROT; ++s) {
      tc::mbar_init(&sm.rot_full[s], 1);
      tc::mbar_init(&sm.rot_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(&sm.s_full[s], 1);
      tc::mbar_init(&sm.s_empty[s], NG * 128);
      tc::mbar_init(&sm.p_ready[s], NG * 128);
      tc::mbar_init(&sm.pv_done[s], 1);
    }
    for (int s = 0; s < OB; ++s) tc::mbar_init(&sm.o_empty[s], NG * 128);
    tc::mbar_init(&sm.q_full, 1);
    tc::mbar_init(&sm.q_empty, 1);
    sm.abort = 0;
    tc::fence_mbar_init();
  }
  if (warp == 1) tc::tmem_alloc(&sm.tmem_base, 512);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  griddep_wait();
  bool listed;
  const ChunkRange rg = plan_range<line_seqs(PAIR)>(a, p, cta, sm.own, &sm.own_range, listed);
  const uint32_t tS = sm.tmem_base, tO = tS + 128;
  if (warp == 0) {
    // ------------------------------------------------------------------ producer
    int it = 0;
    bool ok = true;
    const int oob = a.num_pages * kPage;  // the row past the pool: zeros
    // 64 channels of the tile's two pages
    auto load = [&](uint8_t* to, int x, int ra, int rb, uint64_t* bar) {
      tc::tma_load_2d(to, &tm_k, x, ra, bar);
      tc::tma_load_2d(to + 8192, &tm_k, x, rb, bar);
    };
    for (int at = rg.begin, un = rg.first_unit; ok && at < rg.end; ++un) {
      const ChunkUnit u = load_unit(p, listed, sm.own, un);
      const int j0 = at - u.prefix, j1 = min(u.ntiles, rg.end - u.prefix);
      at = u.prefix + j1;
      const int32_t* bt = a.bt + (size_t)u.b * a.max_pages;
      const int page_end = min(u.npages, u.page0 + 2 * j1);
      // lane i has the table entry of page i of a block of 32 (16 tiles), and the next block's
      auto entry = [&](int c0) -> int {
        const int lp = u.page0 + 2 * c0 + lane;
        return lp < page_end ? bt[lp] : -1;
      };
      int raw = entry(j0);
      for (int c0 = j0; ok && c0 < j1; c0 += 16) {
        const bool there = raw >= 0 && raw < a.num_pages;
        if (!there && u.page0 + 2 * c0 + lane < page_end) flag_error(a.dev_err, HS2_DEV_BAD_PAGE);
        const int row = there ? raw * kPage : oob;
        raw = entry(c0 + 16);
        const int row_next = raw >= 0 && raw < a.num_pages ? raw * kPage : oob;
        const int c1 = min(j1, c0 + 16);
        for (int j = c0; ok && j < c1; ++j, ++it) {
          const int l0 = 2 * (j - c0);
          const int ra = __shfl_sync(0xffffffffu, row, l0), rb = __shfl_sync(0xffffffffu, row, l0 + 1);
          if constexpr (PAIR) {
            // this CTA's page of the tile kAhead on into L2
            const int l1 = l0 + 2 * kAhead + (row0 ? 1 : 0);
            const int here = __shfl_sync(0xffffffffu, row, l1 & 31), later = __shfl_sync(0xffffffffu, row_next, l1 & 31);
            const int ahead = l1 < 32 ? here : later;
            if (lane == 0 && ahead != oob)
              l2_prefetch(reinterpret_cast<const uint8_t*>(a.k) + (size_t)ahead * (2 * (DC + kLatentRot)), kPage * 2 * (DC + kLatentRot));
          }
          for (int c = 0; c < PIECES; ++c) {
            const int n = it * PIECES + c, st = n % RING;
            ok = __all_sync(0xffffffffu, !halted(sm) && tc::mbar_wait(&sm.empty[st], ((n / RING) & 1) ^ 1));
            if (!ok) break;
            if (lane == 0) {
              tc::mbar_arrive_expect_tx(&sm.full[st], kPiece);
#pragma unroll
              for (int x = 0; x < 2; ++x) load(sm.piece[st] + x * 16384, 128 * c + 64 * x, ra, rb, &sm.full[st]);
            }
          }
          if (!ok) break;
          const int st = it % ROT;
          ok = __all_sync(0xffffffffu, !halted(sm) && tc::mbar_wait(&sm.rot_empty[st], ((it / ROT) & 1) ^ 1));
          if (ok && lane == 0) {
            tc::mbar_arrive_expect_tx(&sm.rot_full[st], kRotPiece);
            load(sm.rot[st], DC, ra, rb, &sm.rot_full[st]);
          }
        }
      }
    }
    if (!ok && lane == 0) halt(sm, a.dev_err);
    // copies in flight land before the block leaves (of an aborted tile some pieces may not have been asked for)
    if (lane == 0) {
      const int n = it * PIECES;
      for (int i = max(0, n - RING); i < n; ++i) (void)tc::mbar_wait(&sm.full[i % RING], (i / RING) & 1);
      for (int i = max(0, it - ROT); i < it; ++i) (void)tc::mbar_wait(&sm.rot_full[i % ROT], (i / ROT) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ S^T = K Q^T
    constexpr uint32_t idS = narrow_idesc(true, N, false, false);
    const uint32_t el = tc::elect_one();
    const uint64_t qd = tc::sdesc_sw128(tc::smem_u32(sm.q));
    int it = 0, seg = 0;
    bool ok = true;
    auto all = [&](bool v) { return __all_sync(0xffffffffu, v); };
    for (int at = rg.begin, un = rg.first_unit; ok && at < rg.end; ++un) {
      const ChunkUnit u = load_unit(p, listed, sm.own, un);
      const int end = min(rg.end, u.prefix + u.ntiles);
      ok = all(tc::mbar_wait(&sm.q_full, seg & 1));
      for (; ok && at < end; ++at, ++it) {
        const int b = it & 1;
        ok = all(tc::mbar_wait(&sm.s_empty[b], ((it >> 1) & 1) ^ 1));
        // a block of 64 channels: Q's block `blk` against the keys' at kd
        auto block = [&](uint64_t kd, int blk) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            tc::mma_f16_warp(tS + b * 64, kd + ks * 2, qd + ((blk * (N * 128u) + ks * 32u) >> 4), idS, (blk > 0 || ks > 0) ? 1u : 0u,
                             el);
        };
#pragma unroll
        for (int c = 0; c < PIECES; ++c) {
          const int n = it * PIECES + c, st = n % RING;
          ok = ok && all(tc::mbar_wait(&sm.full[st], (n / RING) & 1));
          if (!ok) break;
          tc::tc_fence_after();
          const uint64_t kd = tc::sdesc_sw128(tc::smem_u32(sm.piece[st]));
          block(kd, 2 * c);
          block(kd + 1024, 2 * c + 1);
        }
        ok = ok && all(tc::mbar_wait(&sm.rot_full[it % ROT], (it / ROT) & 1));
        if (!ok) break;
        tc::tc_fence_after();
        block(tc::sdesc_sw128(tc::smem_u32(sm.rot[it % ROT])), BLOCKS - 1);
        tc::mma_commit_warp(&sm.s_full[b], el);
      }
      if (ok) tc::mma_commit_warp(&sm.q_empty, el);
      ++seg;
    }
    if (!ok && lane == 0) halt(sm, a.dev_err);
    if (it > 0) (void)tc::mbar_wait(&sm.s_full[(it - 1) & 1], ((it - 1) >> 1) & 1);
    if (!ok) (void)tc::mbar_wait(&sm.s_full[it & 1], (it >> 1) & 1, 1000000ull);  // an S that was begun
  } else if (warp == 3) {
    // ------------------------------------------------------------------ O^T += C^T P^T
    constexpr uint32_t idO = narrow_idesc(true, N, true, true);
    const uint32_t el = tc::elect_one();
    int it = 0, seg = 0;
    bool ok = true;
    for (int at = rg.begin, un = rg.first_unit; ok && at < rg.end; ++un) {
      const ChunkUnit u = load_unit(p, listed, sm.own, un);
      const int end = min(rg.end, u.prefix + u.ntiles);
      ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.o_empty[seg % OB], ((seg / OB) & 1) ^ 1));
      const uint32_t o = tO + (seg % OB) * kObuf;
      for (int j = 0; ok && at < end; ++at, ++it, ++j) {
        const int b = it & 1;
        ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.p_ready[b], (it >> 1) & 1));
        if (!ok) break;
        tc::tc_fence_after();
        const uint64_t pd = tc::sdesc_sw128_mn(tc::smem_u32(sm.rot[it % ROT]), 16384u, 1024u);
#pragma unroll
        for (int c = 0; c < PIECES; ++c) {
          const int st = (it * PIECES + c) % RING;
          const uint64_t vd = tc::sdesc_sw128_mn(tc::smem_u32(sm.piece[st]), 16384u, 1024u);
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)  // 16 keys each
            tc::mma_f16_warp(o + c * N, vd + ks * 128, pd + ks * 128, idO, (j > 0 || ks > 0) ? 1u : 0u, el);
          tc::mma_commit_warp(&sm.empty[st], el);
        }
        tc::mma_commit_warp(&sm.rot_empty[it % ROT], el);
        tc::mma_commit_warp(&sm.pv_done[b], el);
      }
      ++seg;
    }
    if (!ok && lane == 0) halt(sm, a.dev_err);
    if (it > 0) (void)tc::mbar_wait(&sm.pv_done[(it - 1) & 1], ((it - 1) >> 1) & 1);
  } else if (warp == 2) {
    // ------------------------------------------------------------------ Q
    int seg = 0;
    bool ok = true;
    for (int at = rg.begin, un = rg.first_unit; ok && at < rg.end; ++un) {
      const ChunkUnit u = load_unit(p, listed, sm.own, un);
      at = min(rg.end, u.prefix + u.ntiles);
      ok = __all_sync(0xffffffffu, !halted(sm) && tc::mbar_wait(&sm.q_empty, (seg & 1) ^ 1));
      if (!ok) break;
      if (lane == 0) {
        tc::mbar_arrive_expect_tx(&sm.q_full, BLOCKS * N * 128);
        for (int c = 0; c < BLOCKS; ++c)
          tc::tma_load_3d(sm.q + c * N * 128, &tm_q, 64 * c, row0 & (a.G - 1), u.row + (row0 >> a.log2G), &sm.q_full);
      }
      ++seg;
    }
    if (!ok && lane == 0) halt(sm, a.dev_err);
    if (seg > 0) (void)tc::mbar_wait(&sm.q_full, (seg - 1) & 1);
  } else {
    // ------------------------------------------------------------------ softmax
    const int grp = (warp - 4) >> 2, bar = 1 + grp;
    const int qd = warp & 3, key = qd * 32 + lane, tid = key;
    const uint32_t lane_off = (uint32_t)(qd * 32) << 16;
    const int n0 = grp * C;  // this group's rows of the CTA
    float* const nm = sm.nm + n0;
    float* const alpha = sm.alpha + n0;
    int it = 0, seg = 0;
    bool run = true;
    for (int at = rg.begin, un = rg.first_unit; run && at < rg.end; ++un) {
      const ChunkUnit u = load_unit(p, listed, sm.own, un);
      const int j0 = at - u.prefix, j1 = min(u.ntiles, rg.end - u.prefix);
      at = u.prefix + j1;
      const int32_t* bt = a.bt + (size_t)u.b * a.max_pages;
      const uint32_t o = tO + (seg % OB) * kObuf + n0;
      float l[C];
#pragma unroll
      for (int n = 0; n < C; ++n) l[n] = 0.f;
      if (tid < C) nm[tid] = kUnset;
      (void)any_of_128(bar, false);
      // the table entry of this key's page, a tile ahead
      auto entry = [&](int j) {
        const int lp = u.page0 + 2 * j + (qd >> 1);
        return lp < u.npages ? bt[lp] : -1;
      };
      int raw = entry(j0);
      bool good = true;
      for (int j = j0; j < j1; ++j, ++it) {
        const int b = it & 1, kb = (u.page0 + 2 * j) * kPage;
        const bool there = raw >= 0 && raw < a.num_pages;
        if (j + 1 < j1) raw = entry(j + 1);
        good = __all_sync(0xffffffffu, good && tc::mbar_wait(&sm.s_full[b], (it >> 1) & 1));
        tc::tc_fence_after();
        // exponents, -inf where the key is hidden
        float x[C];
        auto exponents = [&]() {
          tmem_cols<C>(tS + lane_off + b * 64 + n0, x);
          const float c = a.scale_log2;
#pragma unroll
          for (int n = 0; n < C; n += 4) {
            const float4 m = *reinterpret_cast<const float4*>(nm + n);
            const F2 a0 = fma2({x[n], x[n + 1]}, {c, c}, {m.x, m.y}), a1 = fma2({x[n + 2], x[n + 3]}, {c, c}, {m.z, m.w});
            x[n] = a0.x, x[n + 1] = a0.y, x[n + 2] = a1.x, x[n + 3] = a1.y;
          }
          if (kb + 127 > u.pos0 || !there) {
            // the first column whose token sees this key
            const int ago = kb + key - u.pos0;
            const int lo = !there || ago > 128 ? N : ago <= 0 ? 0 : (ago << a.log2G) - row0;
#pragma unroll
            for (int n = 0; n < C; ++n)
              if (n0 + n < lo) x[n] = -INFINITY;
          }
        };
        // the group's maxima over the 128 keys to warp_m
        auto maxima = [&]() {
#pragma unroll
          for (int n = 0; n < C; ++n) {
            float t;
            asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(t) : "f"(x[n]));
            if (lane == n) sm.warp_m[grp][qd][n] = t;
          }
          (void)any_of_128(bar, false);
        };
        auto top_of = [&](int n) {
          return fmaxf(fmaxf(sm.warp_m[grp][0][n], sm.warp_m[grp][1][n]), fmaxf(sm.warp_m[grp][2][n], sm.warp_m[grp][3][n]));
        };
        exponents();
        float t0 = fmaxf(x[0], x[1]), t1 = fmaxf(x[2], x[3]);
#pragma unroll
        for (int n = 4; n < C; n += 4) t0 = fmax3(t0, x[n], x[n + 1]), t1 = fmax3(t1, x[n + 2], x[n + 3]);
        if (any_of_128(bar, fmaxf(t0, t1) > kTop || !good || halted(sm))) {
          if (any_of_128(bar, !good || halted(sm))) {
            run = false;
            break;
          }
          // ---- some row's reference moves
          if (j > j0) maxima();  // at the first tile every row is unset
          bool fresh = false;
          if (tid < C) {
            const float t = j > j0 ? top_of(tid) : kUnset;
            float al = 1.f;
            if (t > kTop) {  // t = x c + nm: the new nm is 6 - x c
              const float old = nm[tid];
              if (old == kUnset) {  // x c is lost in the sum: the first reference comes from a second look
                fresh = true;
                nm[tid] = 0.f;
                al = 0.f;
              } else {
                const float to = old - t + kBias;
                nm[tid] = to;
                al = exp2f(to - old);
              }
            }
            alpha[tid] = al;
          }
          if (any_of_128(bar, fresh)) {
            exponents();
            maxima();
            if (fresh) {
              const float t = top_of(tid);
              nm[tid] = t > -INFINITY ? kBias - t : kUnset;
            }
            (void)any_of_128(bar, false);
          }
#pragma unroll
          for (int n = 0; n < C; ++n) l[n] *= alpha[n];
          if (j > j0) {
            good = __all_sync(0xffffffffu, tc::mbar_wait(&sm.pv_done[b ^ 1], ((it - 1) >> 1) & 1));
            tc::tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < PIECES; ++c) {
              float ov[C];
              tmem_cols<C>(o + lane_off + c * N, ov);
#pragma unroll
              for (int n = 0; n < C; ++n) ov[n] *= alpha[n];
              tmem_put<C>(o + lane_off + c * N, ov);
            }
          }
          (void)any_of_128(bar, false);  // alpha has been read
          exponents();
        }
        tc::tc_fence_before();
        tc::mbar_arrive(&sm.s_empty[b]);
        // ---- weights
        uint8_t* prow = sm.rot[it % ROT] + key * 128;
#pragma unroll
        for (int n = 0; n < C; n += 8) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const F2 pr{ex2_approx(x[n + 2 * i]), ex2_approx(x[n + 2 * i + 1])};
            const F2 sum = add2({l[n + 2 * i], l[n + 2 * i + 1]}, pr);
            l[n + 2 * i] = sum.x, l[n + 2 * i + 1] = sum.y;
            w[i] = pack_bf16(pr.x, pr.y);
          }
          *reinterpret_cast<uint4*>(prow + ((((n0 + n) >> 3) ^ (key & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (kb + 128 > u.t && kb + key >= u.t) {
          // what lies behind the sequence in the pool may be anything, and 0 times a NaN is a NaN:
          // each group clears its share of the channels
          for (int c = grp; c < 2 * PIECES; c += NG) {
            uint8_t* dead = sm.piece[(it * PIECES + (c >> 1)) % RING] + (c & 1) * 16384 + key * 128;
#pragma unroll
            for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(dead + 16 * i) = make_uint4(0, 0, 0, 0);
          }
        }
        tc::fence_async_smem();
        tc::mbar_arrive(&sm.p_ready[b]);
      }
      if (!run) break;
      // ---- the unit's (or this part's) output
      good = good && tc::mbar_wait(&sm.pv_done[(it - 1) & 1], ((it - 1) >> 1) & 1);
      good = __all_sync(0xffffffffu, good && !halted(sm));
      {
        float t[32];
#pragma unroll
        for (int n = 0; n < 32; ++n) t[n] = n < C ? l[n < C ? n : 0] : 0.f;
        const float s = transpose_sum32(t);
        if (lane < C) sm.sums[grp][qd][lane] = s;
      }
      if (any_of_128(bar, !good)) {
        run = false;
        break;
      }
      tc::tc_fence_after();
      const bool whole = j0 == 0 && j1 == u.ntiles;
      const int rows = (u.ntok << a.log2G) - row0;  // this CTA's
      auto out_row = [&](int n) -> size_t {
        return (size_t)(u.row + ((row0 + n) >> a.log2G)) * a.Hq + ((row0 + n) & (a.G - 1));
      };
      const size_t slot = whole ? 0 : (size_t)part_slot(u, listed ? sm.own_range.per : p.head[1], cta) * p.tile_rows + row0 + n0;
      if (tid < C) {
        const float M = nm[tid] == kUnset ? -INFINITY : -nm[tid];
        const float L = sm.sums[grp][0][tid] + sm.sums[grp][1][tid] + sm.sums[grp][2][tid] + sm.sums[grp][3][tid];
        if (whole) {
          const float sc = exp2_rel(M, M), den = L * sc;
          sm.factor[n0 + tid] = chunk_factor(sc, den);
          if (a.lse && n0 + tid < rows) a.lse[out_row(n0 + tid)] = chunk_lse(den, M);
        } else {
          sm.factor[n0 + tid] = 1.f;
          reinterpret_cast<float2*>(p.part_ml)[slot + tid] = make_float2(M, L);
        }
      }
      (void)any_of_128(bar, false);
#pragma unroll 1
      for (int c = 0; c < PIECES; ++c) {
        float v[C];
        tmem_cols<C>(o + lane_off + c * N, v);
        const int ch = c * 128 + tid;
        if (whole) {
#pragma unroll
          for (int n = 0; n < C; ++n) {
            if (n0 + n >= rows) continue;
            const size_t to = out_row(n0 + n) * DC + ch;
            const float f = v[n] * sm.factor[n0 + n];
            if (a.o_bf16) reinterpret_cast<__nv_bfloat16*>(a.o)[to] = __float2bfloat16(f);
            else reinterpret_cast<float*>(a.o)[to] = f;
          }
        } else {
          float* po = p.part_o + slot * DC + ch;
#pragma unroll
          for (int n = 0; n < C; ++n)
            if (n0 + n < rows) po[(size_t)n * DC] = v[n];
        }
      }
      tc::tc_fence_before();
      tc::mbar_arrive(&sm.o_empty[seg % OB]);
      (void)any_of_128(bar, false);  // the group's arrays are rewritten by the next unit
      ++seg;
    }
    if (!run && lane == 0) halt(sm, a.dev_err);
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) tc::tmem_dealloc(sm.tmem_base, 512);
}

template <int DC, int N, bool PAIR>
static cudaError_t launch_n(const CUtensorMap& tq, const CUtensorMap& tk, const ChunkArgs& a, const ChunkPlan& p, cudaStream_t s) {
  constexpr size_t sm = sizeof(LatentSmem<DC, N>) + 1024;
  static_assert(sm <= 227 * 1024, "shared memory of a CTA");
  auto kern = latent_chunk_kernel<DC, N, PAIR>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(PAIR ? 2 * p.ctas : p.ctas), dim3(LatentSmem<DC, N>::THREADS), sm, s, tq, tk, a, p);
}

template <int DC>
static cudaError_t launch_dc(const CUtensorMap& tq, const CUtensorMap& tk, const ChunkArgs& a, const ChunkPlan& p, cudaStream_t s) {
  switch (p.tile_rows) {
    case 16: return launch_n<DC, 16, false>(tq, tk, a, p, s);
    case 32: return launch_n<DC, 32, false>(tq, tk, a, p, s);
    case 64: return launch_n<DC, 64, false>(tq, tk, a, p, s);
    case 128: return launch_n<DC, 64, true>(tq, tk, a, p, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_latent_chunk(const CUtensorMap& tq, const CUtensorMap& tk, const ChunkArgs& a, const ChunkPlan& p, int dc,
                                cudaStream_t s) {
  return dc == 512 ? launch_dc<512>(tq, tk, a, p, s) : launch_dc<256>(tq, tk, a, p, s);
}

}  // namespace hs2
