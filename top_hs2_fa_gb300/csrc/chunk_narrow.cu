// chunk_narrow.cu — attention of few query rows per KV head (draft tokens, single tokens) on
// tcgen05, straight from the cache's codes.
//
// Bound by the cache's bytes: up to 64 rows share every key, so the keys take the MMAs' M side
// and the rows N = 16, 32 or 64 of it: S^T[128 keys][N] = K Q^T and O^T[d][N] += V^T P^T cost
// tensor time in proportion to N, and a thread of the softmax owns one key. Codes are
// converted once per key whatever N is (a scan that keeps the rows on the MMA's other side pays the
// conversions' instructions per 8 rows). Per 128-key tile, pipelined over rings:
//   warp 0       producer: TMA of the tile's two pages (codes, group scales)
//   warps 4-7, 8-11  operands, a key a thread: K's codes -> f16 (code * group scale, exact) ->
//                tensor memory, S's A operand; V's -> shared memory, O's A operand (MN-major),
//                rows that are not there as zeros. Waits, fences and arrivals cost a warp more
//                than the conversions (2200 cycles a tile, of which 500 convert). FP4: each group
//                takes K and V of every other tile (303 us with a group for K and one for V, 288
//                so, for 4 tokens of 64 sequences; 271 and 262 for single tokens). That holds a
//                ring stage longer, and FP8's ring has three: there one group takes K, the other
//                V (330 us the other way, 300 so, for single tokens)
//   warps 1, 3   MMA issuers, of S and of O: their waits overlap the other's instructions
//   warps 12-19  softmax, four warps for every other tile, each four with references, sums and
//                an O of their own (joined when the unit ends): p = 2^(x c + nm), nm = 6 - m per
//                row; P holds p S_v, S_v the V scale of the key's page, and the reference m moves
//                only when |p S_v| of a key that the row sees would exceed 2^14 (f16 P keeps what
//                is within 2^-30 of a row's largest, whatever other pages' scales are); the
//                normaliser is summed in fp32 from unrounded p, per thread
//   warp 2       Q of the next unit by TMA, then to f16 in place, with an exact power of two
//                where its values would leave f16's range
// A bf16 cache skips the conversions: its TMA tiles are the operands (bf16 Q, P).
// Measured, with plan and merge, 64 sequences of 16K to 32K keys, 32 heads over 4, d = 128: single tokens
// of bf16 471 us (1.02 of the copy bandwidth), FP8 296 (0.82), FP4 260 (0.52); 4 tokens of FP4 275
// (0.50). FP4 is bound by the instructions and waits around its operands, not by any one pipe:
// conversions fill 23 % of a tile's time, the MMAs 26 %.
// The page's K scale multiplies the logits; V's enters P, which rounds to f16, K's and V's type here
// (off by 2^-11 at most; over a bf16 cache to bf16, 2^-8). One V scale for all rows of a tile, P
// relative to the largest so far, cost 1 to 5 % more and lost rows whose own scales lie far below it.
// Units, ranges and merging as in chunk_plan.cuh. Every wait is bounded; the four softmax warps of a
// tile leave their loop together (they meet at a hardware barrier).
#include <cuda.h>
#include <cuda_fp16.h>

#include "chunk_plan.cuh"
#include "f32x2.cuh"
#include "keys_m.cuh"
#include "tc.cuh"

namespace hs2 {

namespace {

constexpr int kNThreads = 640;
// log2 |S_v| as the references take it. From below: p = 2^(14 - log2 |S_v|) at most, of which 2^24
// keys have to add up within fp32, and a scale of zero has to leave p finite.
constexpr float kLeastScale = -64.f, kMostScale = 127.f;
constexpr int kInfo = 16;        // tiles whose pages' scales are kept: more than the pipeline holds

struct __align__(16) TileInfo {
  float k[2], v[2];  // the two pages' slab scales (V's of a page that is not there: 0)
  int there[2];      // whether the page is there
  int pad[2];
};

template <int D, int FMT, int N>
struct NarrowSmem {
  static constexpr bool QUANT = FMT != HS2_BF16;
  static constexpr int RB = FMT == HS2_FP4_E2M1 ? D / 2 : FMT == HS2_FP8_E4M3 ? D : 2 * D;  // bytes of a row
  static constexpr int SF = FMT == HS2_FP4_E2M1 ? D / 16 : 0;                               // group scales of a row
  static constexpr int CODES = 128 * RB;
  static constexpr int STAGE = 2 * CODES + 2 * 128 * SF;
  static constexpr int STAGES = FMT == HS2_BF16 ? 2 : FMT == HS2_FP8_E4M3 ? (D == 128 && N == 64 ? 2 : 3) : D == 128 && N == 64 ? 4 : 5;
  static constexpr int VTILE = 128 * D * 2;
  static constexpr int NB = D / 64;
  uint8_t ring[STAGES][(STAGE + 1023) / 1024 * 1024];
  uint8_t v[QUANT ? 2 : 1][QUANT ? VTILE : 1024];
  uint8_t p[2][128 * 128];
  uint8_t q[2][NB * N * 128];
  // per softmax group (even and odd tiles): nm, the last change's factors, the four warps' maxima
  alignas(16) float nm[2][N], alpha[2][N], warp_m[2][4][N];
  // per unit, by its parity: each group's maxima, the sums of its four warps
  alignas(16) float out_m[2][2][N], out_l[2][2][4][N];
  TileInfo info[kInfo];
  float qmul[2];
  uint64_t info_full[kInfo];
  uint64_t ring_full[STAGES], ring_empty[STAGES];
  uint64_t k_full[2], s_full[2], s_empty[2], pv_ready[2], pv_done[2], q_full[2], q_empty[2], o_empty[2], out_ready[2], q_raw[2];
  uint32_t tmem_base;
  int abort;
};

// Registers per thread of the five 128-thread groups: 40 + 2 * 72 + 2 * 144 = 472 of the 5 * 96
// that the block is launched with.
constexpr int kRegsMisc = 40, kRegsCodes = 72, kRegsSoftmax = 144;
template <int R>
HS2_DEVI void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
HS2_DEVI void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }

HS2_DEVI void bulk_load(void* smem, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   tc::smem_u32(smem)),
               "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
               : "memory");
}

// 16-byte unit c of a row of RB bytes in a TMA tile swizzled by the row's width.
template <int RB>
HS2_DEVI int code_unit(int row, int c) {
  const int x = RB == 128 ? (row & 7) : RB == 64 ? ((row >> 1) & 3) : ((row >> 2) & 1);
  return row * RB + ((c ^ x) << 4);
}

// 32 (FP4) or 16 (FP8) consecutive channels, one 16-byte unit of codes, as f16 pairs.
template <int FMT>
HS2_DEVI void unit_to_f16(const uint4& w, uint32_t sf2, uint32_t* h) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
  if constexpr (FMT == HS2_FP4_E2M1) {
    const uint32_t s0 = e4m3_pair(sf2, sf2), s1 = e4m3_pair(sf2 >> 8, sf2 >> 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      fp4x8_to_f16x8(x[i], h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
#pragma unroll
      for (int j = 0; j < 4; ++j) h[4 * i + j] = hmul2(h[4 * i + j], i < 2 ? s0 : s1);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) fp8x4_to_f16x4(x[i], h[2 * i], h[2 * i + 1]);
  }
}

}  // namespace

template <int D, int FMT, int N>
__global__ void __launch_bounds__(kNThreads, 1)
    chunk_narrow_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k, 
                        const __grid_constant__ CUtensorMap tm_v, const ChunkArgs a, const ChunkPlan p) {
  using Sm = NarrowSmem<D, FMT, N>;
  constexpr bool QUANT = Sm::QUANT, BF = !QUANT;
  constexpr int ST = Sm::STAGES, NB = Sm::NB, CODES = Sm::CODES, SF = Sm::SF, RB = Sm::RB;
  constexpr int C = N < 32 ? N : 32;  // columns of a softmax step
  constexpr bool SPLIT = FMT == HS2_FP8_E4M3;  // K and V by a group each; else a group a tile
  extern __shared__ __align__(1024) uint8_t dsmem[];
  Sm& sm = *reinterpret_cast<Sm*>(dsmem + ((1024 - (tc::smem_u32(dsmem) & 1023)) & 1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      tc::mbar_init(&sm.ring_full[s], 1);
      tc::mbar_init(&sm.ring_empty[s], SPLIT ? 256 : QUANT ? 128 : 2);  // the tile's group or groups; bf16: the two MMAs
    }
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(&sm.k_full[s], 128);
      tc::mbar_init(&sm.s_full[s], 1);
      tc::mbar_init(&sm.s_empty[s], 128);
      tc::mbar_init(&sm.pv_ready[s], 256);  // V's and P's threads
      tc::mbar_init(&sm.pv_done[s], 1);
      tc::mbar_init(&sm.q_full[s], QUANT ? 32 : 1);
      tc::mbar_init(&sm.q_empty[s], 3);  // the last S of the unit, and the two groups' reads of qmul
      tc::mbar_init(&sm.o_empty[s], 256);
      tc::mbar_init(&sm.out_ready[s], 256);
    }
    for (int s = 0; s < kInfo; ++s) tc::mbar_init(&sm.info_full[s], 1);
    tc::mbar_init(&sm.q_raw[0], 1);
    tc::mbar_init(&sm.q_raw[1], 1);
    sm.abort = 0;
    tc::fence_mbar_init();
  }
  if (warp == 1) tc::tmem_alloc(&sm.tmem_base, 512);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  griddep_wait();
  const ChunkRange rg = chunk_range(p, blockIdx.x);
  const int per = p.head[1];
  const uint32_t tK = sm.tmem_base, tS = tK + 128, tO = tK + 256;  // two buffers; O: two groups by two units
  if (warp == 0) {
    // ------------------------------------------------------------------ producer
    regs_down<kRegsMisc>();
    // Lane i has the table entry and the scales of page i of a block of 32 (16 tiles); the next
    // block's are fetched while this one is issued.
    int issued = 0;
    bool ok = true;
    for (int at = rg.begin, un = rg.first_unit; ok && at < rg.end; ++un) {
      const ChunkUnit u = load_unit(p, un);
      const int j0 = at - u.prefix, j1 = min(u.ntiles, rg.end - u.prefix);
      at = u.prefix + j1;
      const int32_t* bt = a.bt + (size_t)u.b * a.max_pages;
      const int page_end = min(u.npages, u.page0 + 2 * j1);
      auto entry = [&](int c0) -> int {  // raw table entry of this lane's page of the block at tile c0
        const int lp = u.page0 + 2 * c0 + lane;
        return lp < page_end ? bt[lp] : -1;
      };
      auto valid = [&](int e) { return e >= 0 && e < a.num_pages; };
      int raw = entry(j0), raw_next = -1;
      float ks = 1.f, vs = 1.f, ks_next = 1.f, vs_next = 1.f;
      if (QUANT && valid(raw)) ks = a.k_scale[(size_t)raw * a.Hkv + u.g], vs = a.v_scale[(size_t)raw * a.Hkv + u.g];
      for (int c0 = j0; ok && c0 < j1; c0 += 16) {
        const int mine = valid(raw) ? raw : -1;
        if (mine < 0 && u.page0 + 2 * c0 + lane < page_end) flag_error(a.dev_err, HS2_DEV_BAD_PAGE);
        raw_next = entry(c0 + 16);
        const int c1 = min(j1, c0 + 16);
        for (int j = c0; j < c1; ++j) {
          if (QUANT && j == c0 + 8 && valid(raw_next)) {
            ks_next = a.k_scale[(size_t)raw_next * a.Hkv + u.g];
            vs_next = a.v_scale[(size_t)raw_next * a.Hkv + u.g];
          }
          const int st = issued % ST, l0 = 2 * (j - c0);
          const int ph0 = __shfl_sync(0xffffffffu, mine, l0), ph1 = __shfl_sync(0xffffffffu, mine, l0 + 1);
          if (!__all_sync(0xffffffffu, !halted(sm) && tc::mbar_wait(&sm.ring_empty[st], ((issued / ST) & 1) ^ 1))) {
            ok = false;
            break;
          }
          if (lane == 0) {
            uint8_t* s = sm.ring[st];
            uint64_t* bar = &sm.ring_full[st];
            if constexpr (QUANT) {
              const int pages = (ph0 >= 0) + (ph1 >= 0);
              if (pages) tc::mbar_arrive_expect_tx(bar, pages * (CODES + 128 * SF));
              else tc::mbar_arrive(bar);
              for (int h = 0; h < 2; ++h) {
                const int ph = h ? ph1 : ph0;
                if (ph < 0) continue;
                const int row = (ph * a.Hkv + u.g) * kPage;
                tc::tma_load_2d(s + h * (CODES / 2), &tm_k, 0, row, bar);
                tc::tma_load_2d(s + CODES + h * (CODES / 2), &tm_v, 0, row, bar);
                if constexpr (SF > 0) {
                  bulk_load(s + 2 * CODES + h * 64 * SF, a.k_sf + (size_t)row * SF, 64 * SF, bar);
                  bulk_load(s + 2 * CODES + 128 * SF + h * 64 * SF, a.v_sf + (size_t)row * SF, 64 * SF, bar);
                }
              }
            } else {
              const int oob = a.num_pages * a.Hkv * kPage;  // the row past the pool: zeros
              tc::mbar_arrive_expect_tx(bar, 2 * CODES);
              for (int h = 0; h < 2; ++h) {
                const int ph = h ? ph1 : ph0;
                const int row = ph >= 0 ? (ph * a.Hkv + u.g) * kPage : oob;
                for (int c = 0; c < NB; ++c) {
                  tc::tma_load_2d(s + c * 16384 + h * 8192, &tm_k, 64 * c, row, bar);
                  tc::tma_load_2d(s + CODES + c * 16384 + h * 8192, &tm_v, 64 * c, row, bar);
                }
              }
            }
          }
          // (the scales have arrived meanwhile)
          if ((lane >> 1) == j - c0) {
            TileInfo& f = sm.info[issued % kInfo];
            const bool here = mine >= 0;  // (else the scales may be those of an earlier page)
            f.k[lane & 1] = here ? ks : 1.f, f.v[lane & 1] = here ? vs : 0.f, f.there[lane & 1] = here;
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sm.info_full[issued % kInfo]);
          ++issued;
        }
        raw = raw_next, ks = ks_next, vs = vs_next;
      }
    }
    if (!ok && lane == 0) halt(sm, a.dev_err);
    if (lane == 0)
      for (int i = max(0, issued - ST); i < issued; ++i) (void)tc::mbar_wait(&sm.ring_full[i % ST], (i / ST) & 1);
  } else if (warp == 1) {
    // ------------------------------------------------------------------ S = K Q^T
    regs_down<kRegsMisc>();
    constexpr uint32_t idS = narrow_idesc(BF, N, false, false);
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
        const int b = it & 1, st = it % ST;
        ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.s_empty[b], ((it >> 1) & 1) ^ 1) &&
                                         (QUANT ? tc::mbar_wait(&sm.k_full[b], (it >> 1) & 1)
                                                : tc::mbar_wait(&sm.ring_full[st], (it / ST) & 1)));
        if (!ok) break;
        tc::tc_fence_after();
        const uint64_t kd = tc::sdesc_sw128(tc::smem_u32(sm.ring[st]));
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t qo = ((ks >> 2) * (N * 128u) + (ks & 3) * 32u) >> 4, ko = ((ks >> 2) * 16384u + (ks & 3) * 32u) >> 4;
          if (QUANT) tc::mma_f16_ts_warp(tS + b * 64, tK + b * 64 + ks * 8, qd + qo, idS, ks > 0 ? 1u : 0u, el);
          else tc::mma_f16_warp(tS + b * 64, kd + ko, qd + qo, idS, ks > 0 ? 1u : 0u, el);
        }
        tc::mma_commit_warp(&sm.s_full[b], el);
        if (!QUANT) tc::mma_commit_warp(&sm.ring_empty[st], el);
      }
      if (ok) tc::mma_commit_warp(&sm.q_empty[qb], el);
    }
    if (!ok && lane == 0) halt(sm, a.dev_err);
    if (it > 0) (void)tc::mbar_wait(&sm.s_full[(it - 1) & 1], ((it - 1) >> 1) & 1);
  } else if (warp == 3) {
    // ------------------------------------------------------------------ O^T += V^T P^T
    regs_down<kRegsMisc>();
    constexpr uint32_t idO = narrow_idesc(BF, N, true, true);
    const uint32_t el = tc::elect_one();
    int it = 0, seg = 0;
    bool ok = true;
    for (int at = rg.begin, un = rg.first_unit; ok && at < rg.end; ++un, ++seg) {
      const int2 pt = *reinterpret_cast<const int2*>(p.units + 12 * (size_t)un + 6);  // ntiles, prefix
      const int end = min(rg.end, pt.y + pt.x);
      ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.o_empty[seg & 1], ((seg >> 1) & 1) ^ 1));
      for (int j = 0; ok && at < end; ++at, ++it, ++j) {
        const int b = it & 1, st = it % ST;
        const uint32_t o = tO + ((seg & 1) * 2 + b) * 64;
        ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.pv_ready[b], (it >> 1) & 1));
        if (!ok) break;
        tc::tc_fence_after();
        const uint64_t vd = tc::sdesc_sw128_mn(QUANT ? tc::smem_u32(sm.v[b]) : tc::smem_u32(sm.ring[st] + CODES), 16384u, 1024u);
        const uint64_t pd = tc::sdesc_sw128_mn(tc::smem_u32(sm.p[b]), 16384u, 1024u);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)  // 16 keys each. D = 64: the upper 64 rows of M are not read back
          tc::mma_f16_warp(o, vd + ks * 128, pd + ks * 128, idO, (j > 1 || ks > 0) ? 1u : 0u, el);
        tc::mma_commit_warp(&sm.pv_done[b], el);
        if (!QUANT) tc::mma_commit_warp(&sm.ring_empty[st], el);
      }
    }
    if (!ok && lane == 0) halt(sm, a.dev_err);
    if (it > 0) (void)tc::mbar_wait(&sm.pv_done[(it - 1) & 1], ((it - 1) >> 1) & 1);
  } else if (warp == 2) {
    // ------------------------------------------------------------------ Q
    regs_down<kRegsMisc>();
    int seg = 0;
    bool ok = true;
    for (int at = rg.begin, un = rg.first_unit; ok && at < rg.end; ++un, ++seg) {
      const ChunkUnit u = load_unit(p, un);
      at = min(rg.end, u.prefix + u.ntiles);
      const int qb = seg & 1;
      ok = __all_sync(0xffffffffu, !halted(sm) && tc::mbar_wait(&sm.q_empty[qb], ((seg >> 1) & 1) ^ 1));
      if (!ok) break;
      uint64_t* landed = QUANT ? &sm.q_raw[qb] : &sm.q_full[qb];
      if (lane == 0) {
        tc::mbar_arrive_expect_tx(landed, NB * N * 128);
        for (int c = 0; c < NB; ++c) tc::tma_load_3d(sm.q[qb] + c * N * 128, &tm_q, 64 * c, u.g * a.G, u.row, landed);
      }
      ok = __all_sync(0xffffffffu, tc::mbar_wait(landed, (seg >> 1) & 1));
      if (!QUANT || !ok) continue;
      // In place: 16-byte unit i of the tile, whatever its place in a row, is row (i / 8) % N. The
      // largest exponent among the unit's own rows decides whether the values fit as they are.
      constexpr int UNITS = NB * N * 8;
      const int rows = u.ntok << a.log2G;
      uint4* q = reinterpret_cast<uint4*>(sm.q[qb]);
      uint32_t top = 0;
#pragma unroll 4
      for (int i = lane; i < UNITS; i += 32) {
        const uint4 w = q[i];
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
        if ((i >> 3) % N < rows)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t lo = (x[k] >> 7) & 0xFFu, hi = (x[k] >> 23) & 0xFFu;
            if (lo != 255u) top = max(top, lo);
            if (hi != 255u) top = max(top, hi);
          }
      }
      top = __reduce_max_sync(0xffffffffu, top);
      const int ex = max((int)top - 127, -100);
      // 1 for ordinary queries; else the largest exponent goes to 14
      const float mul = ex >= -2 && ex <= 14 ? 1.f : __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
#pragma unroll 4
      for (int i = lane; i < UNITS; i += 32) {
        uint4 w = q[i];
        uint32_t* x = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = pack_f16(bf16_lo(x[k]) * mul, bf16_hi(x[k]) * mul);
        q[i] = w;
      }
      if (lane == 0) sm.qmul[qb] = 1.f / mul;
      tc::fence_async_smem();
      tc::mbar_arrive(&sm.q_full[qb]);
    }
    if (!ok && lane == 0) halt(sm, a.dev_err);
  } else if (warp >= 4 && warp < 12) {
    // ------------------------------------------------------------------ K and V operands
    regs_down<kRegsCodes>();
    const int own = (warp - 4) >> 2;  // SPLIT: 0 for K, 1 for V; else the parity of this group's tiles
    const int qd = warp & 3, key = qd * 32 + lane;
    int it = 0;
    bool ok = true;
    auto all = [&](bool v) { return __all_sync(0xffffffffu, v); };
    for (int at = rg.begin, un = rg.first_unit; ok && at < rg.end; ++un) {
      const ChunkUnit u = load_unit(p, un);
      const int j0 = at - u.prefix, j1 = min(u.ntiles, rg.end - u.prefix);
      at = u.prefix + j1;
      for (int j = j0; j < j1; ++j, ++it) {
        if (!SPLIT && (it & 1) != own) continue;
        const int st = it % ST, b = it & 1;
        ok = all(!halted(sm) && tc::mbar_wait(&sm.info_full[it % kInfo], (it / kInfo) & 1) &&
                 tc::mbar_wait(&sm.ring_full[st], (it / ST) & 1));
        if (!ok) break;
        const bool live = sm.info[it % kInfo].there[qd >> 1] != 0 && (u.page0 + 2 * j) * kPage + key < u.t;
        if constexpr (QUANT) {
          constexpr int UN = RB / 16;      // 16-byte units of codes in a row
          constexpr int PER = D / UN / 2;  // f16 pairs of a unit
          uint4 w[UN];
          uint32_t sfw[2] = {0u, 0u};
          auto fetch = [&](int side) {  // this key's row: codes and group scales
            const uint8_t* codes = sm.ring[st] + side * CODES + (qd >> 1) * (CODES / 2);
            const uint8_t* sfp = sm.ring[st] + 2 * CODES + side * 128 * SF + key * SF;
#pragma unroll
            for (int c = 0; c < UN; ++c) w[c] = *reinterpret_cast<const uint4*>(codes + code_unit<RB>(key & 63, c));
            if constexpr (SF == 8) {
              const uint2 s8 = *reinterpret_cast<const uint2*>(sfp);
              sfw[0] = s8.x, sfw[1] = s8.y;
            } else if constexpr (SF == 4) {
              sfw[0] = *reinterpret_cast<const uint32_t*>(sfp);
            }
          };
          if (!SPLIT || own == 0) {
            fetch(0);
            // K's buffer is read by the S of two tiles ago
            ok = all(it < 2 || tc::mbar_wait(&sm.s_full[b], ((it - 2) >> 1) & 1));
            if (!ok) break;
            tc::tc_fence_after();
#pragma unroll
            for (int hb = 0; hb < D / 64; ++hb) {  // 64 channels, 32 columns
              uint32_t h[32];
              constexpr int CU = UN / (D / 64);
#pragma unroll
              for (int c = 0; c < CU; ++c) {
                const int cc = hb * CU + c;
                unit_to_f16<FMT>(w[cc], sfw[cc >> 1] >> (16 * (cc & 1)), h + c * PER);
              }
              if (SPLIT && hb == 0) tc::mbar_arrive(&sm.ring_empty[st]);
              tc::tmem_st32u(tK + ((uint32_t)(qd * 32) << 16) + b * 64 + hb * 32, h);
            }
            if (!SPLIT) fetch(1);
            tc::tc_fence_before();
            tc::mbar_arrive(&sm.k_full[b]);
          }
          if (SPLIT && own == 0) continue;
          if (SPLIT) fetch(1);
          if (!live) {  // a weight of 0 does not cancel what else may be there
#pragma unroll
            for (int c = 0; c < UN; ++c) w[c] = make_uint4(0, 0, 0, 0);
            sfw[0] = sfw[1] = 0u;
          }
          if (!SPLIT) tc::mbar_arrive(&sm.ring_empty[st]);
          // SPLIT: the tile before is handed over here, when its stores have long landed
          if (SPLIT && it > 0) {
            tc::fence_async_smem();
            tc::mbar_arrive(&sm.pv_ready[b ^ 1]);
          }
          // V's buffer is read by the P.V of two tiles ago
          ok = all(it < 2 || tc::mbar_wait(&sm.pv_done[b], ((it - 2) >> 1) & 1));
          if (!ok) break;
#pragma unroll
          for (int c = 0; c < UN; ++c) {
            uint32_t h[PER];
            unit_to_f16<FMT>(w[c], sfw[c >> 1] >> (16 * (c & 1)), h);
#pragma unroll
            for (int i = 0; i < PER / 4; ++i) {
              const int unit = c * (PER / 4) + i;  // of 8 channels
              *reinterpret_cast<uint4*>(sm.v[b] + (unit >> 3) * 16384 + key * 128 + (((unit & 7) ^ (key & 7)) << 4)) =
                  make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
            }
          }
          if (SPLIT) tc::mbar_arrive(&sm.ring_empty[st]);
        } else if (!live) {
          // bf16: the tile is the operand; rows behind the sequence may hold anything
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
            *reinterpret_cast<uint4*>(sm.ring[st] + CODES + (i >> 3) * 16384 + key * 128 + ((i & 7) << 4)) =
                make_uint4(0, 0, 0, 0);
        }
        if (!SPLIT) {
          tc::fence_async_smem();
          tc::mbar_arrive(&sm.pv_ready[b]);
        }
      }
    }
    if (SPLIT && own == 1 && ok && it > 0) {  // the last tile
      tc::fence_async_smem();
      tc::mbar_arrive(&sm.pv_ready[(it - 1) & 1]);
    }
    if (!ok && lane == 0) halt(sm, a.dev_err);
  } else if (warp >= 12) {
    // ------------------------------------------------------------------ softmax
    regs_up<kRegsSoftmax>();
    const int grp = (warp - 12) >> 2, bar = 1 + grp;
    const int qd = warp & 3, key = qd * 32 + lane, tid = key;
    const uint32_t lane_off = (uint32_t)(qd * 32) << 16;
    float* const nm = sm.nm[grp];
    float* const alpha = sm.alpha[grp];
    int it0 = 0, seg = 0;  // tiles of the units before
    bool run = true;
    for (int at = rg.begin, un = rg.first_unit; run && at < rg.end; ++un, ++seg) {
      const ChunkUnit u = load_unit(p, un);
      const int j0 = at - u.prefix, j1 = min(u.ntiles, rg.end - u.prefix);
      at = u.prefix + j1;
      const int pos_last = u.pos0 + u.ntok - 1, sp = seg & 1;
      const uint32_t o = tO + (sp * 2 + grp) * 64;
      const int jf = j0 + ((it0 + grp) & 1);  // this group's first tile: tile j of the line's number it0 + j - j0
      float l[N];
#pragma unroll
      for (int n = 0; n < N; ++n) l[n] = 0.f;
      if (tid < N) nm[tid] = kUnset;
      bool good = tc::mbar_wait(&sm.q_full[sp], (seg >> 1) & 1);
      const float cq = a.scale_log2 * (QUANT && good ? *(volatile float*)&sm.qmul[sp] : 1.f);
      (void)any_of_128(bar, false);  // nm is set, qmul has been read
      if (tid == 0) tc::mbar_arrive(&sm.q_empty[sp]);
      for (int j = jf; j < j1; j += 2) {
        const int it = it0 + j - j0, b = grp;
        good = good && tc::mbar_wait(&sm.info_full[it % kInfo], (it / kInfo) & 1) &&
               tc::mbar_wait(&sm.s_full[b], (it >> 1) & 1) &&
               (it < 2 || tc::mbar_wait(&sm.pv_done[b], ((it - 2) >> 1) & 1));  // P's buffer
        good = __all_sync(0xffffffffu, good);
        tc::tc_fence_after();
        const int pos = (u.page0 + 2 * j) * kPage + key;
        const TileInfo& f = sm.info[it % kInfo];
        const float vs = f.v[qd >> 1], c = cq * f.k[qd >> 1];
        // (NaN: as the least)
        const float lv = BF ? 0.f : fminf(fmaxf(log2f(fabsf(vs)), kLeastScale), kMostScale);
        const bool there = f.there[qd >> 1] != 0;
        const bool edge = (u.page0 + 2 * j) * kPage + 127 > u.pos0 || (a.w > 0 && (u.page0 + 2 * j) * kPage <= pos_last - a.w);
        // exponents of one step's columns, -inf where the key is hidden
        auto exponents = [&](int n0, float (&x)[C]) {
          tmem_cols<C>(tS + lane_off + b * 64 + n0, x);
#pragma unroll
          for (int n = 0; n < C; n += 4) {
            const float4 m = *reinterpret_cast<const float4*>(nm + n0 + n);
            const F2 a0 = fma2({x[n], x[n + 1]}, {c, c}, {m.x, m.y}), a1 = fma2({x[n + 2], x[n + 3]}, {c, c}, {m.z, m.w});
            x[n] = a0.x, x[n + 1] = a0.y, x[n + 2] = a1.x, x[n + 3] = a1.y;
          }
          if (edge || !there) {
            // columns (rows of the unit) that see this key: [lo, hi)
            const int ago = pos - u.pos0;  // tokens before this one do not
            const int lo = ago <= 0 ? 0 : min(ago, 64) << a.log2G;
            int hi = N;
            if (a.w > 0) hi = ago + a.w <= 0 ? 0 : min(ago + a.w, 64) << a.log2G;
            if (!there) hi = 0;
#pragma unroll
            for (int n = 0; n < C; ++n)
              if (n0 + n < lo || n0 + n >= hi) x[n] = -INFINITY;
          }
        };
        // the group's maxima over the 128 keys, with their V scales, to warp_m
        float x[C];
        auto maxima = [&]() {
#pragma unroll
          for (int n0 = 0; n0 < N; n0 += C) {
            exponents(n0, x);
#pragma unroll
            for (int n = 0; n < C; ++n) {
              float t;
              asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(t) : "f"(x[n]));
              if (lane == n) sm.warp_m[grp][qd][n0 + n] = t + lv;
            }
          }
          (void)any_of_128(bar, false);
        };
        auto top_of = [&](int n) {
          return fmaxf(fmaxf(sm.warp_m[grp][0][n], sm.warp_m[grp][1][n]), fmaxf(sm.warp_m[grp][2][n], sm.warp_m[grp][3][n]));
        };
        bool need = false;
#pragma unroll
        for (int n0 = 0; n0 < N; n0 += C) {
          exponents(n0, x);
          float t0 = fmaxf(x[0], x[1]), t1 = fmaxf(x[2], x[3]);
#pragma unroll
          for (int n = 4; n < C; n += 4) t0 = fmax3(t0, x[n], x[n + 1]), t1 = fmax3(t1, x[n + 2], x[n + 3]);
          need |= fmaxf(t0, t1) + lv > kTop;
        }
        bool moved = false;
        if (any_of_128(bar, need || !good || halted(sm))) {
          moved = true;
          if (any_of_128(bar, !good || halted(sm))) {
            run = false;
            break;
          }
          // ---- some row's reference moves
          if (j > jf) maxima();  // at the group's first tile every row is unset
          bool fresh = false;
          if (tid < N) {
            const float t = j > jf ? top_of(tid) : kUnset;
            float al = 1.f;
            if (t > kTop) {  // t = x c + lv + nm: the new nm is 6 - (x c + lv)
              const float old = nm[tid];
              if (old == kUnset) {  // x c is lost in the sum: the first reference comes from a second look
                fresh = true;
                nm[tid] = 0.f;
                al = 0.f;
              } else {
                const float to = old - t + kBias;
                nm[tid] = to;
                al = exp2f(to - old);  // (subnormals count: with scales far apart l can be large beside it)
              }
            }
            alpha[tid] = al;
          }
          if (any_of_128(bar, fresh)) {
            maxima();
            if (fresh) {
              const float t = top_of(tid);
              nm[tid] = t > -INFINITY ? kBias - t : kUnset;
            }
            (void)any_of_128(bar, false);
          }
#pragma unroll
          for (int n = 0; n < N; ++n) l[n] *= alpha[n];
          if (j > jf) {
            // O holds this group's tiles up to the last but this: P's buffer was waited for above
#pragma unroll 1
            for (int n0 = 0; n0 < N; n0 += C) {
              float ov[C];
              tmem_cols<C>(o + lane_off + n0, ov);
#pragma unroll
              for (int n = 0; n < C; ++n) ov[n] *= alpha[n0 + n];
              tmem_put<C>(o + lane_off + n0, ov);
            }
          }
          (void)any_of_128(bar, false);  // alpha has been read
        }
        if (N == C && !moved) {
          tc::tc_fence_before();
          tc::mbar_arrive(&sm.s_empty[b]);
        }
        // ---- weights
#pragma unroll
        for (int n0 = 0; n0 < N; n0 += C) {
          if (N > C || moved) exponents(n0, x);  // one step of columns is still in registers
#pragma unroll
          for (int n = 0; n < C; n += 8) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              F2 pr{ex2_approx(x[n + 2 * i]), ex2_approx(x[n + 2 * i + 1])};
              const F2 sum = add2({l[n0 + n + 2 * i], l[n0 + n + 2 * i + 1]}, pr);
              l[n0 + n + 2 * i] = sum.x, l[n0 + n + 2 * i + 1] = sum.y;
              if (!BF) pr = mul2(pr, {vs, vs});
              w[i] = BF ? pack_bf16(pr.x, pr.y) : pack_f16(pr.x, pr.y);
            }
            *reinterpret_cast<uint4*>(sm.p[b] + key * 128 + ((((n0 + n) >> 3) ^ (key & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        tc::tc_fence_before();
        if (N != C || moved) tc::mbar_arrive(&sm.s_empty[b]);
        tc::fence_async_smem();
        tc::mbar_arrive(&sm.pv_ready[b]);
      }
      if (!run) break;
      // ---- the unit's (or this part's) output: both groups' sums meet, each group writes half the rows
      const int nt = j1 - j0, last = it0 + nt - 1;
      const bool has0 = nt > 1 || (it0 & 1) == 0, has1 = nt > 1 || (it0 & 1) == 1;
      it0 += nt;
      if (has0) good = good && tc::mbar_wait(&sm.pv_done[0], ((last - (last & 1)) >> 1) & 1);
      if (has1) good = good && tc::mbar_wait(&sm.pv_done[1], ((last - 1 + (last & 1)) >> 1) & 1);
      good = __all_sync(0xffffffffu, good && !halted(sm));
      // the normaliser of every row, over the 32 keys of a warp
#pragma unroll
      for (int n0 = 0; n0 < N; n0 += C) {
        float t[32];
#pragma unroll
        for (int n = 0; n < 32; ++n) t[n] = n < C ? l[n0 + n] : 0.f;
        const float s = transpose_sum32(t);
        if (lane < C) sm.out_l[sp][grp][qd][n0 + lane] = s;
      }
      if (tid < N) sm.out_m[sp][grp][tid] = nm[tid] == kUnset ? -INFINITY : -nm[tid];
      tc::mbar_arrive(&sm.out_ready[sp]);
      good = __all_sync(0xffffffffu, good && tc::mbar_wait(&sm.out_ready[sp], (seg >> 1) & 1));
      if (any_of_128(bar, !good)) {
        run = false;
        break;
      }
      tc::tc_fence_after();
      const bool whole = j0 == 0 && j1 == u.ntiles;
      const int rows = u.ntok << a.log2G;
      constexpr int H = N / 2;  // rows of this group: [nb, nb + H)
      const int nb = grp * H;
      auto out_row = [&](int n) -> size_t { return (size_t)(u.row + (n >> a.log2G)) * a.Hq + (size_t)u.g * a.G + (n & (a.G - 1)); };
      // factor of row n's output, and its lse, from its max and sum
      auto finish = [&](int n, float M, float L) -> float {
        const float b2 = sink_b2(a.sink, u.g * a.G + (n & (a.G - 1)));
        const float M2 = fmaxf(M, b2), sc = exp2_rel(M, M2);
        const float den = L * sc + exp2_rel(b2, M2);
        if (a.lse && n < rows) a.lse[out_row(n)] = chunk_lse(den, M2);
        return chunk_factor(sc, den);
      };
      auto put = [&](int n, float v) {
        if (n < rows && tid < D) {
          const size_t at_o = out_row(n) * D + tid;
          if (a.o_bf16) reinterpret_cast<__nv_bfloat16*>(a.o)[at_o] = __float2bfloat16(v);
          else reinterpret_cast<float*>(a.o)[at_o] = v;
        }
      };
      // this thread's row (tid < H): both groups' max and sum; the groups' factors to warp_m
      float M = -INFINITY, L = 0.f;
      if (tid < H) {
        const int n = nb + tid;
        const float m0 = sm.out_m[sp][0][n], m1 = sm.out_m[sp][1][n];
        M = fmaxf(m0, m1);
        const float e0 = exp2_rel(m0, M), e1 = exp2_rel(m1, M);
        L = e0 * (sm.out_l[sp][0][0][n] + sm.out_l[sp][0][1][n] + sm.out_l[sp][0][2][n] + sm.out_l[sp][0][3][n]) +
            e1 * (sm.out_l[sp][1][0][n] + sm.out_l[sp][1][1][n] + sm.out_l[sp][1][2][n] + sm.out_l[sp][1][3][n]);
        const float f = whole ? finish(n, M, L) : 1.f;
        sm.warp_m[grp][0][tid] = e0 * f;
        sm.warp_m[grp][1][tid] = e1 * f;
      }
      (void)any_of_128(bar, false);
      // a group without tiles in this part left nothing in its O
      auto joined = [&](float (&v)[H]) {
#pragma unroll
        for (int n = 0; n < H; ++n) v[n] = 0.f;
        float t[H > 32 ? 32 : H];
        static_assert(H <= 32, "one step of columns");
#pragma unroll
        for (int g2 = 0; g2 < 2; ++g2) {
          if (!(g2 ? has1 : has0)) continue;
          if constexpr (H == 8) {
            float t16[16];
            tmem_cols<16>(tO + (sp * 2 + g2) * 64 + lane_off, t16);
#pragma unroll
            for (int n = 0; n < 8; ++n) t[n] = grp ? t16[8 + n] : t16[n];
          } else {
            tmem_cols<H>(tO + (sp * 2 + g2) * 64 + lane_off + nb, t);
          }
#pragma unroll
          for (int n = 0; n < H; ++n) v[n] = fmaf(sm.warp_m[grp][g2][n], t[n], v[n]);
        }
      };
      {
        float v[H];
        joined(v);
        tc::tc_fence_before();
        tc::mbar_arrive(&sm.o_empty[sp]);
        if (whole) {
#pragma unroll
          for (int n = 0; n < H; ++n) put(nb + n, v[n]);
        } else {
          const int slot = part_slot(u, per, blockIdx.x);
          if (tid < H) reinterpret_cast<float2*>(p.part_ml)[(size_t)slot * N + nb + tid] = make_float2(M, L);
          float* po = p.part_o + ((size_t)slot * N + nb) * D + tid;
          if (tid < D)
#pragma unroll
            for (int n = 0; n < H; ++n) po[(size_t)n * D] = v[n];
        }
      }
      (void)any_of_128(bar, false);  // the group's arrays are rewritten by the next unit
    }
    if (!run && lane == 0) halt(sm, a.dev_err);
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) tc::tmem_dealloc(sm.tmem_base, 512);
}

template <int D, int FMT, int N>
static cudaError_t launch_n(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const ChunkArgs& a, const ChunkPlan& p,
                            cudaStream_t s) {
  const size_t sm = sizeof(NarrowSmem<D, FMT, N>) + 1024;
  static_assert(sizeof(NarrowSmem<D, FMT, N>) + 1024 <= 227 * 1024, "shared memory of a CTA");
  auto kern = chunk_narrow_kernel<D, FMT, N>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sm);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(p.ctas), dim3(kNThreads), sm, s, tq, tk, tv, a, p);
}

template <int D, int FMT>
static cudaError_t launch_fmt(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const ChunkArgs& a, const ChunkPlan& p,
                              cudaStream_t s) {
  switch (p.tile_rows) {
    case 16: return launch_n<D, FMT, 16>(tq, tk, tv, a, p, s);
    case 32: return launch_n<D, FMT, 32>(tq, tk, tv, a, p, s);
    case 64: return launch_n<D, FMT, 64>(tq, tk, tv, a, p, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_chunk_narrow(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const ChunkArgs& a, const ChunkPlan& p,
                                int d, int dtype, cudaStream_t s) {
  if (d == 128) {
    return dtype == HS2_FP4_E2M1   ? launch_fmt<128, HS2_FP4_E2M1>(tq, tk, tv, a, p, s)
           : dtype == HS2_FP8_E4M3 ? launch_fmt<128, HS2_FP8_E4M3>(tq, tk, tv, a, p, s)
                                   : launch_fmt<128, HS2_BF16>(tq, tk, tv, a, p, s);
  }
  return dtype == HS2_FP4_E2M1   ? launch_fmt<64, HS2_FP4_E2M1>(tq, tk, tv, a, p, s)
         : dtype == HS2_FP8_E4M3 ? launch_fmt<64, HS2_FP8_E4M3>(tq, tk, tv, a, p, s)
                                 : launch_fmt<64, HS2_BF16>(tq, tk, tv, a, p, s);
}

}  // namespace hs2
