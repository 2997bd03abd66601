// chunk_plan.cuh — how the work of a chunk-attention call is cut among the CTAs of its kernels.
//
// The batch's queries form units: a KV head g of a sequence and up to TOK of its tokens, whose
// TOK * G rows (token-major, then the head's query heads) share the head's keys. A unit walks
// the 128-key tiles (two pages) that its rows see. The tiles of all units, one after another,
// are a line of `total` tiles that the CTAs of a persistent kernel share out in equal ranges,
// so lengths and batch sizes do not matter to the balance; a unit cut by a range border leaves
// partial results, which a last kernel merges in CTA order (chunk_merge.cu). Where every unit is
// short against a range (a sliding window), the borders move to the nearest unit's and cut none.
// Latent attention's plans hand out whole units by falling length instead where the CTAs' sums come out
// nearly as even, and calls with few keys have no planning kernel (plan_ordered, plan_own below).
#pragma once
#include "common.cuh"
#include "kernels.h"

namespace hs2 {

struct __align__(16) ChunkUnit {
  int b, g, row, ntok;                // row: packed row of the first token
  int pos0, page0, ntiles, prefix;    // position of the first token; first page; tiles before this unit
  int t, slot_page, npages, pad;      // keys; the sequence's first expanded page (packed keys: its first key); pages of the sequence
};

// Where a CTA's range meets the units.
struct ChunkRange {
  int first_unit, begin, end;
};

HS2_DEVI ChunkRange chunk_range(const ChunkPlan& p, int cta) {
  ChunkRange r;
  const int total = p.head[0], first = p.cta_first[cta], begin = p.cta_begin[cta];  // one round of loads
  const int next = p.cta_begin[min(cta + 1, p.ctas - 1)];
  r.begin = min(total, begin);
  r.end = cta + 1 < p.ctas ? min(total, next) : total;
  r.first_unit = r.begin < r.end ? first : 0;
  return r;
}

HS2_DEVI ChunkUnit load_unit(const ChunkPlan& p, int u) {
  ChunkUnit x;
  const int4* s = reinterpret_cast<const int4*>(p.units) + 3 * (size_t)u;
  int4* d = reinterpret_cast<int4*>(&x);
  d[0] = __ldcg(s);
  d[1] = __ldcg(s + 1);
  d[2] = __ldcg(s + 2);
  return x;
}

// Calls of up to 32 sequences whose units are few and stay whole need no planning kernel: unit i of the batch is
// CTA i % ctas's, and a warp of it writes the records of its units, at most kOwnUnits, one after another on
// a line of their own. Returns the line's length. Checks and flags as the planning kernel.
constexpr int kOwnUnits = kOwnPlanUnits;
static_assert(kOwnPlanSeqs == 32, "a lane a sequence");
HS2_DEVI int plan_own(const ChunkArgs& a, const ChunkPlan& p, int cta, ChunkUnit* own) {
  const int lane = threadIdx.x & 31, tok = p.tile_rows / a.G;
  int n = 0, t = 0, r0 = 0, k0 = 0;
  bool descends = false;
  if (lane < a.batch) {
    r0 = a.row_start[lane];
    const int r1 = a.row_start[lane + 1];
    descends = r1 < r0;
    if (a.key_start) {
      k0 = a.key_start[lane];
      const int k1 = a.key_start[lane + 1];
      t = k0 >= 0 && k1 >= k0 && k1 <= a.n_keys ? k1 - k0 : -1;
    } else {
      t = a.seq_len[lane];
    }
    n = r1 - r0;
  }
  bool bad = false;
  if (__any_sync(0xffffffffu, descends)) {
    bad = true;
    n = 0;
  } else if (n != 0 && (r0 < 0 || n > a.max_n || t < n || t > a.max_t || r0 > a.n_rows - n)) {
    bad = true;
    n = 0;
  }
  if (bad && cta == 0) flag_error(a.dev_err, HS2_DEV_BAD_LENGTH);
  const int per_head = (n + tok - 1) / tok, units = per_head * a.Hkv;
  int end = units;  // units of this and the sequences before
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, end, s);
    if (lane >= s) end += v;
  }
  const int total = __shfl_sync(0xffffffffu, end, 31);
  int line = 0;
  for (int i = 0, u = cta; i < kOwnUnits && u < total; ++i, u += p.ctas) {
    const int b = __popc(__ballot_sync(0xffffffffu, end <= u));  // the first sequence that ends behind u
    const int sn = __shfl_sync(0xffffffffu, n, b), st = __shfl_sync(0xffffffffu, t, b), row = __shfl_sync(0xffffffffu, r0, b);
    const int key = __shfl_sync(0xffffffffu, k0, b), ph = __shfl_sync(0xffffffffu, per_head, b);
    const int k = u - __shfl_sync(0xffffffffu, end - units, b), tile = k % ph;
    ChunkUnit x{};
    x.b = b;
    x.g = k / ph;
    x.row = row + tile * tok;
    x.ntok = min(tok, sn - tile * tok);
    x.pos0 = st - sn + tile * tok;
    x.ntiles = (x.pos0 + x.ntok - 1) / (2 * kPage) + 1;
    x.prefix = line;
    x.t = st;
    x.slot_page = key;
    x.npages = (st + kPage - 1) / kPage;
    if (lane == 0) own[i] = x;
    line += x.ntiles;
  }
  return line;
}

// The units of a CTA where the plan has them whole by falling length: the CTAs take them in turn, there and
// back. As plan_own.
HS2_DEVI int ordered_unit(int i, int cta, int ctas) { return i * ctas + (i & 1 ? ctas - 1 - cta : cta); }
HS2_DEVI int plan_ordered(const ChunkPlan& p, int units, int cta, ChunkUnit* own) {
  const int lane = threadIdx.x & 31, i = ordered_unit(lane, cta, p.ctas);
  const bool have = lane < kOwnUnits && i < units;
  ChunkUnit x{};
  if (have) x = load_unit(p, __ldcg(&p.order[i].x));
  int end = have ? x.ntiles : 0;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, end, s);
    if (lane >= s) end += v;
  }
  x.prefix = end - x.ntiles;
  if (have) own[lane] = x;
  return __shfl_sync(0xffffffffu, end, 31);
}

// What a CTA walks: units of its own in `own` (listed), or a range of the line.
HS2_DEVI ChunkRange plan_range(const ChunkArgs& a, const ChunkPlan& p, int cta, ChunkUnit* own, int* own_end, int* listed) {
  const int ordered = p.own || !p.order ? 0 : p.head[3];
  if (!p.own && !ordered) {
    if (threadIdx.x == 0) *listed = 0;
    __syncthreads();
    return chunk_range(p, cta);
  }
  if (threadIdx.x < 32) {
    const int end = p.own ? plan_own(a, p, cta, own) : plan_ordered(p, ordered, cta, own);
    if (threadIdx.x == 0) *own_end = end, *listed = 1;
  }
  __syncthreads();
  ChunkRange r{0, 0, *own_end};
  return r;
}

// A unit's record spread over a warp, a word a lane, so that the next unit's can be on its way while
// this one's tiles are walked; `there`: whether there is one. (listed: own holds the CTA's records)
HS2_DEVI int fetch_unit(const ChunkPlan& p, bool listed, const ChunkUnit* own, int u, bool there) {
  const int lane = threadIdx.x & 31;
  if (!there || lane >= 12) return 0;
  return listed ? reinterpret_cast<const int*>(own)[12 * u + lane] : __ldcg(p.units + 12 * (size_t)u + lane);
}
HS2_DEVI ChunkUnit load_unit(const ChunkPlan& p, bool listed, const ChunkUnit* own, int u) {
  return listed ? own[u] : load_unit(p, u);
}
HS2_DEVI ChunkUnit spread_unit(int word) {
  ChunkUnit x;
  int* d = reinterpret_cast<int*>(&x);
#pragma unroll
  for (int i = 0; i < 11; ++i) d[i] = __shfl_sync(0xffffffffu, word, i);
  return x;
}

// A row's results from its denominator, relative to 2^M: 0 where no key is left, NaN passes on.
HS2_DEVI float chunk_lse(float den, float M) { return den == 0.f ? -INFINITY : (M + log2f(den)) / kLog2e; }
HS2_DEVI float chunk_factor(float num, float den) { return den == 0.f ? 0.f : num / den; }

// Partial slots: a CTA leaves at most two, that of its first and that of its last unit.
HS2_DEVI int part_slot(const ChunkUnit& u, int per, int cta) {
  const int c0 = u.prefix / per;
  return 2 * cta + (cta == c0 && u.prefix != c0 * per ? 1 : 0);
}

}  // namespace hs2
