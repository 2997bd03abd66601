// chunk_plan.cuh — how the work of a chunk-attention call is cut among the CTAs of its kernels.
//
// The batch's queries form units: a KV head g of a sequence and up to TOK of its tokens, whose
// TOK * G rows (token-major, then the head's query heads) share the head's keys. A unit walks
// the 128-key tiles (two pages) that its rows see. The tiles of all units, one after another,
// are a line of `total` tiles that the CTAs of a persistent kernel share out in equal ranges,
// so lengths and batch sizes do not matter to the balance; a unit cut by a range border leaves
// partial results, which a last kernel merges in CTA order (chunk_merge.cu). Where every unit is
// short against a range (a sliding window), the borders move to the nearest unit's and cut none.
#pragma once
#include "common.cuh"
#include "kernels.h"

namespace hs2 {

struct __align__(16) ChunkUnit {
  int b, g, row, ntok;                // row: packed row of the first token
  int pos0, page0, ntiles, prefix;    // position of the first token; first page; tiles before this unit
  int t, slot_page, npages, pad;      // keys; the sequence's first expanded page; pages of the sequence
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

// A row's results from its denominator, relative to 2^M: 0 where no key is left, NaN passes on.
HS2_DEVI float chunk_lse(float den, float M) { return den == 0.f ? -INFINITY : (M + log2f(den)) / kLog2e; }
HS2_DEVI float chunk_factor(float num, float den) { return den == 0.f ? 0.f : num / den; }

// Partial slots: a CTA leaves at most two, that of its first and that of its last unit.
HS2_DEVI int part_slot(const ChunkUnit& u, int per, int cta) {
  const int c0 = u.prefix / per;
  return 2 * cta + (cta == c0 && u.prefix != c0 * per ? 1 : 0);
}

}  // namespace hs2
