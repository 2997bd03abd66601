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
// nearly as even, and calls with few keys or few rows have no planning kernel (plan_ordered, plan_own,
// plan_line below).
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
  int first_unit, begin, end, per;  // per: tiles of a range
};

HS2_DEVI ChunkRange chunk_range(const ChunkPlan& p, int cta) {
  ChunkRange r;
  const int total = p.head[0], first = p.cta_first[cta], begin = p.cta_begin[cta];  // one round of loads
  const int next = p.cta_begin[min(cta + 1, p.ctas - 1)];
  r.per = p.head[1];
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

// What a call without a planning kernel knows of a sequence; checked and flagged as the planning kernel does
// (descends: of any row_start, then no sequence has rows).
struct OwnSeq {
  int row, n, t, key;  // n = 0: no rows, or none that are computed
};
HS2_DEVI OwnSeq own_load(const ChunkArgs& a, int b, bool& descends) {
  OwnSeq x{};
  if (b < a.batch) {
    x.row = a.row_start[b];
    const int r1 = a.row_start[b + 1];
    descends |= r1 < x.row;
    if (a.key_start) {
      x.key = a.key_start[b];
      const int k1 = a.key_start[b + 1];
      x.t = x.key >= 0 && k1 >= x.key && k1 <= a.n_keys ? k1 - x.key : -1;
    } else {
      x.t = a.seq_len[b];
    }
    x.n = r1 - x.row;
  }
  return x;
}
HS2_DEVI void own_check(const ChunkArgs& a, OwnSeq& x, bool descends, bool flag) {
  if (descends || (x.n != 0 && (x.row < 0 || x.n > a.max_n || x.t < x.n || x.t > a.max_t || x.row > a.n_rows - x.n))) {
    x.n = 0;
    if (flag) flag_error(a.dev_err, HS2_DEV_BAD_LENGTH);
  }
}

// Calls of up to 32 sequences whose units are few and stay whole need no planning kernel: unit i of the batch is
// CTA i % ctas's, and a warp of it writes the records of its units, at most kOwnUnits, one after another on
// a line of their own. Returns the line's length.
constexpr int kOwnUnits = kOwnPlanUnits;
static_assert(kOwnPlanSeqs == 32, "a lane a sequence");
HS2_DEVI int plan_own(const ChunkArgs& a, const ChunkPlan& p, int cta, ChunkUnit* own) {
  const int lane = threadIdx.x & 31, tok = p.tile_rows / a.G;
  bool descends = false;
  OwnSeq q = own_load(a, lane, descends);
  own_check(a, q, __any_sync(0xffffffffu, descends), cta == 0);
  const int n = q.n, t = q.t, r0 = q.row, k0 = q.key;
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

// Calls of up to 32 K sequences of a unit each: the line of tiles in equal ranges, as the planning kernel cuts it,
// found by a warp of every CTA. `own` gets all units; `publish`: the plan in memory too, for the merge.
template <int K>  // sequences of a lane, one after another
HS2_DEVI ChunkRange plan_line(const ChunkArgs& a, const ChunkPlan& p, int cta, ChunkUnit* own, bool publish) {
  const int lane = threadIdx.x & 31;
  OwnSeq q[K];
  bool descends = false;
#pragma unroll
  for (int i = 0; i < K; ++i) q[i] = own_load(a, K * lane + i, descends);
  descends = __any_sync(0xffffffffu, descends);
  int tiles = 0, units = 0;  // of the lane, then of it and those before
#pragma unroll
  for (int i = 0; i < K; ++i) {
    own_check(a, q[i], descends, publish);
    if (q[i].n > 0) tiles += (q[i].t - 1) / (2 * kPage) + 1, ++units;
  }
  int prefix = -tiles, at = -units;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, tiles, s), w = __shfl_up_sync(0xffffffffu, units, s);
    if (lane >= s) tiles += v, units += w;
  }
  prefix += tiles, at += units;
  const int total = __shfl_sync(0xffffffffu, tiles, 31), per = max(1, (total + p.ctas - 1) / p.ctas);
  ChunkRange r;
  r.begin = min(total, cta * per);
  r.end = min(total, r.begin + per);
  r.per = per;
  int before = 0, cuts = 0;  // units that end before the range; cut ones
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const bool have = q[i].n > 0;
    ChunkUnit x{};
    x.b = K * lane + i;
    x.row = q[i].row;
    x.ntok = q[i].n;
    x.pos0 = q[i].t - q[i].n;
    x.ntiles = have ? (q[i].t - 1) / (2 * kPage) + 1 : 0;
    x.prefix = prefix;
    x.t = q[i].t;
    x.npages = (q[i].t + kPage - 1) / kPage;
    prefix += x.ntiles;
    if (have) own[at] = x;
    before += have && prefix <= r.begin;
    if (publish) {
      const bool cut = have && x.prefix / per != (prefix - 1) / per;
      const uint32_t m = __ballot_sync(0xffffffffu, cut);
      if (have) {
        int4* d = reinterpret_cast<int4*>(p.units) + 3 * at;
        const int4* s = reinterpret_cast<const int4*>(&x);
        d[0] = s[0], d[1] = s[1], d[2] = s[2];
      }
      if (cut) p.cuts[cuts + __popc(m & ((1u << lane) - 1))] = at;
      cuts += __popc(m);
    }
    at += have;
  }
  r.first_unit = __reduce_add_sync(0xffffffffu, before);
  if (publish && lane == 0) p.head[0] = total, p.head[1] = per, p.head[2] = cuts;
  return r;
}

// What a CTA walks: units of its own in `own` (listed), or a range of the line. own_range: shared memory.
// LINE: 0, or p.own may be 2 in calls of up to so many sequences, and `own` has room for as many units.
template <int LINE>
HS2_DEVI ChunkRange plan_range(const ChunkArgs& a, const ChunkPlan& p, int cta, ChunkUnit* own, ChunkRange* own_range, bool& listed) {
  const int ordered = p.own || !p.order ? 0 : p.head[3];
  listed = p.own || ordered;
  if (!listed) return chunk_range(p, cta);
  if (threadIdx.x < 32) {
    ChunkRange r{0, 0, 0, 1};
    bool line = false;
    if constexpr (LINE > 32) {  // (a batch of up to 32 with 4 a lane: 1.5 us longer)
      line = p.own == 2 && a.batch > 32;
      if (line) r = plan_line<LINE / 32>(a, p, cta, own, blockIdx.x == 0);
    }
    if constexpr (LINE > 0) {
      if (p.own == 2 && !line) r = plan_line<1>(a, p, cta, own, blockIdx.x == 0), line = true;
    }
    if (!line) r.end = p.own ? plan_own(a, p, cta, own) : plan_ordered(p, ordered, cta, own);
    if (threadIdx.x == 0) *own_range = r;
  }
  __syncthreads();
  return *own_range;
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
