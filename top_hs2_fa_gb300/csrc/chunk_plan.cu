// chunk_plan.cu — the planning kernel of a chunk-attention call, and the expansion of FP8 / FP4
// pages to bf16 for the wide kernel.
#include <cuda_fp16.h>

#include "block_scan.cuh"
#include "chunk_plan.cuh"

namespace hs2 {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kLengths = kPlanThreads;  // of whole units: tiles below this

// The first key a token at position p sees.
HS2_DEVI int first_key(int p, int w) { return w > 0 ? max(0, p - w + 1) : 0; }

}  // namespace

// Bound by latency: three rounds of loads and as many prefix sums, about 5 us for a batch of up to
// 1024 sequences and units. One block per plan. Sequences in chunks of 1024: a prefix sum of their units; then a thread
// per unit writes its record and a prefix sum over the units' tiles places it on the line.
__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const ChunkArgs a, const ChunkPlan p0,
                                                                  const ChunkPlan p1) {
  griddep_launch_dependents();  // the attention kernel may set itself up meanwhile
  griddep_wait();
  const ChunkPlan& p = blockIdx.x ? p1 : p0;
  __shared__ int sums[33], ubase[kPlanThreads + 1], s_row[kPlanThreads], s_n[kPlanThreads], s_t[kPlanThreads],
      s_exp[kPlanThreads], n_cuts, longest;
  const int tok = p.tile_rows / a.G;
  int total_tiles = 0, units = 0, exp_pages = 0, n_exp = 0;
  int my_tiles = 0, my_prefix = 0;  // of the last unit this thread wrote
  if (threadIdx.x == 0) n_cuts = longest = 0;
  // rows of two sequences at once would overrun what the host sized for n_rows rows
  bool descends = false;
  int n = 0, t = 0, r0 = 0, k0 = 0;  // this thread's sequence of the chunk
  auto load = [&](int b) {
    n = t = r0 = k0 = 0;
    if (b >= a.batch) return;
    r0 = a.row_start[b];
    if (a.key_start) {  // packed keys; bad starts have no t that a row could have
      k0 = a.key_start[b];
      const int k1 = a.key_start[b + 1];
      t = k0 >= 0 && k1 >= k0 && k1 <= a.n_keys ? k1 - k0 : -1;
    } else {
      t = a.seq_len[b];
    }
    const int r1 = a.row_start[b + 1];
    descends |= r1 < r0;
    n = r1 - r0;
  };
  for (int b0 = 0; b0 < a.batch; b0 += kPlanThreads) load(b0 + threadIdx.x);
  if (__syncthreads_or(descends)) {
    for (int c = threadIdx.x; c < p.ctas; c += kPlanThreads) p.cta_begin[c] = 0;
    if (threadIdx.x == 0) {
      flag_error(a.dev_err, HS2_DEV_BAD_LENGTH);
      p.head[0] = p.head[2] = p.head[3] = 0;
      p.head[1] = 1;
      if (p.expand) p.exp_head[0] = 0;
    }
    return;
  }
  for (int b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    if (a.batch > kPlanThreads) load(b);
    if (b < a.batch) {
      if (n != 0 && (r0 < 0 || n > a.max_n || t < n || t > a.max_t || r0 > a.n_rows - n)) {
        if (blockIdx.x == 0) flag_error(a.dev_err, HS2_DEV_BAD_LENGTH);
        n = 0;
      }
    }
    const long long rows = (long long)n * a.G;
    if (rows <= p.min_rows || rows > p.max_rows) n = 0;
    const int per_head = (n + tok - 1) / tok;
    int here, pages = 0, pg = 0;
    const int ub = block_prefix(per_head * a.Hkv, sums, here);
    ubase[threadIdx.x] = ub;
    if (threadIdx.x == 0) ubase[kPlanThreads] = here;
    s_row[threadIdx.x] = r0;
    s_n[threadIdx.x] = n;
    s_t[threadIdx.x] = t;
    if (p.expand) {
      const int e0 = n > 0 ? first_key(t - n, a.w) / kPage : 0;
      const int np = n > 0 ? (t + kPage - 1) / kPage - e0 : 0;
      pg = exp_pages + block_prefix(np, sums, pages);
      exp_pages += pages;
      int seqs;
      const int at = n_exp + block_prefix(n > 0, sums, seqs);
      n_exp += seqs;
      if (n > 0) {
        p.exp_seq[at] = b;
        p.exp_base[at] = pg;
        p.exp_page[at] = e0;
      }
      s_exp[threadIdx.x] = pg - e0;  // expanded page of the sequence's page 0
    }
    if (a.key_start) s_exp[threadIdx.x] = k0;
    __syncthreads();
    for (int u0 = 0; u0 < here; u0 += kPlanThreads) {
      const int u = u0 + threadIdx.x;
      int cost = 0;
      ChunkUnit x{};
      if (u < here) {
        int lo = 0, hi = kPlanThreads;  // the last sequence with ubase <= u
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (ubase[mid] <= u) lo = mid;
          else hi = mid;
        }
        const int sn = s_n[lo], st = s_t[lo], ph = (sn + tok - 1) / tok;
        const int k = u - ubase[lo], tile = k % ph;
        x.b = b0 + lo;
        x.g = k / ph;
        x.row = s_row[lo] + tile * tok;
        x.ntok = min(tok, sn - tile * tok);
        x.pos0 = st - sn + tile * tok;
        x.page0 = first_key(x.pos0, a.w) / kPage;
        const int last = (x.pos0 + x.ntok - 1) / kPage;
        x.ntiles = (last - x.page0) / 2 + 1;
        x.t = st;
        x.slot_page = p.expand || a.key_start ? s_exp[lo] : 0;
        x.npages = (st + kPage - 1) / kPage;
        cost = x.ntiles;
      }
      int tiles;
      const int top = __reduce_max_sync(0xffffffffu, cost);
      if ((threadIdx.x & 31) == 0 && top > 0) atomicMax(&longest, top);
      x.prefix = total_tiles + block_prefix(cost, sums, tiles);
      total_tiles += tiles;
      my_tiles = cost, my_prefix = x.prefix;
      if (u < here) {  // within max_units: the valid sequences' rows are disjoint and within n_rows
        int4* d = reinterpret_cast<int4*>(p.units) + 3 * (size_t)(units + u);
        const int4* s = reinterpret_cast<const int4*>(&x);
        d[0] = s[0], d[1] = s[1], d[2] = s[2];
      }
    }
    units += here;
    __syncthreads();  // the chunk's arrays are rewritten
  }
  // down to a tile per CTA: ranges of at least 2 (narrow) and 4 (wide) cost more than their merge
  // saves (4 sequences of up to 1500 keys 19.1 us against 16.2, 64 tokens over 2048 keys 25.3, 22.3)
  const int per = max(1, (total_tiles + p.ctas - 1) / p.ctas);
  __syncthreads();  // the records are visible to the block
  // Whole units by falling length, the CTAs taking them in turn there and back, where the longest of the CTAs'
  // sums is at most `whole`: cuts cost a CTA two parts, another start and the merge, cut_tiles tiles or more,
  // and units that share keys run at the same time. Whole and cut, us on the device, with that longest sum and
  // the range, in tiles: absorbed, 8 sequences of 100 tokens of 32 heads over 2000 keys (26, 25) 92 and 102,
  // but 60 of 2 tokens of 64 heads (16, 10) 71 and 63; expanded, 16 of 400 of 32 heads over 6000 (216, 204) 400
  // and 454, 6 of 500 of 16 over 2000 (20, 14) 49 and 58, but one of 1000 over 2000 (16, 6) 38 and 33. The sort
  // takes 1 to 2 us.
  const int whole = per + per / 8 + p.cut_tiles;
  if (p.order && units > 0 && units <= kOwnUnits * p.ctas && longest <= whole && longest < kLengths) {
    __shared__ int place_of[kLengths], span;
    auto tiles_of = [&](int u) {
      return a.batch <= kPlanThreads && units <= kPlanThreads ? my_tiles : p.units[12 * (size_t)u + 6];
    };
    place_of[threadIdx.x] = 0;
    if (threadIdx.x == 0) span = 0;
    __syncthreads();
    for (int u = threadIdx.x; u < units; u += kPlanThreads) atomicAdd(&place_of[kLengths - 1 - tiles_of(u)], 1);
    __syncthreads();
    int all;
    place_of[threadIdx.x] = block_prefix(place_of[threadIdx.x], sums, all);  // of units longer than this
    __syncthreads();
    for (int u = threadIdx.x; u < units; u += kPlanThreads) {
      const int k = tiles_of(u);
      p.order[atomicAdd(&place_of[kLengths - 1 - k], 1)] = make_int2(u, k);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.ctas; c += kPlanThreads) {
      int sum = 0;
      for (int i = 0; i < kOwnUnits; ++i) {
        const int k = ordered_unit(i, c, p.ctas);
        if (k < units) sum += p.order[k].y;
      }
      atomicMax(&span, sum);
    }
    __syncthreads();
    if (span <= whole) {
      if (threadIdx.x == 0) {
        p.head[0] = total_tiles;
        p.head[1] = per;
        p.head[2] = 0;
        p.head[3] = units;
      }
      return;
    }
  }
  const bool snap = (long long)p.snap * longest <= per;
  // each CTA's range start and the unit there, and the list of units that a range border cuts (in
  // any order: the merge treats each by itself)
  auto place = [&](int u, int ntiles, int prefix) {
    for (int c = (prefix + per - 1) / per; c < p.ctas && (long long)c * per < prefix + ntiles; ++c) {
      const bool next = snap && 2 * (c * per - prefix) > ntiles;
      p.cta_first[c] = u + next;
      p.cta_begin[c] = next ? prefix + ntiles : snap ? prefix : c * per;
    }
    if (!snap && prefix / per != (prefix + ntiles - 1) / per) p.cuts[atomicAdd(&n_cuts, 1)] = u;
  };
  for (int c = threadIdx.x; c < p.ctas; c += kPlanThreads)
    if ((long long)c * per >= total_tiles) p.cta_begin[c] = total_tiles;
  if (a.batch <= kPlanThreads && units <= kPlanThreads) {  // they are in registers
    if ((int)threadIdx.x < units) place(threadIdx.x, my_tiles, my_prefix);
  } else {
    for (int u = threadIdx.x; u < units; u += kPlanThreads) {
      const int4 y = reinterpret_cast<const int4*>(p.units)[3 * (size_t)u + 1];
      place(u, y.z, y.w);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    p.head[0] = total_tiles;
    p.head[1] = per;
    p.head[2] = n_cuts;
    p.head[3] = 0;
    if (p.expand) p.exp_head[0] = n_exp;
  }
}

cudaError_t launch_chunk_plan(const ChunkArgs& a, const ChunkPlan* plans, int n_plans, cudaStream_t s) {
  return launch_pdl(chunk_plan_kernel, dim3(n_plans), dim3(kPlanThreads), 0, s, a, plans[0], plans[n_plans - 1]);
}

// ---------------------------------------------------------------------------- expansion
// The pages of the wide kernel's sequences as bf16: code * group scale has at most 6 significant
// bits, and the slab scale's sign and power of two are exponents, so the bf16 value is exact;
// the rest of the slab scale, a factor in [1, 2), goes to `params` ([page][Hkv]: K's factor, -1
// for a page that is not there, and log2 of V's) and into the softmax. Rows behind the
// sequence are zeros, so that weight 0 times them stays 0.
// Bound by the bytes written: 32768 FP4 keys of 4 heads (86 MB) take 18 us from a cold cache.
// grid (pages of a sequence, KV heads, sequences), 256 threads: 8 (FP4: 16) channels each.
template <int D, int FMT>
__global__ void __launch_bounds__(256) chunk_expand_kernel(const ChunkArgs a, const ChunkPlan p, uint4* ek, uint4* ev,
                                                           float2* params) {
  griddep_launch_dependents();
  griddep_wait();
  const int g = blockIdx.y, n = p.exp_head[0];
  for (int i = blockIdx.z; i < n; i += gridDim.z) {
    const int b = p.exp_seq[i], page = p.exp_page[i] + blockIdx.x, t = a.seq_len[b];
    if (page >= (t + kPage - 1) / kPage) continue;
    const int slot = p.exp_base[i] + blockIdx.x;
    if (slot >= p.max_exp_pages) continue;  // never: the host sized the buffer for every sequence
    const int phys = a.bt[(size_t)b * a.max_pages + page];
    const bool there = phys >= 0 && phys < a.num_pages;
    if (!there && threadIdx.x == 0) flag_error(a.dev_err, HS2_DEV_BAD_PAGE);
    const size_t line0 = ((size_t)(there ? phys : 0) * a.Hkv + g) * kPage;
    const size_t out0 = ((size_t)slot * a.Hkv + g) * kPage;
    float f[2], e[2];  // a slab scale S = f * 2^e-with-sign
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const float S = there ? (side ? a.v_scale : a.k_scale)[line0 / kPage] : 0.f;
      const uint32_t u = __float_as_uint(S);
      const bool plain = (u & 0x7F800000u) != 0 && (u & 0x7F800000u) != 0x7F800000u;
      f[side] = plain ? __uint_as_float((u & 0x007FFFFFu) | 0x3F800000u) : 1.f;
      e[side] = plain ? __uint_as_float(u & 0xFF800000u) : S;  // subnormal, zero, inf, NaN: as it is
    }
    if (threadIdx.x == 0) params[(size_t)slot * a.Hkv + g] = make_float2(there ? f[0] : -1.f, log2f(f[1]));
    constexpr int UNITS = kPage * D / 8;  // 16-byte outputs per side
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const uint8_t* pool = reinterpret_cast<const uint8_t*>(side ? a.v : a.k);
      const uint8_t* sf = side ? a.v_sf : a.k_sf;
      uint4* out = (side ? ev : ek) + out0 * (D / 8);
      for (int x = threadIdx.x; x < UNITS; x += 256) {
        const int row = x / (D / 8), u8 = x % (D / 8);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (there && page * kPage + row < t) {
          uint32_t h[4];
          if constexpr (FMT == HS2_FP4_E2M1) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(pool + (line0 + row) * (D / 2) + 4 * u8);
            fp4x8_to_f16x8(w, h[0], h[1], h[2], h[3]);
            const uint32_t s = sf[(line0 + row) * (D / 16) + u8 / 2], s2 = e4m3_pair(s, s);
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = hmul2(h[j], s2);
          } else {
            const uint2 w = *reinterpret_cast<const uint2*>(pool + (line0 + row) * D + 8 * u8);
            fp8x4_to_f16x4(w.x, h[0], h[1]);
            fp8x4_to_f16x4(w.y, h[2], h[3]);
          }
          uint32_t r[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 q = __half22float2(*reinterpret_cast<__half2*>(&h[j]));
            r[j] = pack_bf16(q.x * e[side], q.y * e[side]);
          }
          v = make_uint4(r[0], r[1], r[2], r[3]);
        }
        out[x] = v;
      }
    }
  }
}

cudaError_t launch_chunk_expand(const ChunkArgs& a, const ChunkPlan& p, int d, int dtype, void* ek, void* ev,
                                float2* params, int max_seqs, int max_pages_seq, cudaStream_t s) {
  auto kern = d == 128 ? (dtype == HS2_FP4_E2M1 ? chunk_expand_kernel<128, HS2_FP4_E2M1>
                                                : chunk_expand_kernel<128, HS2_FP8_E4M3>)
                       : (dtype == HS2_FP4_E2M1 ? chunk_expand_kernel<64, HS2_FP4_E2M1>
                                                : chunk_expand_kernel<64, HS2_FP8_E4M3>);
  return launch_pdl(kern, dim3(max_pages_seq, a.Hkv, max_seqs < 65535 ? max_seqs : 65535), dim3(256), 0, s, a, p, (uint4*)ek, (uint4*)ev, params);
}

}  // namespace hs2
