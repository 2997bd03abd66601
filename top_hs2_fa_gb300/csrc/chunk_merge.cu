// chunk_merge.cu — joins the parts of the units that a range border of a chunk-attention kernel cut.
//
// With parts k of a row, each relative to its own reference M_k: M = max M_k, L = sum
// 2^(M_k - M) l_k + 2^(sink - M), o = sum 2^(M_k - M) o_k / L, lse = M + log L, in CTA order.
//
// A kernel of its own: where one sequence is spread over all CTAs a unit has 152 parts, which the
// last CTA to arrive took 45 us to join by itself, and no counters need clearing. Bound by
// latency: a handful of dependent loads, then the parts of all rows at once.
#include "chunk_plan.cuh"

namespace hs2 {

namespace {

constexpr int kMergeWarps = 8;
constexpr int kMergeParts = 256;  // CTAs of a unit at most (the host launches no more)

template <int LPR>
HS2_DEVI float lanes_max(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <int LPR>
HS2_DEVI float lanes_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Rows of a block: a warp has 32 / LPR rows at LPR lanes each, WPR warps share a row's parts.
constexpr int merge_rows_of(int WPR, int LPR) { return kMergeWarps / WPR * (32 / LPR); }

// Block c has the unit that starts in CTA c's range and ends behind it.
template <int D, int WPR, int LPR>
HS2_DEVI void merge_rows(const ChunkArgs& a, const ChunkPlan& p, float (*fac)[kMergeParts], float4* sum_) {
  constexpr int RPW = 32 / LPR, Q = D / (4 * LPR);  // rows of a warp; float4 of a lane
  float4(*sum)[WPR][D / 4] = reinterpret_cast<float4(*)[WPR][D / 4]>(sum_);
  const int c = blockIdx.x;
  const int total = p.head[0], per = p.head[1], next = c + 1 < p.ctas ? p.cta_first[c + 1] : 0;
  if (c + 1 >= p.ctas || (long long)(c + 1) * per >= total) return;
  const ChunkUnit u = load_unit(p, next);
  if (u.prefix / per != c) return;  // whole, or cut at an earlier border
  const int live = u.ntok << a.log2G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ln = lane % LPR;
  const int rr = warp / WPR * RPW + lane / LPR, part = warp % WPR;  // row of the block; share of its parts
  const int n = blockIdx.y * merge_rows_of(WPR, LPR) + rr;
  if ((int)blockIdx.y * merge_rows_of(WPR, LPR) >= live) return;
  const int parts = (u.prefix + u.ntiles - 1) / per - c + 1;
  const bool have = n < live;
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + n;
  float M = -INFINITY, L = 0.f;
  if (have)
    for (int k = ln; k < parts; k += LPR) M = fmaxf(M, __ldcg(ml + (size_t)part_slot(u, per, c + k) * p.tile_rows).x);
  M = lanes_max<LPR>(M);
  if (have)
    for (int k = ln; k < parts; k += LPR) {
      const float2 y = __ldcg(ml + (size_t)part_slot(u, per, c + k) * p.tile_rows);
      const float e = exp2_rel(y.x, M);
      L += e * y.y;
      if (part == 0) fac[rr][k] = e;
    }
  L = lanes_sum<LPR>(L);
  __syncthreads();
  float4 acc[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (have) {
#pragma unroll 4
    for (int k = part; k < parts; k += WPR) {
      const float4* src = reinterpret_cast<const float4*>(p.part_o + ((size_t)part_slot(u, per, c + k) * p.tile_rows + n) * D);
      const float f = fac[rr][k];
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const float4 v = __ldcg(src + q * LPR + ln);
        acc[q].x = fmaf(f, v.x, acc[q].x), acc[q].y = fmaf(f, v.y, acc[q].y);
        acc[q].z = fmaf(f, v.z, acc[q].z), acc[q].w = fmaf(f, v.w, acc[q].w);
      }
    }
  }
  if (WPR > 1) {
#pragma unroll
    for (int q = 0; q < Q; ++q) sum[rr][part][q * LPR + ln] = acc[q];
    __syncthreads();
  }
  if (!have || part != 0) return;
  const int head = (u.g << a.log2G) + (n & (a.G - 1));
  const size_t at = (size_t)(u.row + (n >> a.log2G)) * a.Hq + head;
  const float b2 = sink_b2(a.sink, head);
  const float M2 = fmaxf(M, b2), sc = exp2_rel(M, M2);
  const float den = L * sc + exp2_rel(b2, M2), f = den > 0.f ? sc / den : 0.f;
  if (a.lse && ln == 0) a.lse[at] = den > 0.f ? (M2 + log2f(den)) / kLog2e : -INFINITY;
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    float4 v = acc[q];
    if (WPR > 1)
#pragma unroll
      for (int i = 1; i < WPR; ++i) {
        const float4 t = sum[rr][i][q * LPR + ln];
        v.x += t.x, v.y += t.y, v.z += t.z, v.w += t.w;
      }
    const size_t col = at * D + 4 * (q * LPR + ln);
    if (a.o_bf16)
      *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.o) + col) = make_uint2(pack_bf16(v.x * f, v.y * f), pack_bf16(v.z * f, v.w * f));
    else
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.o) + col) = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
  }
}

constexpr int kWideLanes = 8;  // the wide kernel's units: 256 rows, few parts
constexpr int kNarrowWarps = 4;  // the narrow one's: up to 64 rows, many parts

}  // namespace

// grid (CTAs of the attention kernels, groups of a unit's rows, plans)
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) chunk_merge_kernel(const ChunkArgs a, const ChunkPlan p0, const ChunkPlan p1) {
  constexpr int LPR = D / 4 < 32 ? D / 4 : 32;
  __shared__ float fac[merge_rows_of(1, kWideLanes)][kMergeParts];
  __shared__ float4 sum[merge_rows_of(kNarrowWarps, LPR) * kNarrowWarps * D / 4];
  griddep_launch_dependents();
  griddep_wait();
  const ChunkPlan& p = blockIdx.z ? p1 : p0;
  if (p.tile_rows > 64) merge_rows<D, 1, kWideLanes>(a, p, fac, sum);
  else merge_rows<D, kNarrowWarps, LPR>(a, p, fac, sum);
}

cudaError_t launch_chunk_merge(const ChunkArgs& a, const ChunkPlan* plans, int n_plans, int d, cudaStream_t s) {
  const ChunkPlan &p0 = plans[0], &p1 = plans[n_plans - 1];
  if (p0.ctas > kMergeParts || p1.ctas != p0.ctas) return cudaErrorInvalidValue;
  int groups = 0;
  for (int i = 0; i < n_plans; ++i) {
    const int rows = plans[i].tile_rows > 64 ? merge_rows_of(1, kWideLanes) : merge_rows_of(kNarrowWarps, d == 128 ? 32 : 16);
    groups = groups > plans[i].tile_rows / rows ? groups : plans[i].tile_rows / rows;
  }
  const dim3 grid(p0.ctas, groups, n_plans);
  return launch_pdl(d == 128 ? chunk_merge_kernel<128> : chunk_merge_kernel<64>, grid, dim3(kMergeWarps * 32), 0, s, a, p0, p1);
}

}  // namespace hs2
