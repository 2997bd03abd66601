// chunk_merge.cu — joins the parts of the units that a range border of a chunk-attention kernel cut.
//
// With parts k of a row, each relative to its own reference M_k: M = max M_k, L = sum
// 2^(M_k - M) l_k + 2^(sink - M), o = sum 2^(M_k - M) o_k / L, lse = M + log L, in CTA order.
//
// A kernel of its own: where one sequence is spread over all CTAs a unit has 152 parts, which the
// last CTA to arrive took 45 us to join by itself, and no counters need clearing. Bound by
// latency: a handful of dependent loads, then the parts of all rows at once. 152 cut units of 256
// rows (40 MB of parts) take about 12 us, 152 of 64 rows about 7.
#include "chunk_plan.cuh"

namespace hs2 {

namespace {

constexpr int kMergeWarps = 8;
constexpr int kMergeBlocks = 4;  // per CTA of the attention kernels, and so per cut unit at least; all resident at once

// Rows of a block: a warp has 32 / LPR rows at LPR lanes each, WPR warps share a row's parts.
constexpr int merge_rows_of(int WPR, int LPR) { return kMergeWarps / WPR * (32 / LPR); }
constexpr int kMergeShare = 8;  // warps of a row where blocks abound (4: 19.5 us against 18.9 for a token over 8192 keys)

// Every `step`th group of merge_rows_of() rows of unit u, from group y on.
template <int D, int WPR, int LPR>
HS2_DEVI void merge_rows(const ChunkArgs& a, const ChunkPlan& p, const ChunkUnit& u, int per, int y, int step, float4* sum_, float* sum_l) {
  constexpr int RPW = 32 / LPR, Q = D / (4 * LPR), ROWS = merge_rows_of(WPR, LPR);  // rows of a warp; float4 of a lane
  float4(*sum)[WPR][D / 4] = reinterpret_cast<float4(*)[WPR][D / 4]>(sum_);
  const int live = u.ntok << a.log2G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ln = lane % LPR;
  const int rr = warp / WPR * RPW + lane / LPR, share = warp % WPR;  // row of the group; share of its parts
  const int c = u.prefix / per, parts = (u.prefix + u.ntiles - 1) / per - c + 1;
  for (; y * ROWS < live; y += step) {
    const int n = y * ROWS + rr;
    const bool have = n < live;
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + n;
    float M = -INFINITY, L = 0.f;
    if (have)
      for (int k = ln; k < parts; k += LPR) M = fmaxf(M, __ldcg(ml + (size_t)part_slot(u, per, c + k) * p.tile_rows).x);
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float4 acc[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (have) {
#pragma unroll 2
      for (int k = share; k < parts; k += WPR) {
        const size_t at = (size_t)part_slot(u, per, c + k) * p.tile_rows;
        const float2 x = __ldcg(ml + at);
        const float4* src = reinterpret_cast<const float4*>(p.part_o + (at + n) * D);
        float4 v[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q) v[q] = __ldcg(src + q * LPR + ln);
        const float f = exp2_rel(x.x, M);
        L += f * x.y;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          acc[q].x = fmaf(f, v[q].x, acc[q].x), acc[q].y = fmaf(f, v[q].y, acc[q].y);
          acc[q].z = fmaf(f, v[q].z, acc[q].z), acc[q].w = fmaf(f, v[q].w, acc[q].w);
        }
      }
    }
    if constexpr (WPR > 1) {
#pragma unroll
      for (int q = 0; q < Q; ++q) sum[rr][share][q * LPR + ln] = acc[q];
      if (ln == 0) sum_l[rr * WPR + share] = L;
      __syncthreads();
      if (share == 0) {
#pragma unroll
        for (int i = 1; i < WPR; ++i) {
          L += sum_l[rr * WPR + i];
#pragma unroll
          for (int q = 0; q < Q; ++q) {
            const float4 t = sum[rr][i][q * LPR + ln];
            acc[q].x += t.x, acc[q].y += t.y, acc[q].z += t.z, acc[q].w += t.w;
          }
        }
      }
      __syncthreads();  // the next group's sums
    }
    if (!have || share != 0) continue;
    const int head = (u.g << a.log2G) + (n & (a.G - 1));
    const size_t at = (size_t)(u.row + (n >> a.log2G)) * a.Hq + head;
    const float b2 = sink_b2(a.sink, head);
    const float M2 = fmaxf(M, b2), sc = exp2_rel(M, M2);
    const float den = L * sc + exp2_rel(b2, M2), f = chunk_factor(sc, den);
    if (a.lse && ln == 0) a.lse[at] = chunk_lse(den, M2);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const float4 v = acc[q];
      const size_t col = at * D + 4 * (q * LPR + ln);
      if (a.o_bf16)
        *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.o) + col) = make_uint2(pack_bf16(v.x * f, v.y * f), pack_bf16(v.z * f, v.w * f));
      else
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.o) + col) = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
    }
  }
}

}  // namespace

// grid (kMergeBlocks per CTA of the attention kernels, plans). The cut units share the blocks:
// with many units a block takes many rows of few parts, with few units few rows of many parts.
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32, kMergeBlocks) chunk_merge_kernel(const ChunkArgs a, const ChunkPlan p0,
                                                                                     const ChunkPlan p1) {
  constexpr int LPR = D / 4 < 32 ? D / 4 : 32;
  constexpr int MORE = merge_rows_of(1, LPR), FEW = merge_rows_of(kMergeShare, LPR);
  __shared__ float4 sum[FEW * kMergeShare * D / 4];
  __shared__ float sum_l[FEW * kMergeShare];
  __shared__ int cut_s;
  griddep_launch_dependents();
  griddep_wait();
  const ChunkPlan& p = blockIdx.y ? p1 : p0;
  // the whole list with its length, in one round of loads
  const int per = p.head[1], cuts = p.head[2];
  int mine[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int at = threadIdx.x + k * kMergeWarps * 32;
    mine[k] = at < p.ctas ? p.cuts[at] : 0;
  }
  if (cuts <= 0) return;
  const int blocks = gridDim.x / cuts, i = blockIdx.x / blocks, y = blockIdx.x - i * blocks;
  if (i >= cuts) return;
  if ((int)threadIdx.x == i % (kMergeWarps * 32)) cut_s = mine[i / (kMergeWarps * 32)];
  __syncthreads();
  const ChunkUnit u = load_unit(p, cut_s);
  const int rows = ((u.ntok << a.log2G) + blocks - 1) / blocks;
  if (D <= 128 && rows > MORE) merge_rows<D, 1, D <= 128 ? 8 : LPR>(a, p, u, per, y, blocks, sum, sum_l);  // (wider rows: registers)
  else if (rows > FEW) merge_rows<D, 1, LPR>(a, p, u, per, y, blocks, sum, sum_l);
  else merge_rows<D, kMergeShare, LPR>(a, p, u, per, y, blocks, sum, sum_l);
}

cudaError_t launch_chunk_merge(const ChunkArgs& a, const ChunkPlan* plans, int n_plans, int d, cudaStream_t s) {
  const ChunkPlan &p0 = plans[0], &p1 = plans[n_plans - 1];
  // every plan is cut among as many CTAs; a range of 128-row units is a pair's
  const dim3 grid(kMergeBlocks * p0.ctas * (p0.tile_rows == 128 ? 2 : 1), n_plans);
  auto kern = d == 512 ? chunk_merge_kernel<512> : d == 256 ? chunk_merge_kernel<256> : d == 128 ? chunk_merge_kernel<128>
                                                                                         : chunk_merge_kernel<64>;
  return launch_pdl(kern, grid, dim3(kMergeWarps * 32), 0, s, a, p0, p1);
}

}  // namespace hs2
