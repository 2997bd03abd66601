// chunk_cc.cu — attention of a ragged batch of query chunks over a float32 cache.
//
// x(s) = scale q . k(s) over the row's visible keys, one pass with the running maximum and
// sum: every key costs a warp one 32-lane dot product. On the CUDA cores, because the tensor
// cores have no fp32 product and a float32 cache is kept for its exactness (1e-4, not 2e-2).
#include "chunk_plan.cuh"
#include "ragged.cuh"

namespace hs2 {

namespace {

constexpr int kCcWarps = 8;
constexpr int kCcKeys = 4;  // keys per warp step: their loads and reductions overlap

// V consecutive floats of a row.
template <int V>
HS2_DEVI void load_row(const void* rows, size_t line, int D, int ch, float (&x)[V]) {
  const float* p = reinterpret_cast<const float*>(rows) + line * D + ch;
#pragma unroll
  for (int i = 0; i < V; i += 2) {
    const float2 v = *reinterpret_cast<const float2*>(p + i);
    x[i] = v.x, x[i + 1] = v.y;
  }
}

}  // namespace

// grid (rows, query heads), 8 warps over the row's keys, merged through shared memory.
template <int D>
__global__ void __launch_bounds__(kCcWarps * 32) chunk_cc_kernel(const ChunkArgs a) {
  constexpr int V = D / 32;
  __shared__ float sm_m[kCcWarps], sm_l[kCcWarps], sm_o[kCcWarps][D];
  griddep_launch_dependents();
  griddep_wait();
  const int r = blockIdx.x, h = blockIdx.y, g = h / a.G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int n1[1];
  warp_rows_at_most<1>(a.row_start, a.batch, r, n1);
  if (r == 0 && h == 0 && warp == 0 && warp_bad_starts(a.row_start, a.batch, a.n_rows) && lane == 0)
    flag_error(a.dev_err, HS2_DEV_BAD_LENGTH);
  const RowPlace pl = row_place(a.row_start, a.seq_len, a.batch, a.max_pages, a.n_rows, r, n1[0]);
  if (pl.b < 0) return;
  if (pl.pos < 0 || a.seq_len[pl.b] > a.max_t || a.row_start[pl.b + 1] - a.row_start[pl.b] > a.max_n) {
    if (threadIdx.x == 0) flag_error(a.dev_err, HS2_DEV_BAD_LENGTH);
    return;
  }
  const int32_t* bt = a.bt + (size_t)pl.b * a.max_pages;
  float q[V];
  load_row<V>(a.q, (size_t)r * a.Hq + h, D, V * lane, q);
  const int lo = a.w > 0 ? max(0, pl.pos - a.w + 1) : 0;
  float m = -INFINITY, l = 0.f, o[V];
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = 0.f;
  for (int s0 = lo + warp * kCcKeys; s0 <= pl.pos; s0 += kCcWarps * kCcKeys) {
    float x[kCcKeys], vv[kCcKeys][V];
#pragma unroll
    for (int j = 0; j < kCcKeys; ++j) {
      x[j] = -INFINITY;
#pragma unroll
      for (int i = 0; i < V; ++i) vv[j][i] = 0.f;
      const int s = s0 + j;
      if (s > pl.pos) continue;
      const int phys = bt[s / kPage];
      if (phys < 0 || phys >= a.num_pages) {
        if (lane == 0) flag_error(a.dev_err, HS2_DEV_BAD_PAGE);
        continue;
      }
      const size_t line = ((size_t)phys * a.Hkv + g) * kPage + s % kPage;
      float k[V], dot = 0.f;
      load_row<V>(a.k, line, D, V * lane, k);
      load_row<V>(a.v, line, D, V * lane, vv[j]);
#pragma unroll
      for (int i = 0; i < V; ++i) dot = fmaf(q[i], k[i], dot);
      x[j] = warp_sum(dot) * a.scale_log2;
    }
    float mn = m;
#pragma unroll
    for (int j = 0; j < kCcKeys; ++j) mn = fmaxf(mn, x[j]);
    const float alpha = exp2_rel(m, mn);
    l *= alpha;
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] *= alpha;
#pragma unroll
    for (int j = 0; j < kCcKeys; ++j) {
      const float p = x[j] != x[j] ? x[j] : exp2_rel(x[j], mn);  // the maximum leaves NaN out
      l += p;
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = fmaf(p, vv[j][i], o[i]);
    }
    m = mn;
  }
  if (lane == 0) sm_m[warp] = m, sm_l[warp] = l;
#pragma unroll
  for (int i = 0; i < V; ++i) sm_o[warp][V * lane + i] = o[i];
  __syncthreads();
  if (threadIdx.x >= D) return;
  const float b2 = sink_b2(a.sink, h);
  float M = b2;
#pragma unroll
  for (int k = 0; k < kCcWarps; ++k) M = fmaxf(M, sm_m[k]);
  float L = exp2_rel(b2, M), O = 0.f;
#pragma unroll
  for (int k = 0; k < kCcWarps; ++k) {
    const float f = exp2_rel(sm_m[k], M);
    L += f * sm_l[k];
    O += f * sm_o[k][threadIdx.x];
  }
  const size_t at = (size_t)r * a.Hq + h;
  const float out = chunk_factor(O, L);
  if (a.o_bf16) reinterpret_cast<__nv_bfloat16*>(a.o)[at * D + threadIdx.x] = __float2bfloat16(out);
  else reinterpret_cast<float*>(a.o)[at * D + threadIdx.x] = out;
  if (a.lse && threadIdx.x == 0) a.lse[at] = chunk_lse(L, M);
}

cudaError_t launch_chunk_cc(const ChunkArgs& a, int d, cudaStream_t s) {
  const dim3 grid(a.n_rows, a.Hq);
  return launch_pdl(d == 128 ? chunk_cc_kernel<128> : chunk_cc_kernel<64>, grid, dim3(kCcWarps * 32), 0, s, a);
}

}  // namespace hs2
