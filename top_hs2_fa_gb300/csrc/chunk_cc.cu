// chunk_cc.cu — attention of a ragged batch of query chunks on the CUDA cores.
//
// x(s) = scale q . k(s) over the row's visible keys, one pass with the running maximum and
// sum: every key costs a warp one 32-lane dot product.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "ragged.cuh"

namespace hs2 {

namespace {

constexpr int kCcWarps = 8;
constexpr int kCcKeys = 4;  // keys per warp step: their loads and reductions overlap

// V consecutive channels of a pool row as floats.
template <int FMT, int V>
HS2_DEVI void load_row(const uint8_t* pool, const float* scale, const uint8_t* sf, size_t line, int D, int ch,
                       float (&x)[V]) {
  if constexpr (FMT == HS2_F32) {
    const float* p = reinterpret_cast<const float*>(pool) + line * D + ch;
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 v = *reinterpret_cast<const float2*>(p + i);
      x[i] = v.x, x[i + 1] = v.y;
    }
  } else if constexpr (FMT == HS2_BF16) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(pool) + (line * D + ch) / 2;
#pragma unroll
    for (int i = 0; i < V; i += 2) x[i] = bf16_lo(p[i / 2]), x[i + 1] = bf16_hi(p[i / 2]);
  } else {
    const float S = scale[line / kPage];
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      uint32_t h;
      if constexpr (FMT == HS2_FP8_E4M3) {
        h = fp8x2_to_f16x2(*reinterpret_cast<const uint16_t*>(pool + line * D + ch + i));
      } else {
        uint32_t u1, u2, u3;
        fp4x8_to_f16x8(pool[(line * D + ch + i) / 2], h, u1, u2, u3);
        const uint32_t s = sf[(line * D + ch) / 16];
        h = hmul2(h, e4m3_pair(s, s));
      }
      const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h));
      x[i] = f.x * S, x[i + 1] = f.y * S;
    }
  }
}

}  // namespace

// grid (rows, query heads), 8 warps over the row's keys, merged through shared memory.
template <int D, int FMT>
__global__ void __launch_bounds__(kCcWarps * 32) chunk_cc_kernel(const ChunkArgs a) {
  constexpr int V = D / 32;
  __shared__ float sm_m[kCcWarps], sm_l[kCcWarps], sm_o[kCcWarps][D];
  const int r = blockIdx.x, h = blockIdx.y, g = h / a.G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int n1[1];
  warp_rows_at_most<1>(a.row_start, a.batch, r, n1);
  const RowPlace pl = row_place(a.row_start, a.seq_len, a.batch, a.max_pages, r, n1[0]);
  if (pl.b < 0) return;
  const int end = a.row_start[pl.b + 1];
  if (pl.pos < 0 || a.seq_len[pl.b] > a.max_t || end - a.row_start[pl.b] > a.max_n || end > a.n_rows) {
    if (threadIdx.x == 0) flag_error(a.dev_err, HS2_DEV_BAD_LENGTH);
    return;
  }
  const int32_t* bt = a.bt + (size_t)pl.b * a.max_pages;
  float q[V];
  load_row<FMT == HS2_F32 ? HS2_F32 : HS2_BF16, V>(reinterpret_cast<const uint8_t*>(a.q), nullptr, nullptr,
                                                   (size_t)r * a.Hq + h, D, V * lane, q);
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
      load_row<FMT, V>(reinterpret_cast<const uint8_t*>(a.k), a.k_scale, a.k_sf, line, D, V * lane, k);
      load_row<FMT, V>(reinterpret_cast<const uint8_t*>(a.v), a.v_scale, a.v_sf, line, D, V * lane, vv[j]);
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
      const float p = exp2_rel(x[j], mn);
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
  const float out = L > 0.f ? O / L : 0.f;
  if (a.o_bf16) reinterpret_cast<__nv_bfloat16*>(a.o)[at * D + threadIdx.x] = __float2bfloat16(out);
  else reinterpret_cast<float*>(a.o)[at * D + threadIdx.x] = out;
  if (a.lse && threadIdx.x == 0) a.lse[at] = L > 0.f ? (M + log2f(L)) / kLog2e : -INFINITY;
}

template <int D>
static cudaError_t launch_cc(const ChunkArgs& a, int dtype, cudaStream_t s) {
  const dim3 grid(a.n_rows, a.Hq);
  switch (dtype) {
    case HS2_F32: chunk_cc_kernel<D, HS2_F32><<<grid, kCcWarps * 32, 0, s>>>(a); break;
    case HS2_BF16: chunk_cc_kernel<D, HS2_BF16><<<grid, kCcWarps * 32, 0, s>>>(a); break;
    case HS2_FP8_E4M3: chunk_cc_kernel<D, HS2_FP8_E4M3><<<grid, kCcWarps * 32, 0, s>>>(a); break;
    case HS2_FP4_E2M1: chunk_cc_kernel<D, HS2_FP4_E2M1><<<grid, kCcWarps * 32, 0, s>>>(a); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

cudaError_t launch_chunk_cc(const ChunkArgs& a, int d, int dtype, cudaStream_t s) {
  return d == 128 ? launch_cc<128>(a, dtype, s) : launch_cc<64>(a, dtype, s);
}

}  // namespace hs2
