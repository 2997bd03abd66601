// kv_rows.cu — rows of a ragged batch into a paged cache (quantised on the way) and back.
//
// At prefill each Cross group's cache gains the prompt's bridged K/V rows, at decode one row
// per sequence ("HySparse2：整体架构、KV 生命周期与 PD 分离", §8, §10.1); an FP4 cache keeps E2M1
// codes with one E4M3 scale per 16 channels ("2.3.1 · CSA、HCA 与 CSA2", §3, "KV 字节与 FP4").
//
// The arithmetic of FP4 and FP8 rows is in kv_rows.cuh.
//
// 32768 rows of 2 x 4 x 128 bf16 values to FP4 (86 MB) take 26 us with slab scales of many bits and
// 39 with a power of two, where nearly every group meets a border (comparing every value against the
// borders took 46). With many bits the wait for the rows bounds it (64 registers leave half of the
// warps; ALU 47 % busy, HBM 0.54 of the copy rate over 393216 rows), with a power of two the integer
// pipe (68 %). Their way back to floats (153 MB) takes 29 us.
#include "kv_rows.cuh"

namespace hs2 {

namespace {

// One thread per (row, KV head, 16 channels) of K or V, or of both (SIDES 2); a warp takes 32 / (D / 16) consecutive
// rows of one head, so its codes and group scales fall next to each other in the page.
template <int D, int FMT, bool ROW_F32, int SIDES>
__global__ void __launch_bounds__(kRowThreads) kv_write_kernel(const RowsArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int GPR = D / 16, TOK = 32 / GPR;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r0 = ((blockIdx.x - 1) * (kRowThreads / 32) + warp) * TOK;
  const int tok = lane / GPR, grp = lane % GPR, r = r0 + tok;
  const int g = blockIdx.y, side = SIDES == 1 ? blockIdx.z : 0;
  if (blockIdx.x == 0) {
    check_starts(a);
    return;
  }
  if (r0 >= a.n_rows) return;
  const bool have = r < a.n_rows;
  float x[16], y[16];
  const long long at = (long long)r * a.row_stride + g * D + 16 * grp;
  if (have) load16<ROW_F32>(side ? a.v_rows : a.k_rows, at, x);
  if (SIDES == 2 && have) load16<ROW_F32>(a.v_rows, at, y);
  int n[TOK], n_le = 0;
  warp_rows_at_most<TOK>(a.row_start, a.batch, r0, n);
#pragma unroll
  for (int k = 0; k < TOK; ++k)
    if (k == tok) n_le = n[k];
  if (!have) return;
  const RowPlace pl = row_place(a.row_start, a.seq_len, a.batch, a.max_pages, a.n_rows, r, n_le);
  if (pl.b < 0) return;
  if (pl.pos < 0) {
    flag_error(a.dev_err, HS2_DEV_BAD_LENGTH);
    return;
  }
  const int phys = a.bt[(size_t)pl.b * a.max_pages + pl.pos / kPage];
  if (phys < 0 || phys >= a.num_pages) {
    flag_error(a.dev_err, HS2_DEV_BAD_PAGE);
    return;
  }
  const size_t slab = (size_t)phys * a.Hkv + g;
  const size_t line = slab * kPage + pl.pos % kPage;  // row of the pool
  put16<D, FMT>(a, side, slab, line, grp, x);
  if (SIDES == 2) put16<D, FMT>(a, 1, slab, line, grp, y);
}

// Four channels per lane, so that every store of a warp is contiguous; a warp takes as many
// rows of one head as the writing kernel's.
template <int D, int FMT, bool ROW_F32>
__global__ void __launch_bounds__(kRowThreads) kv_read_kernel(const RowsArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int TOK = 512 / D;        // rows per warp
  constexpr int LPR = D / 4;          // lanes per row
  constexpr int RPS = 32 / LPR;       // rows per step
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r0 = ((blockIdx.x - 1) * (kRowThreads / 32) + warp) * TOK;
  const int g = blockIdx.y, side = blockIdx.z;
  if (blockIdx.x == 0) {
    check_starts(a);
    return;
  }
  if (r0 >= a.n_rows) return;
  int n[TOK];
  warp_rows_at_most<TOK>(a.row_start, a.batch, r0, n);
  // lane k < TOK resolves row r0 + k: its pool row, or -1
  long long mine = -1;
  {
    int n_le = 0;
#pragma unroll
    for (int k = 0; k < TOK; ++k)
      if (k == lane) n_le = n[k];
    if (lane < TOK && r0 + lane < a.n_rows) {
      const RowPlace pl = row_place(a.row_start, a.seq_len, a.batch, a.max_pages, a.n_rows, r0 + lane, n_le);
      if (pl.b >= 0 && pl.pos < 0) flag_error(a.dev_err, HS2_DEV_BAD_LENGTH);
      if (pl.b >= 0 && pl.pos >= 0) {
        const int phys = a.bt[(size_t)pl.b * a.max_pages + pl.pos / kPage];
        if (phys < 0 || phys >= a.num_pages) flag_error(a.dev_err, HS2_DEV_BAD_PAGE);
        else mine = ((long long)phys * a.Hkv + g) * kPage + pl.pos % kPage;
      }
    }
  }
  const uint8_t* pool = reinterpret_cast<const uint8_t*>(side ? a.v : a.k);
  void* rows = const_cast<void*>(side ? a.v_rows : a.k_rows);
#pragma unroll
  for (int st = 0; st < TOK / RPS; ++st) {
    const int tok = st * RPS + lane / LPR, ch = 4 * (lane % LPR);
    const long long line = __shfl_sync(0xffffffffu, mine, tok);
    if (line < 0) continue;
    float x[4];
    if constexpr (FMT == HS2_F32) {
      const float4 v = *reinterpret_cast<const float4*>(pool + (line * D + ch) * 4);
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else if constexpr (FMT == HS2_BF16) {
      const uint2 v = *reinterpret_cast<const uint2*>(pool + (line * D + ch) * 2);
      x[0] = bf16_lo(v.x), x[1] = bf16_hi(v.x), x[2] = bf16_lo(v.y), x[3] = bf16_hi(v.y);
    } else {
      const float S = (side ? a.v_scale : a.k_scale)[line / kPage];
      uint32_t h0, h1;  // four values as f16 pairs, exact
      if constexpr (FMT == HS2_FP8_E4M3) {
        fp8x4_to_f16x4(*reinterpret_cast<const uint32_t*>(pool + line * D + ch), h0, h1);
      } else {
        uint32_t u2, u3;
        fp4x8_to_f16x8(*reinterpret_cast<const uint16_t*>(pool + line * (D / 2) + ch / 2), h0, h1, u2, u3);
        const uint32_t s = (side ? a.v_sf : a.k_sf)[line * (D / 16) + ch / 16];
        h0 = hmul2(h0, e4m3_pair(s, s));
        h1 = hmul2(h1, e4m3_pair(s, s));
      }
      const float2 f0 = __half22float2(*reinterpret_cast<__half2*>(&h0));
      const float2 f1 = __half22float2(*reinterpret_cast<__half2*>(&h1));
      x[0] = f0.x * S, x[1] = f0.y * S, x[2] = f1.x * S, x[3] = f1.y * S;
    }
    const long long at = (long long)(r0 + tok) * a.row_stride + g * D + ch;
    if constexpr (ROW_F32)
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(rows) + at) = make_float4(x[0], x[1], x[2], x[3]);
    else
      *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(rows) + at) =
          make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
  }
}

// From so many rows times heads on a thread finds a row's place once for K and V: 32768 rows of
// 4 heads written and read back 60 us with a thread a side and 55 with both, 4096 rows 13.5 and
// 12.5; below, more threads hide more of the latency: 1024 rows 8.4 and 10.3.
constexpr long long kTwoSides = 8192;

template <int D, int FMT>
cudaError_t launch_fmt(const RowsArgs& a, bool write, bool row_f32, cudaStream_t s) {
  const int per_cta = kRowThreads / (D / 16);
  const bool two = write && a.v && (long long)a.n_rows * a.Hkv >= kTwoSides;
  const dim3 grid((a.n_rows + per_cta - 1) / per_cta + 1, a.Hkv, a.v && !two ? 2 : 1);  // and a block that checks
  auto kern = write ? (two ? (row_f32 ? kv_write_kernel<D, FMT, true, 2> : kv_write_kernel<D, FMT, false, 2>)
                           : (row_f32 ? kv_write_kernel<D, FMT, true, 1> : kv_write_kernel<D, FMT, false, 1>))
                    : (row_f32 ? kv_read_kernel<D, FMT, true> : kv_read_kernel<D, FMT, false>);
  return launch_pdl(kern, grid, dim3(kRowThreads), 0, s, a);
}

template <int D>
cudaError_t launch_d(const RowsArgs& a, int dtype, bool write, bool row_f32, cudaStream_t s) {
  switch (dtype) {
    case HS2_F32: return launch_fmt<D, HS2_F32>(a, write, row_f32, s);
    case HS2_BF16: return launch_fmt<D, HS2_BF16>(a, write, row_f32, s);
    case HS2_FP8_E4M3: return launch_fmt<D, HS2_FP8_E4M3>(a, write, row_f32, s);
    case HS2_FP4_E2M1: return launch_fmt<D, HS2_FP4_E2M1>(a, write, row_f32, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_kv_rows(const RowsArgs& a, int d, int dtype, bool write, bool row_f32, cudaStream_t s) {
  return d == 128 ? launch_d<128>(a, dtype, write, row_f32, s) : launch_d<64>(a, dtype, write, row_f32, s);
}

}  // namespace hs2
