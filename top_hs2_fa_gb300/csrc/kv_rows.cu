// kv_rows.cu — rows of a ragged batch into a paged cache (quantised on the way) and back.
//
// At prefill each Cross group's cache gains the prompt's bridged K/V rows, at decode one row
// per sequence ("HySparse2：整体架构、KV 生命周期与 PD 分离", §8, §10.1); an FP4 cache keeps E2M1
// codes with one E4M3 scale per 16 channels ("2.3.1 · CSA、HCA 与 CSA2", §3, "KV 字节与 FP4").
//
// FP4 of a group of 16 values x_j with slab scale S: A = max |x_j|, s the smallest E4M3 value
// with 6 s S >= A, code_j the E2M1 value nearest to x_j / (s S), ties to the even code, as exact
// arithmetic has it. q = x * (1 / (s S)) in fp32 is within 4 units in the last place of the
// quotient, so rounding q gives that code unless a border between codes (0.25 .. 5, numbers of at most
// 3 significant bits) lies within them; such a q has the low bits of its mantissa near zero
// (low_bits), which one value in 10^5 has by chance, and many have where rows and scales are short
// numbers. A thread that meets one rounds its quotients to odd by their exact remainders, which
// keeps what the rounding to a code has to see (quotients). FP8 likewise, the borders of E4M3
// having at most 5 bits. S in [2^-60, 2^60] keeps all products away from under- and overflow.
//
// 32768 rows of 2 x 4 x 128 bf16 values to FP4 (86 MB) take 26 us with slab scales of many bits and
// 39 with a power of two, where nearly every group meets a border (comparing every value against the
// borders took 46). With many bits the wait for the rows bounds it (64 registers leave half of the
// warps; ALU 47 % busy, HBM 0.54 of the copy rate over 393216 rows), with a power of two the integer
// pipe (68 %). Their way back to floats (153 MB) takes 29 us.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "ragged.cuh"

namespace hs2 {

namespace {

constexpr int kRowThreads = 256;

HS2_DEVI float e4m3_value(uint32_t code) {
  float f;
  asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;}" : "=f"(f) : "r"(fp8x2_to_f16x2(code & 0xFFu)));
  return f;
}
// two floats to E4M3 codes, nearest even, saturating (NaN: 0x7F); a in the low byte
HS2_DEVI uint32_t e4m3_codes(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// The smallest E4M3 code whose value s has 6 s S >= A (A finite or inf); 126 (448) where none has.
HS2_DEVI uint32_t group_scale(float A, float S) {
  // the nearest code to about A / (6 S) is the one sought or the one before it
  const uint32_t c = e4m3_codes(A / (6.f * S), 0.f) & 0xFFu;
  const float a = 6.f * e4m3_value(c), p = a * S;
  const bool short_of = p < A || (p == A && fmaf(a, S, -p) < 0.f);
  return c + (short_of && c < 126u);
}

// Whether a quotient q is within 8 units in its last place of a number of so few significant bits
// (a border between codes) is low_bits(q) < kNear.
template <int BITS>
HS2_DEVI uint32_t low_bits(float q) { return (__float_as_uint(q) + 8u) & ((1u << (24 - BITS)) - 1u); }
constexpr uint32_t kNear = 16;

// q[j]: what rounds to the code of x[j] / (d + e), where d + e is exact, |e| at most half a unit of
// d, inv about 1 / d, and the borders between codes have BITS significant bits. The corrected
// quotient is within a unit, and its remainder exact in sign (a multiple of 2^-126 where the
// quotient is 2^-11 or more; smaller ones have code 0 anyway): a quotient that is not exact
// moves to the odd neighbour on its side, so that it is no border and lies on the same side of
// each as the true one.
template <int BITS>
HS2_DEVI void quotients(const float (&x)[16], float inv, float d, float e, float (&q)[16]) {
  uint32_t low = kNear;
#pragma unroll
  for (int j = 0; j < 16; j += 2) {
    q[j] = x[j] * inv, q[j + 1] = x[j + 1] * inv;
    low = __vimin3_u32(low, low_bits<BITS>(q[j]), low_bits<BITS>(q[j + 1]));
  }
  if (low >= kNear) return;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    if (!(fabsf(q[j]) < 1024.f)) continue;  // saturates, or NaN
    q[j] = copysignf(fmaf(fmaf(-q[j], e, fmaf(-q[j], d, x[j])), inv, q[j]), x[j]);  // (the sign of zeros)
    const float rest = fmaf(-q[j], e, fmaf(-q[j], d, x[j]));
    const uint32_t u = __float_as_uint(q[j]), some = rest != 0.f;
    const uint32_t toward = ((u ^ __float_as_uint(rest)) >> 31) & some;  // the true quotient is smaller
    q[j] = __uint_as_float((u - toward) | some);
  }
}

HS2_DEVI float max_nan3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// eight floats to E2M1 codes, nearest even, saturating; x[0] in the low nibble
HS2_DEVI uint32_t e2m1_codes(const float* x) {
  uint32_t r;
  asm("{.reg .b8 a, b, c, d;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\tmov.b32 %0, {a, b, c, d};}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

template <bool ROW_F32>
HS2_DEVI void load16(const void* rows, long long at, float (&x)[16]) {
  if constexpr (ROW_F32) {
    const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(rows) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = __ldg(p + i);
      x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
    }
  } else {
    const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(rows) + at);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 v = __ldg(p + i);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) x[8 * i + 2 * j] = bf16_lo(w[j]), x[8 * i + 2 * j + 1] = bf16_hi(w[j]);
    }
  }
}

// Faults of the row starts that no row meets, by a block of its own at the front of the grid: 32768
// rows in and out take 0.5 us longer for it, with the block at the end 1.7, by a warp that has rows
// too 1.2 (4.2 once its rows are done: the kernel then needs more registers).
HS2_DEVI void check_starts(const RowsArgs& a) {
  if (threadIdx.x < 32 && blockIdx.y == 0 && blockIdx.z == 0 && warp_bad_starts(a.row_start, a.batch, a.n_rows) &&
      threadIdx.x == 0)
    flag_error(a.dev_err, HS2_DEV_BAD_LENGTH);
}

// One side's 16 channels to their place.
template <int D, int FMT>
HS2_DEVI void put16(const RowsArgs& a, int side, size_t slab, size_t line, int grp, const float (&x)[16]) {
  constexpr int GPR = D / 16;
  uint8_t* pool = reinterpret_cast<uint8_t*>(side ? a.v : a.k);
  if constexpr (FMT == HS2_F32) {
    float4* dst = reinterpret_cast<float4*>(pool + (line * D + 16 * grp) * 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) dst[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  } else if constexpr (FMT == HS2_BF16) {
    uint4* dst = reinterpret_cast<uint4*>(pool + (line * D + 16 * grp) * 2);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      dst[i] = make_uint4(pack_bf16(x[8 * i], x[8 * i + 1]), pack_bf16(x[8 * i + 2], x[8 * i + 3]),
                          pack_bf16(x[8 * i + 4], x[8 * i + 5]), pack_bf16(x[8 * i + 6], x[8 * i + 7]));
  } else {
    const float S = (side ? a.v_scale : a.k_scale)[slab];
    if (!(S >= 0x1p-60f && S <= 0x1p60f)) {
      flag_error(a.dev_err, HS2_DEV_BAD_PAGE);
      return;
    }
    if constexpr (FMT == HS2_FP8_E4M3) {
      const float inv = 1.f / S;
      float q[16];
      quotients<5>(x, inv, S, 0.f, q);
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = e4m3_codes(q[4 * i], q[4 * i + 1]) | (e4m3_codes(q[4 * i + 2], q[4 * i + 3]) << 16);
      *reinterpret_cast<uint4*>(pool + line * D + 16 * grp) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      float top = fabsf(x[0]);  // the largest magnitude, or NaN
#pragma unroll
      for (int j = 1; j < 15; j += 2) top = max_nan3(top, fabsf(x[j]), fabsf(x[j + 1]));
      top = max_nan3(top, fabsf(x[15]), 0.f);
      const bool nan = top != top;
      const uint32_t s = nan ? 0x7Fu : group_scale(top, S);
      const float sv = nan ? 0.f : e4m3_value(s);
      const float d = sv * S, inv = sv > 0.f ? 1.f / d : 0.f;
      float q[16];
      quotients<3>(x, inv, d, fmaf(sv, S, -d), q);
      const uint32_t w[2] = {e2m1_codes(q), e2m1_codes(q + 8)};
      *reinterpret_cast<uint2*>(pool + line * (D / 2) + 8 * grp) = make_uint2(w[0], w[1]);
      (side ? a.v_sf : a.k_sf)[line * GPR + grp] = (uint8_t)s;
    }
  }
}

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
