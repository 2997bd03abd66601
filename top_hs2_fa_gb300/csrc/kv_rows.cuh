// kv_rows.cuh — 16 channels of a row of a ragged batch: loaded, quantised to the cache's type, put
// in their place.
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
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "ragged.cuh"

namespace hs2 {

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

// 16 values as E4M3 codes under slab scale S, four to a word; whether S is one that rows are written under.
HS2_DEVI bool fp8_codes(const RowsArgs& a, float S, const float (&x)[16], uint32_t (&w)[4]) {
  if (!(S >= 0x1p-60f && S <= 0x1p60f)) {
    flag_error(a.dev_err, HS2_DEV_BAD_PAGE);
    return false;
  }
  const float inv = 1.f / S;
  float q[16];
  quotients<5>(x, inv, S, 0.f, q);
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = e4m3_codes(q[4 * i], q[4 * i + 1]) | (e4m3_codes(q[4 * i + 2], q[4 * i + 3]) << 16);
  return true;
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
    if constexpr (FMT == HS2_FP8_E4M3) {
      uint32_t w[4];
      if (fp8_codes(a, S, x, w)) *reinterpret_cast<uint4*>(pool + line * D + 16 * grp) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      if (!(S >= 0x1p-60f && S <= 0x1p60f)) {
        flag_error(a.dev_err, HS2_DEV_BAD_PAGE);
        return;
      }
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

}  // namespace hs2
