// rot.cuh — rotation of a head's channels by a token's position, 16 channels (8 pairs) a lane.
//
// Pair i of a position p with table row (cos_0 .. cos_{R/2-1}, sin_0 .. sin_{R/2-1}), R channels
// rotated: a' = a cos_i - b sin_i, b' = b cos_i + a sin_i, (a, b) = (x_i, x_{i + R/2}) (halves) or
// (x_2i, x_2i+1) (pairs). Each product and sum is rounded on its own, so that the result is the one
// that float32 operations one after another give: a value near a border between two codes of an
// FP8 / FP4 cache falls where a program that rotates first would have it.
#pragma once
#include "common.cuh"
#include "kernels.h"

namespace hs2 {

// A lane's 16 channels of a head of D: 8 from `lo` and 8 from `hi` on, where neighbouring lanes' pieces of
// 8 are neighbours (16 in a row made every access of bfloat16 rows half sectors: 26273 latent rows with 32
// heads took 73 us). Lanes [0, R / 16) have 8 pairs, of halves x[i] with x[8 + i], the others channels
// that are not rotated.
struct LaneChannels {
  int lo, hi;
  bool turn;  // whether they are rotated
};
HS2_DEVI LaneChannels lane_channels(const RotTable& t, int D, int grp) {
  const int n = t.dim / 16;
  if (grp < n) return {8 * grp, 8 * grp + t.dim / 2, true};
  return {t.dim + 8 * (grp - n), t.dim + 8 * (grp - n) + (D - t.dim) / 2, false};
}

// cos and sin of a lane's 8 pairs.
HS2_DEVI void load_angles(const RotTable& t, int pos, int grp, float (&cs)[8], float (&sn)[8]) {
  // halves: pairs [8 g, 8 g + 8); neighbours: 4 of either piece
  const float* row = t.table + (size_t)pos * t.dim + (t.pairs ? 4 * grp : 8 * grp);
  const int next = t.pairs ? t.dim / 4 : 4;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 u = __ldg(reinterpret_cast<const float4*>(row + i * next));
    const float4 v = __ldg(reinterpret_cast<const float4*>(row + t.dim / 2 + i * next));
    cs[4 * i] = u.x, cs[4 * i + 1] = u.y, cs[4 * i + 2] = u.z, cs[4 * i + 3] = u.w;
    sn[4 * i] = v.x, sn[4 * i + 1] = v.y, sn[4 * i + 2] = v.z, sn[4 * i + 3] = v.w;
  }
}

HS2_DEVI void turn_pair(float& a, float& b, float c, float s) {
  const float x = a, y = b;
  a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
  b = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
}
HS2_DEVI void rotate16(const RotTable& t, const float (&cs)[8], const float (&sn)[8], float (&x)[16]) {
  if (t.pairs) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn_pair(x[2 * i], x[2 * i + 1], cs[i], sn[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn_pair(x[i], x[8 + i], cs[i], sn[i]);
  }
}

// 8 channels of a row of floats or bfloat16.
template <bool F32>
HS2_DEVI void load8(const void* rows, long long at, float* x) {
  if constexpr (F32) {
    const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(rows) + at);
    const float4 u = p[0], v = p[1];
    x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(rows) + at);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) x[2 * j] = bf16_lo(w[j]), x[2 * j + 1] = bf16_hi(w[j]);
  }
}
template <bool F32>
HS2_DEVI void store8(void* rows, long long at, const float* x) {
  if constexpr (F32) {
    float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(rows) + at);
    p[0] = make_float4(x[0], x[1], x[2], x[3]), p[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(rows) + at) =
        make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  }
}

}  // namespace hs2
