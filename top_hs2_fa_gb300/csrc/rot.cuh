// rot.cuh — rotation of a head's channels by a token's position, 16 channels a lane.
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

// cos and sin of the 16 channels of group grp (of grp < R / 16 groups): one for each channel.
HS2_DEVI void load_angles(const RotTable& t, int pos, int grp, float (&cs)[16], float (&sn)[16]) {
  const int half = t.dim / 2;
  const float* row = t.table + (size_t)pos * t.dim;
  if (t.pairs) {
    const float4* c = reinterpret_cast<const float4*>(row + 8 * grp);
    const float4* s = reinterpret_cast<const float4*>(row + half + 8 * grp);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 u = __ldg(c + i), v = __ldg(s + i);
      cs[8 * i] = cs[8 * i + 1] = u.x, cs[8 * i + 2] = cs[8 * i + 3] = u.y;
      cs[8 * i + 4] = cs[8 * i + 5] = u.z, cs[8 * i + 6] = cs[8 * i + 7] = u.w;
      sn[8 * i] = sn[8 * i + 1] = v.x, sn[8 * i + 2] = sn[8 * i + 3] = v.y;
      sn[8 * i + 4] = sn[8 * i + 5] = v.z, sn[8 * i + 6] = sn[8 * i + 7] = v.w;
    }
  } else {
    const int at = 16 * grp < half ? 16 * grp : 16 * grp - half;
    const float4* c = reinterpret_cast<const float4*>(row + at);
    const float4* s = reinterpret_cast<const float4*>(row + half + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 u = __ldg(c + i), v = __ldg(s + i);
      cs[4 * i] = u.x, cs[4 * i + 1] = u.y, cs[4 * i + 2] = u.z, cs[4 * i + 3] = u.w;
      sn[4 * i] = v.x, sn[4 * i + 1] = v.y, sn[4 * i + 2] = v.z, sn[4 * i + 3] = v.w;
    }
  }
}

// x rotated, for the lanes with `turn`; the whole warp calls it. Lanes of one head are neighbours,
// lane - grp the first.
HS2_DEVI void rotate16(const RotTable& t, int grp, bool turn, const float (&cs)[16], const float (&sn)[16], float (&x)[16]) {
  if (t.pairs) {
    if (!turn) return;
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float a = x[i], b = x[i + 1];
      x[i] = __fsub_rn(__fmul_rn(a, cs[i]), __fmul_rn(b, sn[i]));
      x[i + 1] = __fadd_rn(__fmul_rn(b, cs[i]), __fmul_rn(a, sn[i]));
    }
    return;
  }
  const int lane = threadIdx.x & 31, h = t.dim / 32;  // groups of a half
  const bool first = grp < h;
  const int other = lane + (first ? h : -h);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float y = __shfl_sync(0xffffffffu, x[i], other & 31);
    const float p = __fmul_rn(x[i], cs[i]), q = __fmul_rn(y, sn[i]);
    if (turn) x[i] = first ? __fsub_rn(p, q) : __fadd_rn(p, q);
  }
}

// 16 channels to a row of floats or bfloat16.
template <bool F32>
HS2_DEVI void store16(void* rows, long long at, const float (&x)[16]) {
  if constexpr (F32) {
    float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(rows) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  } else {
    uint4* p = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(rows) + at);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      p[i] = make_uint4(pack_bf16(x[8 * i], x[8 * i + 1]), pack_bf16(x[8 * i + 2], x[8 * i + 3]),
                        pack_bf16(x[8 * i + 4], x[8 * i + 5]), pack_bf16(x[8 * i + 6], x[8 * i + 7]));
  }
}

}  // namespace hs2
