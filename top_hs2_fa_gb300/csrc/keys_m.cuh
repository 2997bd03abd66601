// keys_m.cuh — what the attention kernels share that take the keys as the M side of tcgen05.mma and
// the query rows as N: S^T[keys][rows], O^T[channels][rows], a softmax thread per key.
#pragma once
#include "tc.cuh"

namespace hs2 {

constexpr float kBias = 6.f;     // log2 of the weight of a key at the reference max
constexpr float kTop = 14.f;     // log2 of the largest weight before the reference moves
constexpr float kUnset = 1e30f;  // nm of a row that has seen no key

template <typename S>
HS2_DEVI bool halted(S& sm) { return *(volatile int*)&sm.abort != 0; }
template <typename S>
HS2_DEVI void halt(S& sm, int32_t* dev_err) {
  flag_error(dev_err, HS2_DEV_TIMEOUT);
  atomicExch(&sm.abort, 1);
}

// Barrier `id` of the 128 threads of a softmax group: whether any of them passes true.
HS2_DEVI bool any_of_128(int id, bool v) {
  int r;
  asm volatile(
      "{.reg .pred p, q; setp.ne.b32 q, %1, 0;\n\tbar.red.or.pred p, %2, 128, q;\n\tselp.b32 %0, 1, 0, p;}"
      : "=r"(r)
      : "r"((int)v), "r"(id)
      : "memory");
  return r != 0;
}

HS2_DEVI float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// C columns of a lane quadrant into registers (8, 16 or 32), or back.
template <int C>
HS2_DEVI void tmem_cols(uint32_t addr, float (&x)[C]) {
  if constexpr (C == 32) {
    tc::tmem_ld32(addr, x);
  } else if constexpr (C == 8) {
    uint32_t r[8];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(addr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(r[i]);
  } else {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(r[i]);
  }
}
template <int C>
HS2_DEVI void tmem_put(uint32_t addr, const float (&x)[C]) {
  if constexpr (C == 32) {
    tc::tmem_st32(addr, x);
  } else if constexpr (C == 8) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n\t"
        "tcgen05.wait::st.sync.aligned;" ::"r"(addr),
        "r"(__float_as_uint(x[0])), "r"(__float_as_uint(x[1])), "r"(__float_as_uint(x[2])), "r"(__float_as_uint(x[3])),
        "r"(__float_as_uint(x[4])), "r"(__float_as_uint(x[5])), "r"(__float_as_uint(x[6])), "r"(__float_as_uint(x[7]))
        : "memory");
  } else {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n\t"
        "tcgen05.wait::st.sync.aligned;" ::"r"(addr),
        "r"(__float_as_uint(x[0])), "r"(__float_as_uint(x[1])), "r"(__float_as_uint(x[2])), "r"(__float_as_uint(x[3])),
        "r"(__float_as_uint(x[4])), "r"(__float_as_uint(x[5])), "r"(__float_as_uint(x[6])), "r"(__float_as_uint(x[7])),
        "r"(__float_as_uint(x[8])), "r"(__float_as_uint(x[9])), "r"(__float_as_uint(x[10])), "r"(__float_as_uint(x[11])),
        "r"(__float_as_uint(x[12])), "r"(__float_as_uint(x[13])), "r"(__float_as_uint(x[14])), "r"(__float_as_uint(x[15]))
        : "memory");
  }
}

// Sums of 32 per-lane values over the warp's lanes: lane i gets the sum of column `i`.
HS2_DEVI float transpose_sum32(float (&v)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    const bool up = lane & s;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (i < s) {
        const float give = up ? v[i] : v[i + s], keep = up ? v[i + s] : v[i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, s);
      }
    }
  }
  return v[0];
}

// kind::f16 instruction descriptor: M = 128, N, fp32 accumulators, f16 or bf16 operands.
HS2_DEVI constexpr uint32_t narrow_idesc(bool bf16, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         ((uint32_t)(N >> 3) << 17) | (8u << 24);
}

}  // namespace hs2
