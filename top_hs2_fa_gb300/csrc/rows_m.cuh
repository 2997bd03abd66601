// rows_m.cuh — what the attention kernels share that take 256 query rows as two M = 128 halves which
// take turns on the tensor pipe: S[rows][keys], a softmax thread per row, P over S in tensor memory.
#pragma once
#include "common.cuh"

namespace hs2 {

constexpr int kWRows = 128;      // rows of a half
constexpr int kWThreads = 384;
constexpr uint32_t kWTmem = 512;
constexpr float kWRescale = 8.f;
// Registers per thread of the three 128-thread groups, of the 3 * 168 of the launch.
constexpr int kWRegsMisc = 64, kWRegsSoftmax = 216;

template <typename S>
HS2_DEVI bool stopped(S& sm) { return *(volatile int*)&sm.abort != 0; }
template <typename S>
HS2_DEVI void stop(S& sm, int32_t* dev_err) {
  flag_error(dev_err, HS2_DEV_TIMEOUT);
  atomicExch(&sm.abort, 1);
}

HS2_DEVI float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Bits 0 .. n of a word (none for n < 0).
HS2_DEVI uint32_t bits_upto(int n) { return n < 0 ? 0u : n >= 31 ? ~0u : (2u << n) - 1u; }

// A whole 32-byte sector from one thread (halves of sectors took 3 to 12 % longer where units are
// cut, e.g. 49 against 43 us for 512 tokens over 2048 keys).
HS2_DEVI void store8(float* p, const float* x) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]),
               "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
               : "memory");
}
template <int R>
HS2_DEVI void wide_regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
HS2_DEVI void wide_regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }

}  // namespace hs2
