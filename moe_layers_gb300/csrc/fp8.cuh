// 8-bit (e4m3) numbers and their scales.
#pragma once

#include "common.cuh"

namespace dec {

// Four floats to e4m3, nearest-even, held at +-448; NaN stays NaN. The first is
// the lowest byte.
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
      "mov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// The two bf16 values of each word added in fp32 and rounded to bf16.
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  return pack_bf16x2(bf_lo(a) + bf_lo(b), bf_hi(a) + bf_hi(b));
}

// The scale of a group whose largest absolute value is `most`, and the factor
// that takes its values to e4m3's range. Both are normal fp32 numbers down to
// 2^-117.2 (the scale; the factor would pass fp32's range at 2^-119.2): below
// 2^-116 a group counts as zeros. An infinity has factor 0 (the
// group's infinities become NaN, the rest 0) and scale infinity.
struct Scale8 {
  float scale, up;
};
__device__ __forceinline__ Scale8 scale_e4m3(float most) {
  if (most < 0x1p-116f) return {0.f, 0.f};
  return {__fdiv_rn(most, 448.f), __fdiv_rn(448.f, most)};
}

// D += A B^T on e4m3 operands: 16 rows x 32 columns of A, 8 x 32 of B, fp32
// accumulators. Lane 4 g + t holds of A the words (row g, word t), (g + 8, t),
// (g, t + 4), (g + 8, t + 4), of B (g, t) and (g, t + 4), and of D the elements
// (g, 2 t), (g, 2 t + 1), (g + 8, 2 t), (g + 8, 2 t + 1).
__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Bounded wait of a pipeline whose next step is near. The first tries do without the global
// timer, whose reading costs more than the wait that is left then; no call, so that a kernel
// that moves registers between its warps can use it. Ends early when another role of the
// CTA has given up (wc.abort null: only by the limit).
__device__ __forceinline__ bool mbar_wait_soon(uint64_t* bar, uint32_t parity, const WaitCtl& wc) {
  uint64_t t0 = 0;
  for (uint32_t n = 1;; ++n) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((n & 31u) != 0) continue;
    if (wc.abort != nullptr && *wc.abort) return false;
    const uint64_t now = globaltimer();
    if (t0 == 0) t0 = now;
    if (now - t0 > wc.limit_ns) {
      if (wc.abort != nullptr) *wc.abort = 1;
      atomicOr(wc.err, DEV_ERR_TIMEOUT);
      return false;
    }
  }
}

}  // namespace dec
