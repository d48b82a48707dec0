// cache.cuh -- what the kernels of the 8-bit key/value cache share: the 8-bit
// formats' conversions and the search for a packed token's sequence.
#pragma once
#include "common.cuh"
#include "ptx.cuh"

namespace fattn {

// Two 8-bit codes (low byte first) -> two fp16 values (low half first), exact.
template <bool E5M2>
__device__ __forceinline__ uint32_t codes_to_f16x2(uint16_t c) {
  uint32_t r;
  if constexpr (E5M2)
    asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(r) : "h"(c));
  else
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
// Four codes (low byte first) -> two pairs of fp16 values.
template <bool E5M2>
__device__ __forceinline__ void codes4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (E5M2)  // the upper byte of the fp16 value
    lo = __byte_perm(w, 0u, 0x1404u), hi = __byte_perm(w, 0u, 0x3424u);
  else
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h) {
  float2 f;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %2;\n\t"
      "cvt.f32.f16 %0, lo;\n\t"
      "cvt.f32.f16 %1, hi;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}
// Two fp32 values -> two codes (lo in the low byte), to nearest even; NaN stays NaN.
template <bool E5M2>
__device__ __forceinline__ uint16_t f32_to_codes(float lo, float hi) {
  uint16_t r;
  if constexpr (E5M2)
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// 0x80 in the byte of each of four codes that stands for NaN (or, in e5m2, for
// infinity): the magnitudes from the first such code on carry into the sign bit.
template <bool E5M2>
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + (E5M2 ? 0x04040404u : 0x01010101u)) & 0x80808080u;
}
// The four codes with zeros in the bytes that `m` (of nan_codes) marks.
__device__ __forceinline__ uint32_t clear_codes(uint32_t w, uint32_t m) {
  return w & ~(m | (m - (m >> 7)));
}

// The largest b in [0, B) with first(b) <= x, for a non-decreasing first() with
// first(0) <= x, found by the whole warp: 32 probes a step, so one step serves
// 32 sequences and two 1024 (a binary search would wait for 5 or 10 loads in
// turn).  Any values keep it inside [0, B).
template <typename First>
__device__ __forceinline__ int warp_search(int B, long long x, First first) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + lane * step;
    const unsigned yes = __ballot_sync(0xffffffffu, lane == 0 || (i < hi && first(i) <= x));
    const int last = yes == 0xffffffffu ? 31 : __ffs(~yes) - 2;  // the last probe that holds
    lo += last * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

}  // namespace fattn
