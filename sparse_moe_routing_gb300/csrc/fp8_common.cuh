// 8-bit floating point (e4m3) with one fp32 scale per block of 128: the
// arithmetic shared by the quantiser and the kernels that quantise on the way.
//
// A block (1 x 128 values of a row, or 128 x 128 of a matrix) with largest
// magnitude a is held as codes q = e4m3(x / s), rounded to nearest even, with
//   s = the smallest power of two with a / s <= 448 (e4m3's largest number),
//       at least 2^-126.
// Dividing by a power of two is exact, so a code is the single rounding of
// its value and does not depend on how a quotient was rounded (with s = a/448
// the quotients of bf16 values fall on ties of e4m3 often enough to move
// 1.7 % of a layer's output). e4m3's relative step is the same at every power
// of two, so no precision is lost but in its subnormals. A block that holds a
// value that is not finite gets the scale NaN and NaN codes.
#pragma once

#include "common.cuh"
#include "tc_ptx.cuh"

namespace moe {

constexpr int kF8Block = 128;      // values per scale along a row
constexpr uint32_t kF8NanScale = 0x7FFFFFFFu;

__host__ __device__ __forceinline__ int f8_blocks(int n) { return (n + kF8Block - 1) / kF8Block; }

// Bits of the scale for a block whose largest magnitude has the bits `amax`
// (sign clear; magnitudes of fp32 numbers order like their bits, with NaN and
// infinity above every finite number).
__device__ __forceinline__ uint32_t f8_scale_bits(uint32_t amax) {
  if (amax >= 0x7F800000u) return kF8NanScale;
  // amax = 1.f * 2^(e - 127); 448 = 1.75 * 2^8: one power higher past 1.75
  const int e = (int)(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)(e < 1 ? 1 : e) << 23;
}
// 1 / s, exactly (NaN for the NaN scale).
__device__ __forceinline__ float f8_inverse(uint32_t scale_bits) {
  return __uint_as_float(scale_bits == kF8NanScale ? kF8NanScale : (254u << 23) - scale_bits);
}
__device__ __forceinline__ uint32_t f8_mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Four values already divided by their scale -> four codes, the first in the
// low byte.
__device__ __forceinline__ uint32_t f8_pack4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n .reg .b16 lo, hi;\n"
      " cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n"
      " cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
      " mov.b32 %0, {lo, hi};\n}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// One thread waits for a phase of `bar`; false when the wait ran out of its
// limit or *abort_flag (if given) was raised.
__device__ __forceinline__ bool f8_lane_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns,
                                             const volatile int* abort_flag) {
  if (tc::mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = 0;
  for (uint32_t n = 1; !tc::mbar_try_wait(bar, parity); ++n) {
    if ((n & 63u) == 0) {
      if (abort_flag && *abort_flag) return false;
      if (t0 == 0) t0 = globaltimer_ns();
      if (globaltimer_ns() - t0 > limit_ns) return false;
    }
  }
  return true;
}
// The whole warp waits. Every lane polls: one lane's poll with its outcome
// shuffled to the others took 1390 cycles for a round trip between one warp
// and sixteen, this 260 (measured alone).
__device__ __forceinline__ bool f8_warp_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns, Ctrl* ctrl,
                                             uint32_t site) {
  const bool ok = __all_sync(0xffffffffu, f8_lane_wait(bar, parity, limit_ns, nullptr));
  if (!ok) {
    if ((threadIdx.x & 31) == 0) report(ctrl, kDevTimeout, site);
    // copies already in flight land before the warp can leave
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000ull) {
    }
  }
  return ok;
}

}  // namespace moe
