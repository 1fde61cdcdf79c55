// 8-bit integer products: what the kernels for few and for many rows share.
//
// out[m][n] = (sum_k a[m][k] b[n][k]) * a_scale[m] * b_scale[n], codes in
// [-128, 127]. The sum is exact (int32; K <= kI8MaxK keeps it below 2^31); then
// fp32: the sum rounded once, two products, one rounding to the result's type.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace moe {

__device__ __forceinline__ float i8_value(int sum, float a_scale, float b_scale) {
  return __int2float_rn(sum) * a_scale * b_scale;
}
__device__ __forceinline__ void i8_store(void* out, size_t at, bool bf16, float v) {
  if (bf16)
    static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(out)[at] = v;
}

// Four codes (the first in the low byte) as fp16 values, exactly: 0x6400 | u is
// 1024 + u in fp16, u = code + 128.
__device__ __forceinline__ void i8_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  lo = __byte_perm(u, 0x64646464u, 0x4140);
  hi = __byte_perm(u, 0x64646464u, 0x4342);
  constexpr uint32_t kBias = 0xE480E480u;  // -1152 twice
  asm("add.rn.f16x2 %0, %0, %1;" : "+r"(lo) : "r"(kBias));
  asm("add.rn.f16x2 %0, %0, %1;" : "+r"(hi) : "r"(kBias));
}

// 16 codes at column k of a row of K: zeros past the row's end, no byte past it
// read.
__device__ __forceinline__ uint4 i8_load16(const uint8_t* row, int k, int K) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (k + 16 <= K) {
    v = *reinterpret_cast<const uint4*>(row + k);
  } else if (k < K) {
    uint32_t w[4] = {};
#pragma unroll
    for (int j = 0; j < 15; ++j)
      if (k + j < K) w[j >> 2] |= (uint32_t)row[k + j] << (8 * (j & 3));
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return v;
}

}  // namespace moe
