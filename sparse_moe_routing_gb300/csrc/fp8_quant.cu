// Quantiser: values -> e4m3 codes and scales (the format of fp8_common.cuh).
//
//  * quant_rows: one scale per 1 x 128 block. Sixteen lanes own a block, eight
//    values each; the largest magnitude is a four-step shuffle maximum of the
//    magnitudes' bits. The values stay in registers between the maximum and
//    the division, so x is read once.
//  * quant_tiles: one scale per 128 x 128 block, one CTA each, the block's
//    values in registers between the two steps.
//  * quant_pack: quant_rows of a layer's tokens straight into the packed row
//    order of the grouped products (one row per routed pair, then the tokens'
//    own rows for the shared expert): the row is read and quantised once and
//    its codes are written k (+ 1) times.
//
// All are bound by HBM: bytes in plus one byte per value out.
#include "fp8_common.cuh"
#include "kernels.h"

namespace moe {
namespace {

// Eight consecutive values at p (16-byte aligned in the vector form).
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8]) {
  Chunk<__nv_bfloat16>::unpack(ldg_stream(p), v);
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
  Chunk<float>::unpack(ldg_stream(p), v);
  Chunk<float>::unpack(ldg_stream(p + 4), v + 4);
}

template <typename T, bool VEC>
__device__ __forceinline__ void load8_upto(const T* row, int c, int cols, float (&v)[8]) {
  if (VEC) {
    if (c < cols) {
      load8(row + c, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c + j < cols ? load_act(row, (size_t)(c + j)) : 0.f;
  }
}

__device__ __forceinline__ uint32_t mag_max8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, f8_mag(v[j]));
  return m;
}
// Maximum over the 16 lanes of a half warp.
__device__ __forceinline__ uint32_t half_max(uint32_t m) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv) {
  return make_uint2(f8_pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                    f8_pack4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
}
// Writes up to eight codes at column c; whole pairs of words where they fit.
template <bool VEC>
__device__ __forceinline__ void store_codes8(uint8_t* row, int c, int cols, uint2 q) {
  if (VEC) {
    if (c < cols) *reinterpret_cast<uint2*>(row + c) = q;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t w = j < 4 ? q.x : q.y;
      if (c + j < cols) row[c + j] = (uint8_t)(w >> (8 * (j & 3)));
    }
  }
}

constexpr int kQuantThreads = 256;
constexpr int kQuantUnroll = 4;  // blocks per half warp in flight

template <typename T, bool VEC>
__global__ void __launch_bounds__(kQuantThreads) quant_rows_kernel(F8QuantArgs a) {
  pdl_wait();
  pdl_trigger();
  const int nb = f8_blocks(a.cols);
  const long long total = (long long)a.rows * nb;
  const int lane16 = threadIdx.x & 15;
  const long long half = (long long)blockIdx.x * (kQuantThreads / 16) + (threadIdx.x >> 4);
  const long long step = (long long)gridDim.x * (kQuantThreads / 16);
  // whole warps stay in the loop: both halves of a warp shuffle together
  for (long long b0 = half; b0 - (half & 1) < total; b0 += step * kQuantUnroll) {
    float v[kQuantUnroll][8];
    long long row[kQuantUnroll];
    int blk[kQuantUnroll];
#pragma unroll
    for (int u = 0; u < kQuantUnroll; ++u) {
      const long long b = b0 + u * step;
      row[u] = b < total ? b / nb : -1;
      blk[u] = b < total ? (int)(b - row[u] * nb) : 0;
      const T* src = static_cast<const T*>(a.x) + (row[u] < 0 ? 0 : row[u]) * a.ldx;
      load8_upto<T, VEC>(src, blk[u] * kF8Block + lane16 * 8, row[u] < 0 ? 0 : a.cols, v[u]);
    }
#pragma unroll
    for (int u = 0; u < kQuantUnroll; ++u) {
      const uint32_t sb = f8_scale_bits(half_max(mag_max8(v[u])));
      if (row[u] < 0) continue;
      store_codes8<VEC>(a.codes + row[u] * a.ldq, blk[u] * kF8Block + lane16 * 8, a.cols,
                        codes8(v[u], f8_inverse(sb)));
      if (lane16 == 0) a.scales[row[u] * nb + blk[u]] = __uint_as_float(sb);
    }
  }
}

// One 128 x 128 block per CTA: 256 threads, 16 per row, 8 row groups of 16.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kQuantThreads) quant_tiles_kernel(F8QuantArgs a) {
  __shared__ uint32_t s_max[kQuantThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int nb = f8_blocks(a.cols), nr = f8_blocks(a.rows);
  const long long tile = blockIdx.x;
  const int cb = (int)(tile % nb);
  const long long rest = tile / nb;
  const int rb = (int)(rest % nr);
  const long long mat = rest / nr;
  const int r0 = rb * kF8Block + (threadIdx.x >> 4), c = cb * kF8Block + (threadIdx.x & 15) * 8;
  const T* x = static_cast<const T*>(a.x) + mat * (long long)a.rows * a.ldx;
  uint8_t* codes = a.codes + mat * (long long)a.rows * a.ldq;
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 16 * i;
    load8_upto<T, VEC>(x + (long long)min(r, a.rows - 1) * a.ldx, c, r < a.rows ? a.cols : 0, v[i]);
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, mag_max8(v[i]));
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kQuantThreads / 32; ++w) m = max(m, s_max[w]);
  const uint32_t sb = f8_scale_bits(m);
  const float inv = f8_inverse(sb);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 16 * i;
    if (r < a.rows) store_codes8<VEC>(codes + (long long)r * a.ldq, c, a.cols, codes8(v[i], inv));
  }
  if (threadIdx.x == 0) a.scales[(mat * nr + rb) * nb + cb] = __uint_as_float(sb);
}

// Half warp per (token, block); d is a multiple of 16.
__global__ void __launch_bounds__(kQuantThreads) quant_pack_kernel(F8PackArgs a) {
  pdl_wait();
  pdl_trigger();
  const int nb = f8_blocks(a.d);
  const long long total = (long long)a.T * nb;
  const int lane16 = threadIdx.x & 15;
  const long long half = (long long)blockIdx.x * (kQuantThreads / 16) + (threadIdx.x >> 4);
  const long long b = half;
  float v[8];
  const long long t = b < total ? b / nb : 0;
  const int blk = (int)(b - t * nb), c = blk * kF8Block + lane16 * 8;
  load8_upto<__nv_bfloat16, true>(a.x + t * a.d, c, b < total ? a.d : 0, v);
  const uint32_t sb = f8_scale_bits(half_max(mag_max8(v)));
  if (b >= total) return;
  const uint2 q = codes8(v, f8_inverse(sb));
  for (int s = 0; s < a.k + a.own_rows; ++s) {
    const long long row = s < a.k ? a.pos[t * a.k + s] : (long long)a.T * a.k + t;
    if (c < a.d) *reinterpret_cast<uint2*>(a.codes + row * a.d + c) = q;
    if (lane16 == 0) a.scales[row * nb + blk] = __uint_as_float(sb);
  }
}

template <typename T>
cudaError_t launch_quant_t(const F8QuantArgs& a, bool tiles, cudaStream_t st) {
  const size_t es = sizeof(T);
  const bool vec = a.cols % 8 == 0 && (a.ldx * es) % 16 == 0 && a.ldq % 8 == 0 &&
                   ((uintptr_t)a.x & 15) == 0 && ((uintptr_t)a.codes & 7) == 0;
  if (tiles) {
    const long long n = (long long)a.count * f8_blocks(a.rows) * f8_blocks(a.cols);
    return vec ? launch_pdl(quant_tiles_kernel<T, true>, dim3((unsigned)n), kQuantThreads, 0, st, a)
               : launch_pdl(quant_tiles_kernel<T, false>, dim3((unsigned)n), kQuantThreads, 0, st, a);
  }
  const long long blocks = (long long)a.rows * f8_blocks(a.cols);
  const long long per = (long long)(kQuantThreads / 16) * kQuantUnroll;
  const long long most = (long long)tc_sm_count() * 8;
  // small calls: one block per half warp, spread over the SMs
  long long grid = (blocks + kQuantThreads / 16 - 1) / (kQuantThreads / 16);
  if (grid > most) grid = (blocks + per - 1) / per;
  if (grid > most) grid = most;
  return vec ? launch_pdl(quant_rows_kernel<T, true>, dim3((unsigned)grid), kQuantThreads, 0, st, a)
             : launch_pdl(quant_rows_kernel<T, false>, dim3((unsigned)grid), kQuantThreads, 0, st, a);
}

}  // namespace

cudaError_t launch_f8_quant(const F8QuantArgs& a, bool bf16, bool tiles, cudaStream_t st) {
  if (!tiles) {
    F8QuantArgs b = a;  // row blocks do not cross matrices: one tall matrix
    b.rows = a.rows * a.count;
    b.count = 1;
    return bf16 ? launch_quant_t<__nv_bfloat16>(b, false, st) : launch_quant_t<float>(b, false, st);
  }
  return bf16 ? launch_quant_t<__nv_bfloat16>(a, true, st) : launch_quant_t<float>(a, true, st);
}

cudaError_t launch_f8_pack(const F8PackArgs& a, cudaStream_t st) {
  const long long blocks = (long long)a.T * f8_blocks(a.d);
  const int per = kQuantThreads / 16;
  return launch_pdl(quant_pack_kernel, dim3((unsigned)((blocks + per - 1) / per)), kQuantThreads, 0,
                    st, a);
}

}  // namespace moe
