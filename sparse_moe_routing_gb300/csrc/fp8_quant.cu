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
// All are bound by HBM: bytes in plus one byte per value out. Measured:
// 14336 x 4096 bf16 in 128 x 128 blocks 28.0 us (6.3 TB/s), 4097 x 4096 fp32 rows
// 14.9 us (5.7 TB/s), 8 x 2048 1.9 us (launch).
#include "fp8_common.cuh"
#include "kernels.h"

namespace moe {
namespace {

// Eight consecutive values of a row as they lie in memory, zeros past its end.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 raw;
  template <bool VEC>
  __device__ __forceinline__ void load(const __nv_bfloat16* row, int c, int cols) {
    raw = make_uint4(0u, 0u, 0u, 0u);
    if (VEC) {
      if (c < cols) raw = ldg_stream(row + c);
    } else {
      uint32_t w[4] = {};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < cols)
          w[j >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(row)[c + j] << (16 * (j & 1));
      raw = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    Chunk<__nv_bfloat16>::unpack(raw, v);
  }
  // Largest magnitude's bits: those of a bf16 number order like its value too,
  // two at a time.
  __device__ __forceinline__ uint32_t mag() const {
    constexpr uint32_t kAbs = 0x7FFF7FFFu;
    const uint32_t m = __vmaxu2(__vmaxu2(raw.x & kAbs, raw.y & kAbs), __vmaxu2(raw.z & kAbs, raw.w & kAbs));
    return max(m << 16, m & 0xFFFF0000u);
  }
};
template <>
struct Eight<float> {
  uint4 raw[2];
  template <bool VEC>
  __device__ __forceinline__ void load(const float* row, int c, int cols) {
    raw[0] = raw[1] = make_uint4(0u, 0u, 0u, 0u);
    if (VEC) {
      if (c < cols) {
        raw[0] = ldg_stream(row + c);
        raw[1] = ldg_stream(row + c + 4);
      }
    } else {
      uint32_t w[8] = {};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < cols) w[j] = __float_as_uint(row[c + j]);
      raw[0] = make_uint4(w[0], w[1], w[2], w[3]);
      raw[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    Chunk<float>::unpack(raw[0], v);
    Chunk<float>::unpack(raw[1], v + 4);
  }
  __device__ __forceinline__ uint32_t mag() const {
    constexpr uint32_t kAbs = 0x7FFFFFFFu;
    return max(max(max(raw[0].x & kAbs, raw[0].y & kAbs), max(raw[0].z & kAbs, raw[0].w & kAbs)),
               max(max(raw[1].x & kAbs, raw[1].y & kAbs), max(raw[1].z & kAbs, raw[1].w & kAbs)));
  }
};

// Maximum over the 16 lanes of a half warp.
__device__ __forceinline__ uint32_t half_max(uint32_t m) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}
template <typename T>
__device__ __forceinline__ uint2 codes8(const Eight<T>& e, float inv) {
  float v[8];
  e.values(v);
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

// UNROLL blocks per half warp, all in flight at once. One pass per CTA: the
// hardware hands CTAs out as others end (a grid of eight per SM that walked on
// left the last of 1.7 rounds half empty: 17.5 us for 4097 x 4096 fp32).
template <typename T, bool VEC, int UNROLL>
__global__ void __launch_bounds__(kQuantThreads) quant_rows_kernel(F8QuantArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int kHalves = kQuantThreads / 16;
  const int nb = f8_blocks(a.cols);
  const long long total = (long long)a.rows * nb;
  const int lane16 = threadIdx.x & 15;
  const long long b0 = (long long)blockIdx.x * (kHalves * UNROLL) + (threadIdx.x >> 4);
  Eight<T> v[UNROLL];
  long long row[UNROLL];
  int blk[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const long long b = b0 + u * kHalves;
    const bool in = b < total;
    row[u] = in ? (total <= 0x7FFFFFFF ? (long long)((int)b / nb) : b / nb) : -1;
    blk[u] = in ? (int)(b - row[u] * nb) : 0;
    const T* src = static_cast<const T*>(a.x) + (in ? row[u] : 0) * a.ldx;
    v[u].template load<VEC>(src, blk[u] * kF8Block + lane16 * 8, in ? a.cols : 0);
  }
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const uint32_t sb = f8_scale_bits(half_max(v[u].mag()));
    if (row[u] < 0) continue;
    store_codes8<VEC>(a.codes + row[u] * a.ldq, blk[u] * kF8Block + lane16 * 8, a.cols,
                      codes8(v[u], f8_inverse(sb)));
    if (lane16 == 0) a.scales[row[u] * nb + blk[u]] = __uint_as_float(sb);
  }
}

// One 128 x 128 block per CTA: 256 threads, 16 per row, 8 row groups of 16.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kQuantThreads) quant_tiles_kernel(F8QuantArgs a) {
  __shared__ uint32_t s_max[kQuantThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int nb = f8_blocks(a.cols), nr = f8_blocks(a.rows);
  const int tile = blockIdx.x;
  const int cb = tile % nb, rest = tile / nb;
  const int rb = rest % nr;
  const long long mat = rest / nr;
  const int r0 = rb * kF8Block + (threadIdx.x >> 4), c = cb * kF8Block + (threadIdx.x & 15) * 8;
  const T* x = static_cast<const T*>(a.x) + mat * (long long)a.rows * a.ldx;
  uint8_t* codes = a.codes + mat * (long long)a.rows * a.ldq;
  Eight<T> v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 16 * i;
    v[i].template load<VEC>(x + (long long)min(r, a.rows - 1) * a.ldx, c, r < a.rows ? a.cols : 0);
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, v[i].mag());
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
  Eight<__nv_bfloat16> v;
  const long long t = b < total ? b / nb : 0;
  const int blk = (int)(b - t * nb), c = blk * kF8Block + lane16 * 8;
  v.load<true>(a.x + t * a.d, c, b < total ? a.d : 0);
  const uint32_t sb = f8_scale_bits(half_max(v.mag()));
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
  // one block per half warp until every SM has eight CTAs of them, then four
  constexpr int kHalves = kQuantThreads / 16;
  const bool one = blocks <= (long long)tc_sm_count() * 8 * kHalves;
  const long long per = one ? kHalves : kHalves * 4;
  const dim3 grid((unsigned)((blocks + per - 1) / per));
  if (one)
    return vec ? launch_pdl(quant_rows_kernel<T, true, 1>, grid, kQuantThreads, 0, st, a)
               : launch_pdl(quant_rows_kernel<T, false, 1>, grid, kQuantThreads, 0, st, a);
  return vec ? launch_pdl(quant_rows_kernel<T, true, 4>, grid, kQuantThreads, 0, st, a)
             : launch_pdl(quant_rows_kernel<T, false, 4>, grid, kQuantThreads, 0, st, a);
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
