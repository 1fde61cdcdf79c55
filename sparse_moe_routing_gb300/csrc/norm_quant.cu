// Rows: root-mean-square norm with the residual's addition, and 8-bit output.
//
//   s = x + r,  t = s * gain,  f = 1 / sqrt(mean(s^2) + eps),  out = t * f
//
// and, in 8 bits, codes of t with a scale that takes the factor f:
//   integers  m = max(max |t|, 127 * 2^-126): code = rint(t * (127 / m)), scale = (m / 127) * f, one per row;
//   e4m3      p = the smallest power of two >= 2^-126 with max |t| / p <= 448: code = e4m3(t / p),
//             scale = p * f, one per 1 x 128 block.
// A row's factor is the same for all of its values, so that taking it into the
// scale changes nothing but the roundings: s, t and t * (127 / m) are rounded
// once each whatever order the squares are summed in (codes do not depend on
// it), and the largest magnitude needs no second pass behind the sum: one
// reduction serves both. The integer quantiser of plain rows is the same kernel
// without norm (f = 1, t = x).
//
// A row belongs to a group of threads (a warp where it is short and there are
// many, a CTA else) and stays in its registers: x and the residual are read
// once, everything is written once. Bound by HBM for many rows (8192 x 4096 bf16 +
// fp32 residual -> int8 61 us, 6.0 TB/s, -> e4m3 63; 14336 x 4096 bf16 quantised 27.5
// us, 6.4 TB/s), by latency for few (a load, one reduction, a store: 1 x 2048 2.2 us).
// Rows of more than 8192 columns with norm have one CTA an SM, whose barrier nothing
// covers (4096 x 14336 -> int8 131 us, 0.73 of HBM), and past 16384 spill registers as
// well (2048 x 28672 136 us; without a residual 68, 0.38).
//
// The squares are summed as they are and, eight at a time, in units of 2^13; a row whose
// sum overflows takes its mean from the second (a row of 32768 values of 6e18 sums to
// 2^140). Rows that do not overflow have the first sum's bits.
//
// Rows that are not finite: the norm of a row with an infinity or a NaN is NaN
// there and 0 or NaN elsewhere; an integer row gets the scale NaN and codes 0, an
// e4m3 block the scale NaN and NaN codes.
#include "fp8_common.cuh"
#include "kernels.h"

namespace moe {
namespace {

// Threads of a CTA at most: as many as keep a row's values in registers.
constexpr int max_threads(int ch) { return ch <= 2 ? 1024 : 512; }
constexpr int kWarpRows = 8;  // rows per CTA where a warp has one

// Plain loads: the residual may be the sum's own place.
__device__ __forceinline__ uint4 ld16(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// The eight values of a lane in piece `piece` of its row. VEC: eight
// consecutive columns, 16 lanes a block of 128. Otherwise lane + 32 j of a
// warp's 256 columns: accesses of a warp stay side by side whatever the row's
// start and length, and a block of 128 is the whole warp's four values.
template <bool VEC>
__device__ __forceinline__ int col_of(int unit, int lane, int j) {
  return VEC ? (unit * 32 + lane) * 8 + j : unit * 256 + j * 32 + lane;
}

template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = ld16(p); }
  __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
  // the largest magnitude's bits: those of a bf16 number order like its value too
  __device__ __forceinline__ uint32_t mag() const {
    constexpr uint32_t kAbs = 0x7FFF7FFFu;
    const uint32_t m = __vmaxu2(__vmaxu2(v.x & kAbs, v.y & kAbs), __vmaxu2(v.z & kAbs, v.w & kAbs));
    return max(m << 16, m & 0xFFFF0000u);
  }
  __device__ __forceinline__ void values(float (&o)[8]) const { Chunk<__nv_bfloat16>::unpack(v, o); }
};
template <>
struct Raw<float> {
  uint4 v[2];
  __device__ __forceinline__ void load(const float* p) {
    v[0] = ld16(p);
    v[1] = ld16(p + 4);
  }
  __device__ __forceinline__ void zero() { v[0] = v[1] = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ uint32_t mag() const {
    constexpr uint32_t kAbs = 0x7FFFFFFFu;
    return max(max(max(v[0].x & kAbs, v[0].y & kAbs), max(v[0].z & kAbs, v[0].w & kAbs)),
               max(max(v[1].x & kAbs, v[1].y & kAbs), max(v[1].z & kAbs, v[1].w & kAbs)));
  }
  __device__ __forceinline__ void values(float (&o)[8]) const {
    Chunk<float>::unpack(v[0], o);
    Chunk<float>::unpack(v[1], o + 4);
  }
};

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }

// Loads the CH pieces of a row into v (zeros past its end).
template <typename T, bool VEC, int CH>
__device__ __forceinline__ void load_row(const T* row, int unit0, int units, int lane, int cols,
                                         float (&v)[CH][8]) {
  if (VEC) {
    Raw<T> raw[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = col_of<true>(unit0 + c * units, lane, 0);
      if (col < cols) raw[c].load(row + col);
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (col_of<true>(unit0 + c * units, lane, 0) < cols) {
        raw[c].values(v[c]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c][j] = 0.f;
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int col = col_of<false>(unit0 + c * units, lane, j);
        v[c][j] = col < cols ? widen(row[col]) : 0.f;
      }
  }
}

template <bool VEC>
__device__ __forceinline__ void store_values(void* base, long long at, bool bf16, int unit, int lane,
                                             int cols, const float (&v)[8]) {
  if (VEC) {
    const int col = col_of<true>(unit, lane, 0);
    if (col >= cols) return;
    if (bf16) {
      tc::st_global_v4(static_cast<__nv_bfloat16*>(base) + at + col, pack_bf16x2(v[0], v[1]),
                       pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    } else {
      float* p = static_cast<float*>(base) + at + col;
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = col_of<false>(unit, lane, j);
      if (col >= cols) continue;
      if (bf16)
        static_cast<__nv_bfloat16*>(base)[at + col] = __float2bfloat16_rn(v[j]);
      else
        static_cast<float*>(base)[at + col] = v[j];
    }
  }
}

template <bool VEC>
__device__ __forceinline__ void store_codes(uint8_t* row, int unit, int lane, int cols, uint2 q) {
  if (VEC) {
    const int col = col_of<true>(unit, lane, 0);
    if (col < cols) *reinterpret_cast<uint2*>(row + col) = q;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = col_of<false>(unit, lane, j);
      if (col < cols) row[col] = (uint8_t)((j < 4 ? q.x : q.y) >> (8 * (j & 3)));
    }
  }
}

// rint(v * inv) of four values as bytes, |v * inv| <= 127 (1 + 2^-23): adding
// 1.5 * 2^23 rounds to a whole number, to nearest even, and leaves it in the low
// bits. The product is rounded by itself (no fma).
__device__ __forceinline__ uint32_t int8x4(const float* v, float inv) {
  uint32_t b[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) b[j] = __float_as_uint(__fadd_rn(__fmul_rn(v[j], inv), 12582912.f));
  return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
}

constexpr int kFewRows = 8;  // an SM: up to here a row has a CTA, whatever its length
// 32768 values are 4096 pieces, so that pieces of up to 2^128 sum to 2^127 at most
constexpr float kSquareUnit = 1.f / 8192.f;
constexpr float kLeastMax = 127.f * 1.17549435e-38f;  // 127 * 2^-126, an fp32 number

// TX: x's type. RES: 0 no residual, 1 fp32, 2 bf16. NORM: with the factor f (and
// gain, sum, values); else the integer quantiser alone. CH pieces of eight
// values a thread. A CTA has one row, or one per warp where a.warp_rows.
template <typename TX, int RES, bool NORM, bool VEC, int CH>
__global__ void __launch_bounds__(max_threads(CH)) rows_kernel(RowsArgs a) {
  __shared__ float s_sum[32];
  __shared__ uint32_t s_max[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int units = a.warp_rows ? 1 : blockDim.x >> 5;  // warps of a row
  const int unit0 = a.warp_rows ? 0 : warp;
  const long long row = a.warp_rows ? (long long)blockIdx.x * kWarpRows + warp : blockIdx.x;
  pdl_wait();
  pdl_trigger();
  if (row >= a.rows) return;  // (whole warps, and only where no barrier follows)

  float t[CH][8];
  load_row<TX, VEC, CH>(static_cast<const TX*>(a.x) + row * a.ldx, unit0, units, lane, a.cols, t);
  if (NORM && RES != 0) {
    float r[CH][8];
    if (RES == 1)
      load_row<float, VEC, CH>(static_cast<const float*>(a.residual) + row * a.ldr, unit0, units, lane, a.cols, r);
    else
      load_row<__nv_bfloat16, VEC, CH>(static_cast<const __nv_bfloat16*>(a.residual) + row * a.ldr, unit0, units,
                                       lane, a.cols, r);
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) t[c][j] += r[c][j];
  }
  float sum = 0.f, scaled = 0.f;
  if (NORM) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (a.sum) store_values<VEC>(a.sum, row * a.lds, a.sum_bf16, unit0 + c * units, lane, a.cols, t[c]);
      float q = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) q = fmaf(t[c][j], t[c][j], q);
      sum += q;
      scaled = fmaf(q, kSquareUnit, scaled);
    }
    if (a.gain) {
      float g[CH][8];
      if (a.gain_bf16)
        load_row<__nv_bfloat16, VEC, CH>(static_cast<const __nv_bfloat16*>(a.gain), unit0, units, lane, a.cols, g);
      else
        load_row<float, VEC, CH>(static_cast<const float*>(a.gain), unit0, units, lane, a.cols, g);
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) t[c][j] = __fmul_rn(t[c][j], g[c][j]);
    }
    sum = warp_sum(sum);
  }
  uint32_t mx = 0;
  if (a.kind == kRowsInt8) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) mx = max(mx, f8_mag(t[c][j]));
    mx = __reduce_max_sync(0xffffffffu, mx);
  }
  if (!a.warp_rows) {
    if (lane == 0) {
      s_sum[warp] = sum;
      s_max[warp] = mx;
    }
    __syncthreads();
    // warps' sums in warp order in every lane
    float ws = lane < units ? s_sum[lane] : 0.f;
    const uint32_t wm = lane < units ? s_max[lane] : 0u;
    if (NORM) sum = warp_sum(ws);
    mx = __reduce_max_sync(0xffffffffu, wm);
  }
  float f = 1.f;
  if (NORM) {
    float mean = sum / (float)a.cols;
    if (__float_as_uint(sum) == 0x7F800000u) {  // (the same in all of the row's threads)
      scaled = warp_sum(scaled);
      if (!a.warp_rows) {
        __syncthreads();  // every warp has read s_sum
        if (lane == 0) s_sum[warp] = scaled;
        __syncthreads();
        scaled = warp_sum(lane < units ? s_sum[lane] : 0.f);
      }
      mean = scaled / ((float)a.cols * kSquareUnit);
    }
    f = 1.f / sqrtf(mean + a.eps);
  }

  if (NORM && a.out) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = t[c][j] * f;
      store_values<VEC>(a.out, row * a.ldo, a.out_bf16, unit0 + c * units, lane, a.cols, y);
    }
  }
  if (a.kind == kRowsInt8) {
    const bool finite = mx < 0x7F800000u;
    const float m = fmaxf(__uint_as_float(mx), kLeastMax);
    const float inv = finite ? 127.f / m : 0.f;
    uint8_t* codes = a.codes + row * a.ldq;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const uint2 q = make_uint2(int8x4(t[c], inv), int8x4(t[c] + 4, inv));
      store_codes<VEC>(codes, unit0 + c * units, lane, a.cols, finite ? q : make_uint2(0u, 0u));
    }
    if (unit0 == 0 && lane == 0) a.scales[row] = finite ? (m / 127.f) * f : __uint_as_float(kF8NanScale);
  } else if (NORM && a.kind == kRowsE4m3) {
    const int nb = f8_blocks(a.cols);
    float* scales = a.scales + row * nb;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int unit = unit0 + c * units;
      // the largest magnitudes of the warp's two blocks: VEC by half warps,
      // else of values 0-3 and 4-7 over the warp
      uint32_t m[2] = {0u, 0u};
#pragma unroll
      for (int j = 0; j < 8; ++j) m[VEC ? 0 : j >> 2] = max(m[VEC ? 0 : j >> 2], f8_mag(t[c][j]));
      if (VEC) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m[0] = max(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
        m[1] = m[0];
      } else {
        m[0] = __reduce_max_sync(0xffffffffu, m[0]);
        m[1] = __reduce_max_sync(0xffffffffu, m[1]);
      }
      const uint32_t sb[2] = {f8_scale_bits(m[0]), f8_scale_bits(m[1])};
      const float i0 = f8_inverse(sb[0]), i1 = f8_inverse(sb[1]);
      store_codes<VEC>(a.codes + row * a.ldq, unit, lane, a.cols,
                       make_uint2(f8_pack4(t[c][0] * i0, t[c][1] * i0, t[c][2] * i0, t[c][3] * i0),
                                  f8_pack4(t[c][4] * i1, t[c][5] * i1, t[c][6] * i1, t[c][7] * i1)));
      // one lane a block: lanes 0 and 16 (VEC), else lanes 0 and 1
      const int blk = 2 * unit + (VEC ? lane >> 4 : lane);
      if ((VEC ? (lane & 15) == 0 : lane < 2) && blk < nb)
        scales[blk] = __uint_as_float(VEC || lane == 0 ? sb[0] : sb[1]) * f;
    }
  }
}

// The integer quantiser of rows that are read in 16-byte pieces: these stay as they
// came until the scale is known (half the registers of bf16 rows' values), so that
// a thread has eight of them in flight.
template <typename TX, int CH>
__global__ void __launch_bounds__(512) quant_kernel(RowsArgs a) {
  __shared__ uint32_t s_max[16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int units = a.warp_rows ? 1 : blockDim.x >> 5;
  const int unit0 = a.warp_rows ? 0 : warp;
  const long long row = a.warp_rows ? (long long)blockIdx.x * kWarpRows + warp : blockIdx.x;
  pdl_wait();
  pdl_trigger();
  if (row >= a.rows) return;  // (whole warps, and only where no barrier follows)
  const TX* x = static_cast<const TX*>(a.x) + row * a.ldx;
  Raw<TX> raw[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = col_of<true>(unit0 + c * units, lane, 0);
    if (col < a.cols)
      raw[c].load(x + col);
    else
      raw[c].zero();
  }
  uint32_t mx = 0;
#pragma unroll
  for (int c = 0; c < CH; ++c) mx = max(mx, raw[c].mag());
  mx = __reduce_max_sync(0xffffffffu, mx);
  if (!a.warp_rows) {
    if (lane == 0) s_max[warp] = mx;
    __syncthreads();
    mx = __reduce_max_sync(0xffffffffu, lane < units ? s_max[lane] : 0u);
  }
  const bool finite = mx < 0x7F800000u;
  const float m = fmaxf(__uint_as_float(mx), kLeastMax);
  const float inv = finite ? 127.f / m : 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    float t[8];
    raw[c].values(t);
    const uint2 q = make_uint2(int8x4(t, inv), int8x4(t + 4, inv));
    store_codes<true>(a.codes + row * a.ldq, unit0 + c * units, lane, a.cols, finite ? q : make_uint2(0u, 0u));
  }
  if (unit0 == 0 && lane == 0) a.scales[row] = finite ? m / 127.f : __uint_as_float(kF8NanScale);
}

// Many rows of up to 1024 values are a warp's each (16384 x 1024 bf16 9.8 us, a CTA
// 17.2), others a CTA's. Eight pieces a thread
// past 2048 values, one where rows are few: 14336 x 4096 bf16 27.5 us (four: 28.8,
// two in the general kernel above: 36.7), 4096 x 14336 28.6 (four: 35.8 there); a warp
// for 2048 fp32 values lost (15.3 against 13.7).
template <typename TX>
cudaError_t launch_quant(RowsArgs a, cudaStream_t st) {
  const int units = (a.cols + 255) / 256;
  const bool few = a.rows <= kFewRows * tc_sm_count();
  a.warp_rows = units <= 4 && !few;
  const dim3 grid((unsigned)(a.warp_rows ? ((long long)a.rows + kWarpRows - 1) / kWarpRows : a.rows));
  const int ch = a.warp_rows ? units : few && units <= 16 ? 1 : units <= 8 ? 4 : 8;
  const int threads = a.warp_rows ? 32 * kWarpRows : 32 * ((units + ch - 1) / ch);
  if (ch == 1) return launch_pdl(quant_kernel<TX, 1>, grid, threads, 0, st, a);
  if (ch == 2) return launch_pdl(quant_kernel<TX, 2>, grid, threads, 0, st, a);
  if (ch <= 4) return launch_pdl(quant_kernel<TX, 4>, grid, threads, 0, st, a);
  return launch_pdl(quant_kernel<TX, 8>, grid, threads, 0, st, a);
}

template <typename TX, int RES, bool NORM, bool VEC>
cudaError_t launch_ch(RowsArgs a, cudaStream_t st) {
  const int units = (a.cols + 255) / 256;
  const bool few = a.rows <= kFewRows * tc_sm_count();
  // A warp a row up to 512 columns (to 1024: 8192 x 1024 22.1 against 19.5 us) where
  // rows are many (333 x 1001 5.8 against 2.2 us); else a CTA a row, with one piece a
  // thread where rows are few, two while a row fits a CTA that way.
  a.warp_rows = units <= 2 && !few;
  const int ch = a.warp_rows ? units : few && units <= 32 ? 1 : units <= 64 ? 2 : 8;
  const dim3 grid((unsigned)(a.warp_rows ? ((long long)a.rows + kWarpRows - 1) / kWarpRows : a.rows));
  const int threads = a.warp_rows ? 32 * kWarpRows : 32 * ((units + ch - 1) / ch);
  if (ch == 1) return launch_pdl(rows_kernel<TX, RES, NORM, VEC, 1>, grid, threads, 0, st, a);
  if (ch == 2) return launch_pdl(rows_kernel<TX, RES, NORM, VEC, 2>, grid, threads, 0, st, a);
  return launch_pdl(rows_kernel<TX, RES, NORM, VEC, 8>, grid, threads, 0, st, a);
}

template <typename TX, bool VEC>
cudaError_t launch_rows_t(const RowsArgs& a, cudaStream_t st) {
  if (!a.norm) return VEC ? launch_quant<TX>(a, st) : launch_ch<TX, 0, false, false>(a, st);
  if (!a.residual) return launch_ch<TX, 0, true, VEC>(a, st);
  return a.res_bf16 ? launch_ch<TX, 2, true, VEC>(a, st) : launch_ch<TX, 1, true, VEC>(a, st);
}

}  // namespace

cudaError_t launch_rows(const RowsArgs& a, cudaStream_t st) {
  const auto wide = [&](const void* p, long long ld, int bytes, int align) {
    return !p || (((uintptr_t)p & (align - 1)) == 0 && ld * bytes % align == 0);
  };
  const bool vec = a.cols % 8 == 0 && wide(a.x, a.ldx, a.x_bf16 ? 2 : 4, 16) &&
                   wide(a.residual, a.ldr, a.res_bf16 ? 2 : 4, 16) && wide(a.gain, 0, 1, 16) &&
                   wide(a.sum, a.lds, a.sum_bf16 ? 2 : 4, 16) && wide(a.out, a.ldo, a.out_bf16 ? 2 : 4, 16) &&
                   wide(a.codes, a.ldq, 1, 8);
  if (a.x_bf16) return vec ? launch_rows_t<__nv_bfloat16, true>(a, st) : launch_rows_t<__nv_bfloat16, false>(a, st);
  return vec ? launch_rows_t<float, true>(a, st) : launch_rows_t<float, false>(a, st);
}

}  // namespace moe
