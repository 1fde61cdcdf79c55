// 8-bit integer products for up to eight rows: the weights' bytes, streamed past
// the rows of A.
//
// A warp takes tiles of 16 weight rows, a lane 16-byte pieces of two of them (rows
// g and g + 8, k 16 q of every 64, lane = 4 g + q) as they lie in memory: no
// conversion, no shared memory before the end. Gated, the 16 rows are 8 of gate
// and the same 8 of up, so that a lane holds both sums of an output.
//
//  * one or two rows: dp4a, the lane's pieces with the same piece of each row of
//    A; the four lanes of a row add up at the end;
//  * more: mma.sync m16n8k32 (s8 x s8 -> s32), for which the pieces are the
//    fragments (a contraction does not care in which order k is visited as long as
//    both operands agree).
//
// Bound by the stream: HBM brings an SM some 23 bytes a cycle. This GPU runs
// m16n8k32 at dp4a's rate (150 TOP/s for either): 32 bytes a cycle at n = 8 however
// many of the eight rows there are, which one or two on dp4a undercut (us, dp4a /
// mma.sync: 1 x 5632 x 2048 4.5 / 5.4, 2 x 4096 x 14336 12.4 / 13.5, but four rows of
// it 19.4 / 13.5: dp4a loads every row of A for every lane).
//
// Measured, weights rotated beyond L2: 1 x 5632 x 2048 4.5 us, 8 x 4096 x 14336 13.3
// (4.4 TB/s), gated 8 x 14336 x 4096 21.0 us (5.6 TB/s), 8 x 57344 x 8192 79 us (6.0).
//
// The warps of a CTA are tiles x slices of k (ks of them), whose sums are added
// in int32 through shared memory: any order gives the same bits.
#include "i8_common.cuh"

namespace moe {
namespace {

constexpr int kUnit = 64;  // k of one 16-byte piece per lane quad

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                       uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ int dot16(const uint4& a, const uint4& b, int c) {
  c = __dp4a((int)a.x, (int)b.x, c);
  c = __dp4a((int)a.y, (int)b.y, c);
  c = __dp4a((int)a.z, (int)b.z, c);
  return __dp4a((int)a.w, (int)b.w, c);
}

// The sums of a lane's two weight rows.
template <int ROWS>
struct Sums {  // dp4a: by row of A
  int s[2][ROWS] = {};
  const uint8_t* x[ROWS];
  __device__ __forceinline__ void start(const I8FewArgs& a, int) {
#pragma unroll
    for (int m = 0; m < ROWS; ++m) x[m] = a.a + min(m, a.M - 1) * a.lda;
  }
  struct Piece {
    uint4 v[ROWS];
  };
  __device__ __forceinline__ void load(Piece& p, int k) const {
#pragma unroll
    for (int m = 0; m < ROWS; ++m) p.v[m] = *reinterpret_cast<const uint4*>(x[m] + k);
  }
  __device__ __forceinline__ void load_end(Piece& p, int k, int K) const {
#pragma unroll
    for (int m = 0; m < ROWS; ++m) p.v[m] = i8_load16(x[m], k, K);
  }
  __device__ __forceinline__ void add(const uint4& w0, const uint4& w1, const Piece& p) {
#pragma unroll
    for (int m = 0; m < ROWS; ++m) {
      s[0][m] = dot16(w0, p.v[m], s[0][m]);
      s[1][m] = dot16(w1, p.v[m], s[1][m]);
    }
  }
  // into [16 weight rows][8 rows of A]
  __device__ __forceinline__ void out(int (*to)[9], int lane) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int m = 0; m < ROWS; ++m) {
        int v = s[h][m];
        v += __shfl_xor_sync(0xffffffffu, v, 1);
        v += __shfl_xor_sync(0xffffffffu, v, 2);
        if ((lane & 3) == 0) to[(lane >> 2) + 8 * h][m] = v;
      }
  }
};
template <>
struct Sums<8> {  // mma.sync: two chains
  int d[2][4] = {};
  const uint8_t* x;
  bool in;
  __device__ __forceinline__ void start(const I8FewArgs& a, int lane) {
    in = (lane >> 2) < a.M;
    x = a.a + (in ? lane >> 2 : 0) * a.lda;
  }
  struct Piece {
    uint4 v;
  };
  __device__ __forceinline__ void load(Piece& p, int k) const {
    p.v = in ? *reinterpret_cast<const uint4*>(x + k) : make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void load_end(Piece& p, int k, int K) const { p.v = i8_load16(x, k, in ? K : 0); }
  __device__ __forceinline__ void add(const uint4& w0, const uint4& w1, const Piece& p) {
    mma_s8(d[0], w0.x, w1.x, w0.y, w1.y, p.v.x, p.v.y);
    mma_s8(d[1], w0.z, w1.z, w0.w, w1.w, p.v.z, p.v.w);
  }
  __device__ __forceinline__ void out(int (*to)[9], int lane) {
#pragma unroll
    for (int j = 0; j < 4; ++j) to[(lane >> 2) + (j & 2) * 4][2 * (lane & 3) + (j & 1)] = d[0][j] + d[1][j];
  }
};

template <bool GATED, int ROWS, int WARPS, int UNROLL>
__global__ void __launch_bounds__(WARPS * 32) i8_few_kernel(I8FewArgs a) {
  __shared__ int s_sum[WARPS][16][9];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const int per = WARPS / a.ks;  // tiles of this CTA
  const int slice = warp % a.ks;
  const long long tile0 = (long long)blockIdx.x * per, tile = tile0 + warp / a.ks;
  // rows of the tile: consecutive columns of the result, or 8 of gate and up; a row
  // past the end stands for row 0, and its sums are not stored
  const long long n0 = GATED ? tile * 8 + g : tile * 16 + g;
  const bool in0 = n0 < a.N, in1 = GATED ? in0 : n0 + 8 < a.N;
  const uint8_t* r0 = a.b0 + (in0 ? n0 : 0) * a.ldb;
  const uint8_t* r1 = GATED ? a.b1 + (in0 ? n0 : 0) * a.ldb : a.b0 + (in1 ? n0 + 8 : 0) * a.ldb;
  const int units = (a.K + kUnit - 1) / kUnit;
  const int u0 = (int)((long long)slice * units / a.ks), u1 = (int)((long long)(slice + 1) * units / a.ks);
  Sums<ROWS> sums;
  sums.start(a, lane);
  pdl_wait();
  pdl_trigger();
  int u = u0;
  const int full = min(u1, a.K / kUnit);  // whole units
  for (; u + UNROLL <= full; u += UNROLL) {
    uint4 w0[UNROLL], w1[UNROLL];
    typename Sums<ROWS>::Piece x[UNROLL];
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
      const int k = (u + i) * kUnit + q * 16;
      w0[i] = ldg_stream(r0 + k);
      w1[i] = ldg_stream(r1 + k);
    }
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) sums.load(x[i], (u + i) * kUnit + q * 16);
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) sums.add(w0[i], w1[i], x[i]);
  }
  // what is left, and the last, cut unit
  for (; u < u1; ++u) {
    const int k = u * kUnit + q * 16;
    const uint4 w0 = i8_load16(r0, k, a.K), w1 = i8_load16(r1, k, a.K);
    typename Sums<ROWS>::Piece x;
    sums.load_end(x, k, a.K);
    sums.add(w0, w1, x);
  }
  sums.out(s_sum[warp], lane);
  __syncthreads();
  constexpr int kCols = GATED ? 8 : 16;
  const int outs = per * kCols * a.M;
  for (int o = threadIdx.x; o < outs; o += WARPS * 32) {
    const int c = o % kCols, t = o / kCols % per, m = o / (kCols * per);
    const long long n = (tile0 + t) * kCols + c;
    if (n >= a.N) continue;
    const float sa = a.a_scale[m], b0 = a.b_scale0[n], b1 = GATED ? a.b_scale1[n] : 0.f;
    int s0 = 0, s1 = 0;
    for (int z = 0; z < a.ks; ++z) {
      s0 += s_sum[t * a.ks + z][c][m];
      if (GATED) s1 += s_sum[t * a.ks + z][c + 8][m];
    }
    float v = i8_value(s0, sa, b0);
    if (GATED) v = siluf_(v) * i8_value(s1, sa, b1);
    i8_store(a.out, m * a.ldo + n, a.out_bf16, v);
  }
}

template <bool GATED, int ROWS>
cudaError_t launch_t(I8FewArgs a, cudaStream_t st) {
  const int cols = GATED ? 8 : 16, sms = tc_sm_count();
  const long long tiles = ((long long)a.N + cols - 1) / cols;
  const int units = (a.K + kUnit - 1) / kUnit;
  // Slices of k, four units each at least, until there are 96 warps an SM (short
  // work evens out the last of it: 8 x 57344 x 8192 98.0 us with 24, 78.7 with 96);
  // sixteen warps a CTA where eight slices of every tile are less than 24 an SM
  // (8 x 4096 x 14336 17.0 -> 13.4 us; 8 x 14336 x 4096 gated, with more, 22.2 -> 24.2).
  const bool wide = tiles * 8 < 24 * sms && units >= 64;
  const int warps = wide ? 16 : 8;
  a.ks = 1;
  while (a.ks < warps && units >= 8 * a.ks && tiles * a.ks < 96 * sms) a.ks *= 2;
  const long long per = warps / a.ks;
  const dim3 grid((unsigned)((tiles + per - 1) / per));
  return wide ? launch_pdl(i8_few_kernel<GATED, ROWS, 16, 2>, grid, 512, 0, st, a)
              : launch_pdl(i8_few_kernel<GATED, ROWS, 8, 4>, grid, 256, 0, st, a);
}
template <bool GATED>
cudaError_t launch_rows_of(const I8FewArgs& a, cudaStream_t st) {
  if (a.M == 1) return launch_t<GATED, 1>(a, st);
  if (a.M == 2) return launch_t<GATED, 2>(a, st);
  return launch_t<GATED, 8>(a, st);
}

}  // namespace

cudaError_t launch_i8_few(const I8FewArgs& a, bool gated, cudaStream_t st) {
  return gated ? launch_rows_of<true>(a, st) : launch_rows_of<false>(a, st);
}

}  // namespace moe
