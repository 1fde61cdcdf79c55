// 8-bit integer products for up to eight rows: the weights' bytes, streamed
// through mma.sync (s8 x s8 -> s32).
//
// m16n8k32 takes 16 weight rows as its m side and the rows of A as its n side. A
// contraction does not care in which order k is visited as long as both operands
// agree, so a lane's fragment registers are 16-byte pieces of the rows as they
// lie in memory: no conversion, no shuffles, no shared memory before the end.
// The gated form pairs 8 gate and 8 up rows in one m16 tile, so that a lane
// holds both sums of an output.
//
// Bound by the stream: HBM brings an SM some 23 bytes a cycle. This GPU runs the
// instruction at dp4a's rate (16 cycles an SM for 512 weight bytes, measured
// 150 TOP/s for either), 32 bytes a cycle at n = 8: enough for eight rows, not
// for sixteen.
//
// A CTA's eight warps are tiles x slices of k (ks of them), whose sums are added
// in int32 through shared memory: any order gives the same bits.
#include "i8_common.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kUnit = 64;    // k of one 16-byte piece per lane quad
constexpr int kUnroll = 4;   // units in flight

__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                       uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <bool GATED>
__global__ void __launch_bounds__(kWarps * 32) i8_few_kernel(I8FewArgs a) {
  __shared__ int s_sum[kWarps][4][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const int per = kWarps / a.ks;  // tiles of this CTA
  const int slice = warp % a.ks;
  const long long tile0 = (long long)blockIdx.x * per, tile = tile0 + warp / a.ks;
  // rows of the m16 tile: consecutive columns of the result, or 8 of gate and up
  const long long n0 = GATED ? tile * 8 + g : tile * 16 + g;
  const bool in0 = n0 < a.N, in1 = GATED ? in0 : n0 + 8 < a.N;
  const uint8_t* r0 = a.b0 + (in0 ? n0 : 0) * a.ldb;
  const uint8_t* r1 = GATED ? a.b1 + (in0 ? n0 : 0) * a.ldb : a.b0 + (in1 ? n0 + 8 : 0) * a.ldb;
  const uint8_t* ra = a.a + (g < a.M ? g : 0) * a.lda;
  const int units = (a.K + kUnit - 1) / kUnit;
  const int u0 = (int)((long long)slice * units / a.ks), u1 = (int)((long long)(slice + 1) * units / a.ks);
  const int K0 = in0 ? a.K : 0, K1 = in1 ? a.K : 0, KA = g < a.M ? a.K : 0;
  int d[2][4] = {};
  pdl_wait();
  pdl_trigger();
  int u = u0;
  // whole units
  const int full = min(u1, a.K / kUnit);
  for (; u + kUnroll <= full; u += kUnroll) {
    uint4 w0[kUnroll], w1[kUnroll], x[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int k = (u + i) * kUnit + q * 16;
      w0[i] = ldg_stream(r0 + k);
      w1[i] = ldg_stream(r1 + k);
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int k = (u + i) * kUnit + q * 16;
      x[i] = KA ? *reinterpret_cast<const uint4*>(ra + k) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      mma_s8(d[0], w0[i].x, w1[i].x, w0[i].y, w1[i].y, x[i].x, x[i].y);
      mma_s8(d[1], w0[i].z, w1[i].z, w0[i].w, w1[i].w, x[i].z, x[i].w);
    }
  }
  // what is left, and the last, cut unit
  for (; u < u1; ++u) {
    const int k = u * kUnit + q * 16;
    const uint4 w0 = i8_load16(r0, k, K0), w1 = i8_load16(r1, k, K1), x = i8_load16(ra, k, KA);
    mma_s8(d[0], w0.x, w1.x, w0.y, w1.y, x.x, x.y);
    mma_s8(d[1], w0.z, w1.z, w0.w, w1.w, x.z, x.w);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) s_sum[warp][j][lane] = d[0][j] + d[1][j];
  __syncthreads();
  // a lane's registers j: row g (j < 2) or g + 8 of the tile, row 2 q + j % 2 of A
  constexpr int kCols = GATED ? 8 : 16;
  const int outs = per * kCols * a.M;
  for (int o = threadIdx.x; o < outs; o += kWarps * 32) {
    const int c = o % kCols, t = o / kCols % per, m = o / (kCols * per);
    const long long n = (tile0 + t) * kCols + c;
    if (n >= a.N) continue;
    const int at = (c & 7) * 4 + (m >> 1), j = (m & 1) + (!GATED && c >= 8 ? 2 : 0);
    int s0 = 0, s1 = 0;
    for (int z = 0; z < a.ks; ++z) {
      s0 += s_sum[t * a.ks + z][j][at];
      if (GATED) s1 += s_sum[t * a.ks + z][j + 2][at];
    }
    const float sa = a.a_scale[m];
    float v = i8_value(s0, sa, a.b_scale0[n]);
    if (GATED) v = siluf_(v) * i8_value(s1, sa, a.b_scale1[n]);
    i8_store(a.out, m * a.ldo + n, a.out_bf16, v);
  }
}

}  // namespace

cudaError_t launch_i8_few(I8FewArgs a, bool gated, cudaStream_t st) {
  const int cols = gated ? 8 : 16;
  const long long tiles = ((long long)a.N + cols - 1) / cols;
  const int units = (a.K + kUnit - 1) / kUnit;
  // slices of k: until the warps fill the SMs three CTAs deep, four units each at least
  a.ks = 1;
  while (a.ks < kWarps && units >= 2 * a.ks * kUnroll && tiles * a.ks < 24ll * tc_sm_count()) a.ks *= 2;
  const long long per = kWarps / a.ks;
  const dim3 grid((unsigned)((tiles + per - 1) / per));
  return gated ? launch_pdl(i8_few_kernel<true>, grid, kWarps * 32, 0, st, a)
               : launch_pdl(i8_few_kernel<false>, grid, kWarps * 32, 0, st, a);
}

}  // namespace moe
