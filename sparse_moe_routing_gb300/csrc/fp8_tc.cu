// Products in 8-bit floating point on the fifth-generation tensor cores:
// D = sum over blocks of 128 k of sa[row][block] sb[col / 128][block] * (A B^T of
// that block), A with a scale per 1 x 128 and B with one per 128 x 128.
//
// One persistent CTA per SM. TMA brings 128 x 128 A and 256 x 128 B codes per
// step (128-byte swizzle, 4 stages of 48 KB); one thread issues the four
// tcgen05.mma (e4m3, fp32, K = 32) of a step into one of two 256-column TMEM
// buffers. The scales change with every block of 128 k, so a buffer holds one
// step's products only: eight epilogue warps read it back, multiply by the two
// scales and add into fp32 sums that stay in their registers (128 a thread),
// while the tensor core fills the other buffer.
//
// Three uses:
//  * gate/up: B = 128 gate and 128 up rows; the epilogue applies SwiGLU and
//    quantises h: a thread holds half of a row's 128 columns, the other half's
//    maximum comes through shared memory, and codes and scale go out in the
//    form that the down product reads;
//  * down: the routing weight (or the shared gate) applied, rows out in bf16;
//  * dense: one product, bf16 or fp32 out, k split over CTAs when there are
//    few tiles (fp32 partial sums; the part of a tile that ends last adds them
//    in split order).
#include <cuda.h>
#include <cudaTypedefs.h>

#include "fp8_common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace moe {
namespace {

using namespace tc;

constexpr int BM = 128, BN = 256, BK = 128;
constexpr int kStages = 4;
constexpr int kStageA = BM * BK, kStageB = BN * BK;
constexpr uint32_t kTmemCols = 512;
constexpr int kEpiWarps = 8;
// Three warpgroups: warp 0 the producer, warp 1 the MMA issuer (2 and 3 idle),
// warps 4-11 the epilogue. Launched with 168 registers a thread (64,512 in
// all); the first group hands registers to the epilogue, whose 128 fp32 sums
// and 32 values in flight do not fit 168: 128 x 64 + 256 x 216 = 63,488.
constexpr int kEpiWarp0 = 4;
constexpr int kThreads = 128 + 32 * kEpiWarps;

struct Smem {
  static constexpr size_t kA = 0;
  static constexpr size_t kB = kA + (size_t)kStages * kStageA;
  static constexpr size_t kMax = kB + (size_t)kStages * kStageB;  // [2][2][BM] row maxima
  static constexpr size_t kBars = kMax + 4 * BM * 4;
  static constexpr size_t kBytes = 1024 + kBars + (2 * kStages + 5) * 8 + 16;
};
static_assert(Smem::kBytes <= 227 * 1024, "shared memory plan exceeds 227 KB");

// kind::f8f6f4: fp32 accumulate, A and B e4m3, both K-major.
constexpr uint32_t kIdesc = (1u << 4) | ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);

__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(kIdesc), "r"(accumulate));
}

// Two fp32 sums in one 64-bit register: sum += v * s.
__device__ __forceinline__ void fma2(uint64_t& sum, uint32_t v0, uint32_t v1, uint64_t s) {
  asm("{\n .reg .b64 v;\n mov.b64 v, {%1, %2};\n fma.rn.f32x2 %0, v, %3, %0;\n}"
      : "+l"(sum)
      : "r"(v0), "r"(v1), "l"(s));
}
__device__ __forceinline__ uint64_t both(float s) {
  const uint32_t b = __float_as_uint(s);
  return (uint64_t)b << 32 | b;
}
__device__ __forceinline__ float lo(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

struct Item {
  int g, m, nt;     // group, row block in it, N tile
  int row0, rows;   // the group's rows in A
  int kb0, kb1;     // blocks of k
  int tile, split;  // dense: tile index and k split
  bool shared;
};

// Items walk bands of 8 row blocks N tile by N tile, so that the CTAs in
// flight share B tiles across the band's row blocks through L2.
constexpr int kBand = 8;

template <int MODE>
__device__ __forceinline__ Item item_at(const F8TcArgs& a, int t, int n_rb, int KB) {
  Item it;
  it.split = 0;
  it.kb0 = 0;
  it.kb1 = KB;
  if (MODE == kF8Dense && a.ksplit > 1) {
    it.split = t % a.ksplit;
    t /= a.ksplit;
    it.kb0 = it.split * KB / a.ksplit;
    it.kb1 = (it.split + 1) * KB / a.ksplit;
  }
  it.tile = t;
  const int span = kBand * a.n_tiles;
  const int band = t / span, rb0 = band * kBand;
  const int width = min(kBand, n_rb - rb0);
  const int w = t - band * span;
  const int rb = rb0 + w % width;
  it.nt = w / width;
  it.shared = false;
  if (MODE == kF8Dense) {
    it.g = 0;
    it.m = rb;
    it.row0 = 0;
    it.rows = a.rows;
  } else if (a.shared_only) {
    it.g = a.E;
    it.m = rb;
    it.row0 = a.P;
    it.rows = a.T;
    it.shared = true;
  } else {
    const int2 r = a.rowblocks[rb];
    it.g = r.x;
    it.m = r.y;
    it.shared = r.x >= a.E;
    it.row0 = it.shared ? a.P : a.offsets[r.x];
    it.rows = it.shared ? a.T : a.offsets[r.x + 1] - it.row0;
  }
  return it;
}

__device__ __forceinline__ void give_up(const F8TcArgs& a, volatile int* abort_flag) {
  *abort_flag = 1;
  report(a.ctrl, kDevTimeout, kSiteTcFp8);
}

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    f8_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB0,
                 const __grid_constant__ CUtensorMap tmB1, const __grid_constant__ CUtensorMap tmB2,
                 const __grid_constant__ CUtensorMap tmB3, const F8TcArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem + Smem::kA;
  uint8_t* sB = smem + Smem::kB;
  uint32_t* sMax = reinterpret_cast<uint32_t*>(smem + Smem::kMax);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Smem::kBars);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* xbar = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(xbar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], kEpiWarps);
    }
    mbar_init(xbar, kEpiWarps);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint64_t lim = a.wait_ns;
  pdl_wait();
  pdl_trigger();

  const int n_rb = MODE == kF8Dense ? (a.rows + BM - 1) / BM
                                    : (a.shared_only ? (a.T + BM - 1) / BM : *a.n_rowblocks);
  const int total = n_rb * a.n_tiles * (MODE == kF8Dense ? a.ksplit : 1);
  const int KB = (a.K + BK - 1) / BK;

  // Every role loop is run by its whole warp, so that each warp reaches the
  // closing CTA barrier converged; a wait's outcome is lane 0's.
  if (warp < kEpiWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 0) {
      // -------------------------------------------------------------- producer
      const uint32_t bytes = (uint32_t)a.arows * BK + kStageB;
      int stage = 0;
      uint32_t ph = 0;
      bool alive = true;
      for (int t = blockIdx.x; t < total && alive; t += gridDim.x) {
        const Item it = item_at<MODE>(a, t, n_rb, KB);
        const CUtensorMap* b0 = it.shared ? &tmB2 : &tmB0;
        const CUtensorMap* b1 = it.shared ? &tmB3 : &tmB1;
        const int arow = it.row0 + it.m * BM;
        const int brow = (MODE == kF8Dense || it.shared ? 0 : it.g * a.brows) +
                         it.nt * (MODE == kF8GateUp ? BN / 2 : BN);
        for (int kb = it.kb0; kb < it.kb1; ++kb) {
          bool ok = lane == 0 ? mbar_wait(&empty[stage], ph ^ 1u, lim) : true;
          ok = __shfl_sync(0xffffffffu, ok, 0) && !*abort_flag;
          if (!ok) {
            if (lane == 0) give_up(a, abort_flag);
            alive = false;
            break;
          }
          if (lane == 0) {
            uint64_t* bar = &full[stage];
            mbar_expect_tx(bar, bytes);
            tma_load_2d(sA + stage * kStageA, &tmA, bar, kb * BK, arow);
            tma_load_2d(sB + stage * kStageB, b0, bar, kb * BK, brow);
            if (MODE == kF8GateUp)
              tma_load_2d(sB + stage * kStageB + kStageB / 2, b1, bar, kb * BK, brow);
          }
          __syncwarp();
          if (++stage == kStages) {
            stage = 0;
            ph ^= 1u;
          }
        }
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      int stage = 0, acc = 0;
      uint32_t ph = 0, aph = 0;
      bool alive = true;
      if (a.stall) {
        // failure self-test: wait on a barrier that only this warp completes
        bool ok = lane == 0 ? mbar_wait(&tfull[0], 0u, lim) : true;
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) {
          if (lane == 0) give_up(a, abort_flag);
          alive = false;
        }
      }
      for (int t = blockIdx.x; t < total && alive; t += gridDim.x) {
        const Item it = item_at<MODE>(a, t, n_rb, KB);
        for (int kb = it.kb0; kb < it.kb1; ++kb) {
          bool ok = true;
          if (lane == 0) ok = mbar_wait(&tempty[acc], aph ^ 1u, lim) && mbar_wait(&full[stage], ph, lim);
          ok = __shfl_sync(0xffffffffu, ok, 0) && !*abort_flag;
          if (!ok) {
            if (lane == 0) give_up(a, abort_flag);
            alive = false;
            break;
          }
          tc_fence_after();
          if (lane == 0) {
            const uint32_t d = tmem_base + (uint32_t)(acc * BN);
            const uint32_t a_base = smem_u32(sA + stage * kStageA), b_base = smem_u32(sB + stage * kStageB);
  #pragma unroll
            for (int k = 0; k < BK / 32; ++k)
              mma_f8(d, sw128_desc(a_base + k * 32), sw128_desc(b_base + k * 32), k != 0 ? 1u : 0u);
            mma_commit(&empty[stage]);
            mma_commit(&tfull[acc]);
          }
          __syncwarp();
          if (++stage == kStages) {
            stage = 0;
            ph ^= 1u;
          }
          acc ^= 1;
          if (acc == 0) aph ^= 1u;
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    // -------------------------------------------------------------- epilogue
    const int q = warp & 3;             // TMEM lane quarter this warp may access
    const int half = (warp - kEpiWarp0) >> 2;  // half of the tile's columns
    const int r = q * 32 + lane;
    const uint32_t tq = tmem_base + ((uint32_t)(q * 32) << 16);
    int acc = 0;
    uint32_t aph = 0, xph = 0;
    bool alive = true;
    for (int t = blockIdx.x; t < total && alive; t += gridDim.x) {
      const Item it = item_at<MODE>(a, t, n_rb, KB);
      const int i = it.m * BM + r;  // row inside the group
      const bool valid = i < it.rows;
      // rows past the group's end take the scale zero: their sums are never
      // stored
      const float* sap = a.a_scale + (size_t)(it.row0 + (valid ? i : 0)) * a.a_blocks;
      // the scale rows of B: gate and up of N tile nt, or this half's 128 columns
      const int sb_row = MODE == kF8GateUp ? it.nt : min(2 * it.nt + half, a.b_blocks - 1);
      const size_t sb_at =
          ((MODE == kF8Dense || it.shared ? 0 : (size_t)it.g * a.b_blocks) + sb_row) * KB;
      const float* sb0 = (it.shared ? a.b_scale2 : a.b_scale0) + sb_at;
      const float* sb1 = (it.shared ? a.b_scale3 : a.b_scale1) + sb_at;
      uint64_t sum[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) sum[j] = 0;
      float sa = valid ? sap[it.kb0] : 0.f, s0 = __ldg(sb0 + it.kb0);
      float s1 = MODE == kF8GateUp ? __ldg(sb1 + it.kb0) : 0.f;
      for (int kb = it.kb0; kb < it.kb1; ++kb) {
        const uint64_t c0 = both(sa * s0), c1 = both(sa * s1);
        if (kb + 1 < it.kb1) {
          sa = valid ? sap[kb + 1] : 0.f;
          s0 = __ldg(sb0 + kb + 1);
          if (MODE == kF8GateUp) s1 = __ldg(sb1 + kb + 1);
        }
        bool ok = lane == 0 ? mbar_wait(&tfull[acc], aph, lim) : true;
        ok = __shfl_sync(0xffffffffu, ok, 0) && !*abort_flag;
        if (!ok) {
          if (lane == 0) give_up(a, abort_flag);
          alive = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int col = MODE == kF8GateUp ? (c >> 1) * 128 + half * 64 + (c & 1) * 32
                                            : half * 128 + c * 32;
          uint32_t v[32];
          tmem_ld32(tq + (uint32_t)(acc * BN + col), v);
          tmem_ld_wait();
          const uint64_t s = MODE == kF8GateUp && c >= 2 ? c1 : c0;
#pragma unroll
          for (int j = 0; j < 16; ++j) fma2(sum[c * 16 + j], v[2 * j], v[2 * j + 1], s);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[acc]);
        acc ^= 1;
        if (acc == 0) aph ^= 1u;
      }
      if (!alive) break;
      if (MODE == kF8GateUp) {
        // h = silu(gate) * up for this half's 64 columns, in place
        const int left = a.n_cols - it.nt * 128 - half * 64;  // valid columns (16s)
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float h0 = siluf_(lo(sum[j])) * lo(sum[32 + j]);
          const float h1 = siluf_(hi(sum[j])) * hi(sum[32 + j]);
          sum[j] = (uint64_t)__float_as_uint(h1) << 32 | __float_as_uint(h0);
          if (2 * j < left) m = max(m, max(f8_mag(h0), f8_mag(h1)));
        }
        uint32_t* mx = sMax + xph * 2 * BM;
        mx[half * BM + r] = m;
        __syncwarp();
        bool ok = true;
        if (lane == 0) {
          mbar_arrive(xbar);
          ok = mbar_wait(xbar, xph, lim);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) {
          if (lane == 0) give_up(a, abort_flag);
          break;
        }
        __syncwarp();
        const uint32_t sbits = f8_scale_bits(max(m, mx[(half ^ 1) * BM + r]));
        const float inv = f8_inverse(sbits);
        xph ^= 1u;
        if (valid) {
          const size_t row = (size_t)it.row0 + i;
          uint8_t* dst = static_cast<uint8_t*>(a.out) + row * a.ldo + it.nt * 128 + half * 64;
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            if (16 * v < left) {
              uint32_t w[4];
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                const uint64_t p = sum[8 * v + 2 * z], p2 = sum[8 * v + 2 * z + 1];
                w[z] = f8_pack4(lo(p) * inv, hi(p) * inv, lo(p2) * inv, hi(p2) * inv);
              }
              st_global_v4(dst + 16 * v, w[0], w[1], w[2], w[3]);
            }
          }
          if (half == 0) a.out_scale[row * a.out_blocks + it.nt] = __uint_as_float(sbits);
        }
      } else if (MODE == kF8Down) {
        if (valid) {
          const float al = it.shared ? a.s_shared[i] : a.alpha[a.perm[it.row0 + i]];
          const int col = it.nt * BN + half * 128;
          __nv_bfloat16* dst =
              static_cast<__nv_bfloat16*>(a.out) + ((size_t)it.row0 + i) * a.ldo + col;
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            if (col + 8 * v < a.n_cols) {
              uint32_t w[4];
#pragma unroll
              for (int z = 0; z < 4; ++z)
                w[z] = pack_bf16x2(al * lo(sum[4 * v + z]), al * hi(sum[4 * v + z]));
              st_global_v4(dst + 8 * v, w[0], w[1], w[2], w[3]);
            }
          }
        }
      } else {
        const int col = it.nt * BN + half * 128;
        bool write = true;
        if (a.ksplit > 1) {
          // this warp's 32 rows x 128 columns of the tile, fp32, columns in
          // fours: [split][tile][64 column groups][128 rows]
          const int tiles = n_rb * a.n_tiles;
          float4* mine = a.partial + (((size_t)it.split * tiles + it.tile) * 64 + half * 32) * BM + r;
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (valid)
              __stcg(mine + (size_t)j * BM, make_float4(lo(sum[2 * j]), hi(sum[2 * j]),
                                                        lo(sum[2 * j + 1]), hi(sum[2 * j + 1])));
          __threadfence();
          __syncwarp();
          unsigned prev = 0;
          unsigned* ctr = a.counters + it.tile * kEpiWarps + (warp - kEpiWarp0);
          if (lane == 0) prev = atomicAdd(ctr, 1u);
          prev = __shfl_sync(0xffffffffu, prev, 0);
          write = (int)prev == a.ksplit - 1;
          if (write) {
            if (lane == 0) *ctr = 0u;
            __threadfence();
#pragma unroll
            for (int j = 0; j < 64; ++j) sum[j] = 0;
            for (int s = 0; s < a.ksplit; ++s) {
              const float4* o = a.partial + (((size_t)s * tiles + it.tile) * 64 + half * 32) * BM + r;
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const float4 p = valid ? __ldcg(o + (size_t)j * BM) : make_float4(0.f, 0.f, 0.f, 0.f);
                const uint64_t one = both(1.f);
                fma2(sum[2 * j], __float_as_uint(p.x), __float_as_uint(p.y), one);
                fma2(sum[2 * j + 1], __float_as_uint(p.z), __float_as_uint(p.w), one);
              }
            }
          }
        }
        if (write && valid) {
          if (a.out_bf16) {
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + (size_t)i * a.ldo + col;
#pragma unroll
            for (int v = 0; v < 16; ++v) {
              if (a.out_vec && col + 8 * v + 8 <= a.n_cols) {
                uint32_t w[4];
#pragma unroll
                for (int z = 0; z < 4; ++z) w[z] = pack_bf16x2(lo(sum[4 * v + z]), hi(sum[4 * v + z]));
                st_global_v4(dst + 8 * v, w[0], w[1], w[2], w[3]);
              } else {
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                  const int c = 8 * v + 2 * z;
                  if (col + c < a.n_cols) dst[c] = __float2bfloat16_rn(lo(sum[4 * v + z]));
                  if (col + c + 1 < a.n_cols) dst[c + 1] = __float2bfloat16_rn(hi(sum[4 * v + z]));
                }
              }
            }
          } else {
            float* dst = static_cast<float*>(a.out) + (size_t)i * a.ldo + col;
#pragma unroll
            for (int v = 0; v < 32; ++v) {
              if (a.out_vec && col + 4 * v + 4 <= a.n_cols) {
                st_global_v4(dst + 4 * v, (uint32_t)sum[2 * v], (uint32_t)(sum[2 * v] >> 32),
                             (uint32_t)sum[2 * v + 1], (uint32_t)(sum[2 * v + 1] >> 32));
              } else {
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                  const int c = 4 * v + 2 * z;
                  if (col + c < a.n_cols) dst[c] = lo(sum[2 * v + z]);
                  if (col + c + 1 < a.n_cols) dst[c + 1] = hi(sum[2 * v + z]);
                }
              }
            }
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) {
    // let copies and MMAs already in flight land before the CTA exits
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 2000000ull) {
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(kTmemCols));
  }
}

template <int MODE>
cudaError_t launch_t(const F8TcMaps& m, const F8TcArgs& a, int max_items, cudaStream_t st) {
  static int attr[64] = {};
  cudaError_t e = ensure_smem_limit(f8_tc_kernel<MODE>, (int)Smem::kBytes, attr);
  if (e != cudaSuccess) return e;
  int grid = tc_sm_count();
  if (max_items < grid) grid = max_items < 1 ? 1 : max_items;
  return launch_pdl(f8_tc_kernel<MODE>, dim3(grid), kThreads, Smem::kBytes, st, m.A, m.B0, m.B1, m.B2,
                    m.B3, a);
}

}  // namespace

bool f8_make_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint64_t pitch,
                 uint32_t box_rows) {
  auto fn = tc_encode_fn();
  if (!fn || !base) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {pitch};
  cuuint32_t box[2] = {(cuuint32_t)BK, box_rows};
  cuuint32_t es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_f8_tc(int mode, const F8TcMaps& m, const F8TcArgs& a, int max_items,
                         cudaStream_t st) {
  if (mode == kF8GateUp) return launch_t<kF8GateUp>(m, a, max_items, st);
  if (mode == kF8Down) return launch_t<kF8Down>(m, a, max_items, st);
  if (mode == kF8Dense) return launch_t<kF8Dense>(m, a, max_items, st);
  return cudaErrorInvalidValue;
}

}  // namespace moe
