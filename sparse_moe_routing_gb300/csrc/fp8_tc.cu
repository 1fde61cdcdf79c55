// Products in 8-bit floating point on the fifth-generation tensor cores:
// D = sum over blocks of 128 k of sa[row][block] sb[col / 128][block] * (A B^T of
// that block), A with a scale per 1 x 128 and B with one per 128 x 128.
//
// One persistent CTA per SM. TMA brings 128 x 128 A and 256 x 128 B codes per
// step (128-byte swizzle, 4 stages of 48 KB); a thread issues the four
// tcgen05.mma (e4m3, fp32, K = 32) of a step into one of two 256-column TMEM
// buffers. The scales change with every block of 128 k, so a buffer holds one
// step's products only: sixteen epilogue warps read it back, multiply by the two
// scales and add into fp32 sums that stay in their registers (64 a thread),
// while the tensor core fills the other buffer.
//
// What bounds it where HBM does not: the step. Its MMAs take 512 cycles, a
// step about 1,000: the read-back, the sums and the hand-overs between issuer
// and epilogue (issue slots 68 % busy, the tensor pipe 36-50 %). 8192 x 14336 x 4096
// 480-500 us (1.9-2.0 PFLOP/s), grouped gate/up of 8 wide experts at
// 2048 tokens 1.7 PFLOP/s; decode batches stream weights at 5.7 TB/s (gate/up,
// 64 tokens of the 256-expert shape). Tried and slower: two column halves with
// an issuer and two 128-column buffers each (504 us).
//
// Three uses:
//  * gate/up: B = 128 gate and 128 up rows; the epilogue applies SwiGLU and
//    quantises h: a thread holds 32 of a row's 128 columns, the others'
//    maxima come through shared memory, and codes and scale go out in the
//    form that the down product reads;
//  * down: the routing weight (or the shared gate) applied, rows out in fp32;
//  * dense: one product, bf16 or fp32 out, k split over CTAs when there are
//    few tiles (fp32 partial sums, which a second launch adds in split order).
//
// A thread's results are one row's, so that storing them as they lie would
// touch 32 rows an instruction; eight lanes first exchange 16-byte pieces, and
// an instruction then writes whole 128-byte lines of four rows.
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
constexpr int kEpiWarps = 16;
constexpr int kParts = kEpiWarps / 4;     // column parts of a tile, one per warp of a lane quarter
constexpr int kPartCols = BN / kParts;    // 64
// Warp 0 is the producer, warps 1 and 2 issue the MMAs, warp 3 brings the
// scales, warps 4-19 are the epilogue: four a scheduler, so that one warp's
// wait for TMEM is covered by the others' arithmetic (eight warps: 959 us where
// sixteen took 668 on the 8192 x 14336 x 4096 product). Launched with 96
// registers a thread (61,440 in all); the first warpgroup hands some to the
// epilogue, which holds 64 fp32 sums and 32 values in flight a thread:
// 128 x 64 + 512 x 104 = 61,440. (gate/up, at 96, spills one register: 4 bytes
// stored, 20 loaded.)
constexpr int kEpiWarp0 = 4;
constexpr int kThreads = 128 + 32 * kEpiWarps;

// Scales, kChunk steps at a time: A's [kChunks][kChunk][128 rows], then B's
// [kChunks][kChunk][2: gate, up | left, right half of the columns].
constexpr int kChunk = 4, kChunks = 8;

struct Smem {
  static constexpr size_t kA = 0;
  static constexpr size_t kB = kA + (size_t)kStages * kStageA;
  static constexpr size_t kMax = kB + (size_t)kStages * kStageB;  // [2][kParts][BM] row maxima
  static constexpr size_t kScale = kMax + 2 * kParts * BM * 4;
  static constexpr size_t kBars = kScale + kChunks * kChunk * (BM + 2) * 4;
  static constexpr size_t kBytes = 1024 + kBars + (2 * kStages + 2 * kChunks + 5) * 8 + 16;
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

// Asynchronous copy of one fp32 value to shared memory, or of zero.
__device__ __forceinline__ void copy4_async(float* dst, const float* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(valid ? 4 : 0)
               : "memory");
}
// Arrives on `bar` once this thread's copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// c[j] is piece j of this lane's row; afterwards c[i] is piece lane % 8 of row
// 8 (lane / 8) + i of the warp's 32.
__device__ __forceinline__ void exchange8(uint4 (&c)[8], int lane) {
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int a = 0; a < 8; ++a) {
      if (a & o) continue;
      const int b = a | o;
      uint4 send = up ? c[a] : c[b];
      send.x = __shfl_xor_sync(0xffffffffu, send.x, o);
      send.y = __shfl_xor_sync(0xffffffffu, send.y, o);
      send.z = __shfl_xor_sync(0xffffffffu, send.z, o);
      send.w = __shfl_xor_sync(0xffffffffu, send.w, o);
      if (up)
        c[a] = send;
      else
        c[b] = send;
    }
  }
}
__device__ __forceinline__ uint4 four_floats(const float* v) {
  return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                    __float_as_uint(v[3]));
}
__device__ __forceinline__ uint4 eight_bf16(const float* v) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}
// Stores the exchanged pieces: `at` the address of the lane's piece in the
// warp's first row, rows `pitch` elements apart of which `rows` exist, `left`
// columns from the lane's piece on; whole pieces where `vec`.
template <typename T>
__device__ __forceinline__ void store8(T* at, long long pitch, const uint4 (&c)[8], int rows, int left,
                                       bool vec, int lane) {
  constexpr int kPer = 16 / sizeof(T);
  const int r0 = lane & 24;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (r0 + i >= rows) break;
    T* dst = at + (r0 + i) * pitch;
    if (vec && left >= kPer) {
      st_global_v4(dst, c[i].x, c[i].y, c[i].z, c[i].w);
    } else {
      const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
#pragma unroll
      for (int z = 0; z < kPer; ++z) {
        if (z >= left) continue;
        if (sizeof(T) == 4)
          reinterpret_cast<uint32_t*>(dst)[z] = w[z & 3];
        else
          reinterpret_cast<uint16_t*>(dst)[z] = (uint16_t)(w[z >> 1] >> (16 * (z & 1)));
      }
    }
  }
}

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

// Waits of one thread and of a whole warp; a warp that gives up raises the flag.
__device__ __forceinline__ bool lane_wait(uint64_t* bar, uint32_t parity, const F8TcArgs& a,
                                          volatile int* abort_flag) {
  return f8_lane_wait(bar, parity, a.wait_ns, abort_flag);
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const F8TcArgs& a,
                                          volatile int* abort_flag) {
  const bool ok = __all_sync(0xffffffffu, lane_wait(bar, parity, a, abort_flag));
  if (!ok && (threadIdx.x & 31) == 0) give_up(a, abort_flag);
  return ok;
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
  float* sScale = reinterpret_cast<float*>(smem + Smem::kScale);
  float* sScaleB = sScale + kChunks * kChunk * BM;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Smem::kBars);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* cfull = tempty + 2;
  uint64_t* cempty = cfull + kChunks;
  uint64_t* xbar = cempty + kChunks;
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
    for (int b = 0; b < kChunks; ++b) {
      mbar_init(&cfull[b], 32);
      mbar_init(&cempty[b], kEpiWarps);
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
  pdl_wait();
  pdl_trigger();

  const int n_rb = MODE == kF8Dense ? (a.rows + BM - 1) / BM
                                    : (a.shared_only ? (a.T + BM - 1) / BM : *a.n_rowblocks);
  const int total = n_rb * a.n_tiles * (MODE == kF8Dense ? a.ksplit : 1);
  const int KB = (a.K + BK - 1) / BK;

  if (warp < kEpiWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    // The producer's and the issuer's loops are lane 0's alone: an issue waits
    // for room in the tensor core's short queue, and cycles between two issues
    // leave it idle.
    if (warp == 0) {
      // -------------------------------------------------------------- producer
      if (lane == 0) {
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
            if (!lane_wait(&empty[stage], ph ^ 1u, a, abort_flag)) {
              give_up(a, abort_flag);
              alive = false;
              break;
            }
            uint64_t* bar = &full[stage];
            mbar_expect_tx(bar, kStageA + kStageB);
            tma_load_2d(sA + stage * kStageA, &tmA, bar, kb * BK, arow);
            tma_load_2d(sB + stage * kStageB, b0, bar, kb * BK, brow);
            if (MODE == kF8GateUp)
              tma_load_2d(sB + stage * kStageB + kStageB / 2, b1, bar, kb * BK, brow);
            if (++stage == kStages) {
              stage = 0;
              ph ^= 1u;
            }
          }
        }
      }
      __syncwarp();
    } else if (warp <= 2) {
      // ----------------------------------------------------------- MMA issuers
      // Two, each with every second step and its TMEM buffer: issuing a step
      // takes its MMAs' 512 cycles, and the commits and the next step's waits
      // some 600 more, which one issuer would leave the tensor core idle.
      if (lane == 0) {
        const uint32_t me = warp - 1;
        // failure self-test: wait on a barrier that only this warp completes
        bool alive = !a.stall || lane_wait(&tfull[me], 0u, a, abort_flag);
        if (!alive) give_up(a, abort_flag);
        const uint32_t d = tmem_base + me * BN;
        uint32_t n = 0;  // steps so far
        for (int t = blockIdx.x; t < total && alive; t += gridDim.x) {
          const Item it = item_at<MODE>(a, t, n_rb, KB);
          for (int kb = it.kb0; kb < it.kb1; ++kb, ++n) {
            if ((n & 1u) != me) continue;
            const uint32_t stage = n % kStages;
            if (!lane_wait(&full[stage], n / kStages & 1u, a, abort_flag) ||
                !lane_wait(&tempty[me], (n >> 1 & 1u) ^ 1u, a, abort_flag)) {
              give_up(a, abort_flag);
              alive = false;
              break;
            }
            tc_fence_after();
            const uint64_t a_desc = sw128_desc(smem_u32(sA + stage * kStageA));
            const uint64_t b_desc = sw128_desc(smem_u32(sB + stage * kStageB));
#pragma unroll
            for (int k = 0; k < BK / 32; ++k)  // 32 bytes on: 2 in the descriptor
              mma_f8(d, a_desc + 2 * k, b_desc + 2 * k, k != 0 ? 1u : 0u);
            mma_commit(&tfull[me]);
            mma_commit(&empty[stage]);
          }
        }
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------------- scales
      // Four rows a lane, copied asynchronously up to kChunks chunks ahead of
      // the epilogue (loading a step's scales in the epilogue, one step ahead,
      // waited out the latency of L2 there: 2432 x 4096 x 4096 100 us against
      // 63 with constant scales).
      const int r0 = lane;
      int cb = 0;
      uint32_t cph = 0;
      bool alive = true;
      for (int t = blockIdx.x; t < total && alive; t += gridDim.x) {
        const Item it = item_at<MODE>(a, t, n_rb, KB);
        const float* sa[4];
        bool valid[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const int i = it.m * BM + r0 + 32 * h;  // rows past the group's end take zeros
          valid[h] = i < it.rows;
          sa[h] = a.a_scale + (size_t)(it.row0 + (valid[h] ? i : 0)) * a.a_blocks;
        }
        // the scale rows of B: gate and up of N tile nt, or two blocks of 128 columns
        const size_t g0 = MODE == kF8Dense || it.shared ? 0 : (size_t)it.g * a.b_blocks;
        const float* sb0 = (it.shared ? a.b_scale2 : a.b_scale0) +
                           (g0 + (MODE == kF8GateUp ? it.nt : 2 * it.nt)) * KB;
        const float* sb1 = MODE == kF8GateUp
                               ? (it.shared ? a.b_scale3 : a.b_scale1) + (g0 + it.nt) * KB
                               : (it.shared ? a.b_scale2 : a.b_scale0) +
                                     (g0 + min(2 * it.nt + 1, a.b_blocks - 1)) * KB;
        for (int k0 = it.kb0; k0 < it.kb1; k0 += kChunk) {
          if (!warp_wait(&cempty[cb], cph ^ 1u, a, abort_flag)) {
            alive = false;
            break;
          }
          const int n = min(kChunk, it.kb1 - k0);
#pragma unroll
          for (int j = 0; j < kChunk; ++j)
#pragma unroll
            for (int h = 0; h < 4; ++h)
              if (j < n)
                copy4_async(sScale + (cb * kChunk + j) * BM + r0 + 32 * h, sa[h] + k0 + j, valid[h]);
          if (r0 < 2 * n)
            copy4_async(sScaleB + cb * kChunk * 2 + r0, ((r0 & 1) ? sb1 : sb0) + k0 + (r0 >> 1), true);
          copies_arrive(&cfull[cb]);
          if (++cb == kChunks) {
            cb = 0;
            cph ^= 1u;
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    // -------------------------------------------------------------- epilogue
    const int q = warp & 3;             // TMEM lane quarter this warp may access
    const int part = (warp - kEpiWarp0) >> 2;  // this warp's columns of the tile
    const int r = q * 32 + lane;
    const uint32_t tq = tmem_base + ((uint32_t)(q * 32) << 16);
    int acc = 0, cb = 0;
    uint32_t aph = 0, cph = 0, xph = 0;
    bool alive = true;
    Item next = item_at<MODE>(a, min((int)blockIdx.x, total - 1), n_rb, KB);
    for (int t = blockIdx.x; t < total && alive; t += gridDim.x) {
      const Item it = next;
      if (t + (int)gridDim.x < total) next = item_at<MODE>(a, t + gridDim.x, n_rb, KB);
      const int i = it.m * BM + r;  // row inside the group
      const bool valid = i < it.rows;
      float al = 0.f;  // down: the row's weight, in flight during the steps
      if (MODE == kF8Down && valid) al = it.shared ? a.s_shared[i] : a.alpha[a.perm[it.row0 + i]];
      float sum[kPartCols];
#pragma unroll
      for (int j = 0; j < kPartCols; ++j) sum[j] = 0.f;
      for (int kb = it.kb0; kb < it.kb1; ++kb) {
        const int step = (kb - it.kb0) & (kChunk - 1);
        if (step == 0) {
          if (!warp_wait(&cfull[cb], cph, a, abort_flag)) {
            alive = false;
            break;
          }
        }
        const float sa = sScale[(cb * kChunk + step) * BM + r];
        const float* sb = sScaleB + (cb * kChunk + step) * 2;
        const float c0 = sa * sb[MODE == kF8GateUp ? 0 : part >> 1];
        const float c1 = MODE == kF8GateUp ? sa * sb[1] : c0;
        if (!warp_wait(&tfull[acc], aph, a, abort_flag)) {
          alive = false;
          break;
        }
        tc_fence_after();
        uint32_t v[2][16];
        auto col = [&](int c) {
          return tq + (uint32_t)(acc * BN + (MODE == kF8GateUp ? (c >> 1) * 128 + part * 32 + (c & 1) * 16
                                                               : part * kPartCols + c * 16));
        };
        tmem_ld16(col(0), v[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          tmem_ld_wait();
          // The read's registers hold their values from here on: the compiler
          // sees this as their definition and moves no use above the wait.
#pragma unroll
          for (int j = 0; j < 16; ++j) asm volatile("" : "+r"(v[c & 1][j]));
          if (c < 3) tmem_ld16(col(c + 1), v[(c + 1) & 1]);
          const float s = c >= 2 ? c1 : c0;
#pragma unroll
          for (int j = 0; j < 16; ++j)
            sum[c * 16 + j] = fmaf(__uint_as_float(v[c & 1][j]), s, sum[c * 16 + j]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[acc]);
        acc ^= 1;
        if (acc == 0) aph ^= 1u;
        if (step == kChunk - 1 || kb == it.kb1 - 1) {
          if (lane == 0) mbar_arrive(&cempty[cb]);
          if (++cb == kChunks) {
            cb = 0;
            cph ^= 1u;
          }
        }
      }
      if (!alive) break;
      if (MODE == kF8GateUp) {
        // h = silu(gate) * up for this warp's 32 columns, in place
        const int left = a.n_cols - it.nt * 128 - part * 32;  // valid columns (16s)
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          sum[j] = siluf_(sum[j]) * sum[32 + j];
          if (j < left) m = max(m, f8_mag(sum[j]));
        }
        uint32_t* mx = sMax + xph * kParts * BM + r;
        mx[part * BM] = m;
        __syncwarp();
        if (lane == 0) mbar_arrive(xbar);
        if (!warp_wait(xbar, xph, a, abort_flag)) break;
#pragma unroll
        for (int z = 0; z < kParts; ++z) m = max(m, mx[z * BM]);
        const uint32_t sbits = f8_scale_bits(m);
        const float inv = f8_inverse(sbits);
        xph ^= 1u;
        if (valid) {
          const size_t row = (size_t)it.row0 + i;
          uint8_t* dst = static_cast<uint8_t*>(a.out) + row * a.ldo + it.nt * 128 + part * 32;
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            if (16 * v < left) {
              uint32_t w[4];
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                const float* h = sum + 16 * v + 4 * z;
                w[z] = f8_pack4(h[0] * inv, h[1] * inv, h[2] * inv, h[3] * inv);
              }
              st_global_v4(dst + 16 * v, w[0], w[1], w[2], w[3]);
            }
          }
          if (part == 0) a.out_scale[row * a.out_blocks + it.nt] = __uint_as_float(sbits);
        }
      } else {
        // this warp's 32 rows x 64 columns, the first at row wrow of the group
        const int wrow = it.m * BM + q * 32, rows = it.rows - wrow;
        const int col = it.nt * BN + part * kPartCols;
        const int left = (MODE == kF8Dense && a.ksplit > 1 ? BN * a.n_tiles : a.n_cols) - col;
        uint4 c[8];
        if (MODE == kF8Dense && a.ksplit == 1 && a.out_bf16) {
          const int piece = 8 * (lane & 7);
#pragma unroll
          for (int j = 0; j < 8; ++j) c[j] = eight_bf16(sum + 8 * j);
          exchange8(c, lane);
          store8(static_cast<__nv_bfloat16*>(a.out) + (size_t)wrow * a.ldo + col + piece, a.ldo, c, rows,
                 left - piece, a.out_vec, lane);
        } else {
          // split k: fp32 rows of the tile, [split][tile][128 rows][256 columns]
          const bool part_sum = MODE == kF8Dense && a.ksplit > 1;
          float* out = part_sum ? a.partial + (((size_t)it.split * n_rb * a.n_tiles + it.tile) * BM + q * 32) * BN +
                                      part * kPartCols
                                : static_cast<float*>(a.out) + ((size_t)it.row0 + wrow) * a.ldo + col;
          if (MODE == kF8Down) {
#pragma unroll
            for (int j = 0; j < kPartCols; ++j) sum[j] *= al;
          }
          const long long pitch = part_sum ? BN : a.ldo;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int piece = 32 * h + 4 * (lane & 7);
#pragma unroll
            for (int j = 0; j < 8; ++j) c[j] = four_floats(sum + 32 * h + 4 * j);
            exchange8(c, lane);
            store8(out + piece, pitch, c, rows, left - piece, MODE == kF8Down || part_sum || a.out_vec, lane);
          }
        }
      }
    }
  }

  asm volatile("cp.async.wait_all;" ::: "memory");
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

// out = the splits' partial sums, added in split order; a thread per four
// columns of a row.
__global__ void __launch_bounds__(256) f8_split_sum_kernel(F8TcArgs a) {
  const int fours = (a.n_cols + 3) / 4;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const int row = (int)(i / fours), col = (int)(i - (long long)row * fours) * 4;
  pdl_wait();
  pdl_trigger();
  if (row >= a.rows) return;
  // the products' tile order (item_at)
  const int n_rb = (a.rows + BM - 1) / BM, rb = row / BM, nt = col / BN;
  const int band = rb / kBand, width = min(kBand, n_rb - band * kBand);
  const int tile = band * kBand * a.n_tiles + nt * width + (rb - band * kBand);
  const size_t plane = (size_t)n_rb * a.n_tiles * BM * BN;
  const float* p = a.partial + ((size_t)tile * BM + row % BM) * BN + col % BN;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int s = 0; s < a.ksplit; ++s) {
    const float4 o = __ldcg(reinterpret_cast<const float4*>(p + s * plane));
    v.x += o.x;
    v.y += o.y;
    v.z += o.z;
    v.w += o.w;
  }
  const float y[4] = {v.x, v.y, v.z, v.w};
  const size_t at = (size_t)row * a.ldo + col;
  if (a.out_bf16) {
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + at;
    if (a.out_vec && col + 4 <= a.n_cols) {
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
    } else {
#pragma unroll
      for (int z = 0; z < 4; ++z)
        if (col + z < a.n_cols) dst[z] = __float2bfloat16_rn(y[z]);
    }
  } else {
    float* dst = static_cast<float*>(a.out) + at;
    if (a.out_vec && col + 4 <= a.n_cols) {
      *reinterpret_cast<float4*>(dst) = v;
    } else {
#pragma unroll
      for (int z = 0; z < 4; ++z)
        if (col + z < a.n_cols) dst[z] = y[z];
    }
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

cudaError_t launch_f8_split_sum(const F8TcArgs& a, cudaStream_t st) {
  const long long n = (long long)a.rows * ((a.n_cols + 3) / 4);
  return launch_pdl(f8_split_sum_kernel, dim3((unsigned)((n + 255) / 256)), 256, 0, st, a);
}

}  // namespace moe
