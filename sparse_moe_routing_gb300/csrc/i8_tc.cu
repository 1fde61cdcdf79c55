// 8-bit integer products on the fifth-generation tensor cores.
//
// sm_103a's tensor cores multiply no 8-bit integers at speed (mma.sync s8 runs at
// 150 TOP/s), but fp16 holds every code exactly, a product of two codes is at
// most 2^14, and fp32 adds 1024 of them without a rounding (2^24). So the
// codes are widened to fp16 on the way to tcgen05.mma (kind::f16, 1.9 PFLOP/s),
// and after every 1024 k the sums are read from TMEM, converted and added
// into int32 registers: the result is the integers' exact sum, whatever the
// codes and whatever the order.
//
// The weights are the m side of the products (128 columns of the result), the
// tokens the n side. Weights come by TMA as 8-bit codes, 128 x 128 a step; four
// warps widen them, a thread one row, and write them to TMEM, from where
// tcgen05.mma takes its first operand: the widened weights cost no shared
// memory traffic. The tokens are few bytes and are widened once, by a launch
// before this one, into the workspace, and come by TMA as fp16.
//
// TMEM: columns 0-255 two accumulators of up to 128 columns, 256-511 four slots of
// widened weights (64 columns: 128 k of fp16 pairs). Accumulators:
//  * kI8Two   two blocks of `half` rows of A; one drains while the other fills;
//  * kI8Gated the gate and the up product of one block; the same;
//  * kI8One   one block; the accumulators take turns by 1024 k.
//
// Warps: 0 brings weights, 3 tokens, 1 and 2 issue the MMAs (an accumulator each;
// kI8One has one issuer), 4-7 widen, 8-15 read back, scale and store.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "fp8_common.cuh"
#include "i8_common.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

using namespace tc;

constexpr int kRows = 128;    // weight rows of a tile
constexpr int kStep = 128;    // k of a step
constexpr int kChunk = 8;     // steps whose sums fp32 holds exactly
constexpr int kSlots = 4;     // widened weights in TMEM
constexpr uint32_t kAccCols = 128, kSlotCol0 = 256, kSlotCols = 64, kTmemCols = 512;
constexpr int kStageW = kRows * kStep;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (8 + kEpiWarps);
static_assert(kChunk * kStep * 128 * 128 <= 1 << 24, "a chunk's sums are exact in fp32");

// Stages of the two rings: about 208 KB whatever the tokens' block.
template <int HALF>
struct Plan {
  static constexpr int kStageT = HALF * kStep * 2;
  static constexpr int kT = HALF == 128 ? 4 : HALF == 64 ? 6 : 8;
  static constexpr int kW = HALF == 128 ? 5 : HALF == 64 ? 7 : HALF == 32 ? 9 : 11;
  static constexpr size_t kToken = 0;
  static constexpr size_t kWeight = kToken + (size_t)kT * kStageT;
  static constexpr size_t kBars = kWeight + (size_t)kW * kStageW;
  static constexpr size_t kBytes = 1024 + kBars + (2 * kT + 2 * kW + 2 * kSlots + 4) * 8 + 16;
  static_assert(kBytes <= 227 * 1024, "shared memory plan exceeds 227 KB");
};

// kind::f16: fp32 accumulate, A and B fp16, both K-major, 128 x n.
constexpr uint32_t idesc_f16(int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
}
// D (TMEM) [+]= A (TMEM) B (shared memory).
__device__ __forceinline__ void mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
      "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]),
      "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

struct Item {
  int mt, nt;     // block of rows of A, tile of columns
  int kb0, kb1;   // steps
  int tile, split;
};
// Items walk bands of 8 token tiles, column tile by column tile, so that the
// CTAs in flight share both operands through L2.
constexpr int kBand = 8;
__host__ __device__ __forceinline__ void tile_at(int t, int m_tiles, int n_tiles, int& mt, int& nt) {
  const int span = kBand * n_tiles, band = t / span, w = t - band * span;
  const int left = m_tiles - band * kBand, width = left < kBand ? left : kBand;
  mt = band * kBand + w % width;
  nt = w / width;
}
__device__ __forceinline__ Item item_at(const I8TcArgs& a, int t) {
  Item it;
  it.split = t % a.ksplit;
  it.tile = t / a.ksplit;
  it.kb0 = it.split * a.steps / a.ksplit;
  it.kb1 = (it.split + 1) * a.steps / a.ksplit;
  tile_at(it.tile, a.m_tiles, a.n_tiles, it.mt, it.nt);
  return it;
}

__device__ __forceinline__ void give_up(const I8TcArgs& a, volatile int* abort_flag) {
  *abort_flag = 1;
  report(a.ctrl, kDevTimeout, kSiteTcI8);
}
__device__ __forceinline__ bool lane_wait(uint64_t* bar, uint32_t parity, const I8TcArgs& a,
                                          volatile int* abort_flag) {
  const bool ok = f8_lane_wait(bar, parity, a.wait_ns, abort_flag);
  if (!ok) give_up(a, abort_flag);
  return ok;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const I8TcArgs& a,
                                          volatile int* abort_flag) {
  const bool ok = __all_sync(0xffffffffu, f8_lane_wait(bar, parity, a.wait_ns, abort_flag));
  if (!ok && (threadIdx.x & 31) == 0) give_up(a, abort_flag);
  return ok;
}
// A ring's place: stage and parity after n uses.
struct Place {
  int at = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next(int n) {
    if (++at == n) {
      at = 0;
      ph ^= 1u;
    }
  }
};

template <int KIND, int HALF>
__global__ void __launch_bounds__(kThreads, 1)
    i8_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB0,
                 const __grid_constant__ CUtensorMap tmB1, const I8TcArgs a) {
  using P = Plan<HALF>;
  constexpr int kBlocks = KIND == kI8Two ? 2 : 1;    // token blocks of a tile
  constexpr int kWeights = KIND == kI8Gated ? 2 : 1; // weight matrices
  constexpr int kSums = KIND == kI8One ? 1 : 2;      // accumulators that an item ends with
  constexpr uint32_t kIdesc = idesc_f16(HALF);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sT = smem + P::kToken;
  uint8_t* sW = smem + P::kWeight;
  uint64_t* tfull = reinterpret_cast<uint64_t*>(smem + P::kBars);
  uint64_t* tempty = tfull + P::kT;
  uint64_t* wfull = tempty + P::kT;
  uint64_t* wempty = wfull + P::kW;
  uint64_t* sfull = wempty + P::kW;   // slots of widened weights
  uint64_t* sempty = sfull + kSlots;
  uint64_t* dfull = sempty + kSlots;  // accumulators
  uint64_t* dempty = dfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(dempty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < P::kT; ++s) {
      mbar_init(&tfull[s], 1);
      mbar_init(&tempty[s], kWeights);  // one commit per issuer that reads the stage
    }
    for (int s = 0; s < P::kW; ++s) {
      mbar_init(&wfull[s], 1);
      mbar_init(&wempty[s], 4);
    }
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&sfull[s], 4);
      mbar_init(&sempty[s], kBlocks);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&dfull[b], 1);
      mbar_init(&dempty[b], kEpiWarps);
    }
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
  const int total = a.m_tiles * a.n_tiles * a.ksplit;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0) {
      // --------------------------------------------------------------- weights
      if (lane == 0) {
        Place p;
        bool alive = true;
        for (int t = blockIdx.x; t < total && alive; t += gridDim.x) {
          const Item it = item_at(a, t);
          for (int kb = it.kb0; kb < it.kb1 && alive; ++kb) {
#pragma unroll
            for (int w = 0; w < kWeights; ++w) {
              if (!(alive = lane_wait(&wempty[p.at], p.ph ^ 1u, a, abort_flag))) break;
              mbar_expect_tx(&wfull[p.at], kStageW);
              tma_load_2d(sW + p.at * kStageW, w ? &tmB1 : &tmB0, &wfull[p.at], kb * kStep, it.nt * kRows);
              p.next(P::kW);
            }
          }
        }
      }
    } else if (warp == 3) {
      // ---------------------------------------------------------------- tokens
      if (lane == 0) {
        Place p;
        bool alive = true;
        for (int t = blockIdx.x; t < total && alive; t += gridDim.x) {
          const Item it = item_at(a, t);
          for (int kb = it.kb0; kb < it.kb1 && alive; ++kb) {
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
              if (!(alive = lane_wait(&tempty[p.at], p.ph ^ 1u, a, abort_flag))) break;
              uint8_t* dst = sT + p.at * P::kStageT;
              const int row = (it.mt * kBlocks + b) * HALF;
              mbar_expect_tx(&tfull[p.at], P::kStageT);
              tma_load_2d(dst, &tmA, &tfull[p.at], kb * kStep, row);
              tma_load_2d(dst + P::kStageT / 2, &tmA, &tfull[p.at], kb * kStep + kStep / 2, row);
              p.next(P::kT);
            }
          }
        }
      }
    } else if (warp - 1 < kSums) {
      // --------------------------------------------------------------- issuers
      if (lane == 0) {
        const int me = warp - 1;
        Place tp, sp;         // this issuer's next token stage and weight slot
        if (KIND == kI8Two && me) tp.next(P::kT);
        if (KIND == kI8Gated && me) sp.next(kSlots);
        uint32_t used[2] = {0, 0};  // chunks that an accumulator has had
        int acc = me;
        // failure self-test: wait on a barrier that only this warp completes
        bool alive = !a.stall || lane_wait(&dfull[me], 0u, a, abort_flag);
        for (int t = blockIdx.x; t < total && alive; t += gridDim.x) {
          const Item it = item_at(a, t);
          for (int kb = it.kb0; kb < it.kb1; ++kb) {
            const int in_chunk = (kb - it.kb0) % kChunk;
            if (in_chunk == 0 && !(alive = lane_wait(&dempty[acc], (used[acc] & 1u) ^ 1u, a, abort_flag))) break;
            if (!(alive = lane_wait(&sfull[sp.at], sp.ph, a, abort_flag) &&
                          lane_wait(&tfull[tp.at], tp.ph, a, abort_flag)))
              break;
            tc_fence_after();
            const uint32_t d = tmem_base + acc * kAccCols;
            const uint32_t w = tmem_base + kSlotCol0 + sp.at * kSlotCols;
            const uint64_t b = sw128_desc(smem_u32(sT + tp.at * P::kStageT));
            constexpr uint64_t kHalfStage = (P::kStageT / 2) >> 4;
#pragma unroll
            for (int k = 0; k < kStep / 16; ++k)  // 16 k: 8 columns of A, 32 bytes of B's rows
              mma_f16_ta(d, w + 8 * k, b + (k >> 2) * kHalfStage + 2 * (k & 3), kIdesc,
                         in_chunk != 0 || k != 0 ? 1u : 0u);
            mma_commit(&tempty[tp.at]);
            mma_commit(&sempty[sp.at]);
            if (in_chunk == kChunk - 1 || kb == it.kb1 - 1) {
              mma_commit(&dfull[acc]);
              ++used[acc];
              if (KIND == kI8One) acc ^= 1;
            }
            for (int i = 0; i < kBlocks; ++i) tp.next(P::kT);
            for (int i = 0; i < kWeights; ++i) sp.next(kSlots);
          }
        }
      }
    }
    __syncwarp();
  } else if (warp < 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    // ------------------------------------------------------------------- widen
    const int r = (warp & 3) * 32 + lane;  // this thread's weight row, and TMEM lane
    const uint32_t tq = tmem_base + ((uint32_t)((warp & 3) * 32) << 16) + kSlotCol0;
    Place wp, sp;
    bool alive = true;
    for (int t = blockIdx.x; t < total && alive; t += gridDim.x) {
      const int split = t % a.ksplit;
      const int tiles = ((split + 1) * a.steps / a.ksplit - split * a.steps / a.ksplit) * kWeights;
      for (int i = 0; i < tiles; ++i) {
        if (!(alive = warp_wait(&wfull[wp.at], wp.ph, a, abort_flag) &&
                      warp_wait(&sempty[sp.at], sp.ph ^ 1u, a, abort_flag)))
          break;
        tc_fence_after();
        const uint8_t* row = sW + wp.at * kStageW + r * kStep;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t v[32];
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // 16-byte pieces, swizzled by the row
            const uint4 w = ld_shared_v4(row + (((h * 4 + c) ^ (r & 7)) << 4));
            i8_to_f16(w.x, v[8 * c], v[8 * c + 1]);
            i8_to_f16(w.y, v[8 * c + 2], v[8 * c + 3]);
            i8_to_f16(w.z, v[8 * c + 4], v[8 * c + 5]);
            i8_to_f16(w.w, v[8 * c + 6], v[8 * c + 7]);
          }
          tmem_st32(tq + sp.at * kSlotCols + h * 32, v);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&wempty[wp.at]);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sfull[sp.at]);
        wp.next(P::kW);
        sp.next(kSlots);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    // ---------------------------------------------------------------- epilogue
    constexpr int kCols = HALF / 2;  // columns of an accumulator that a warp reads
    constexpr int kPiece = kCols < 16 ? 8 : 16;
    const int part = (warp - 8) >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t tq = tmem_base + ((uint32_t)((warp & 3) * 32) << 16) + part * kCols;
    int acc = 0;
    uint32_t ph[2] = {0, 0};
    bool alive = true;
    for (int t = blockIdx.x; t < total && alive; t += gridDim.x) {
      const Item it = item_at(a, t);
      int sum[kSums][kCols];
#pragma unroll
      for (int s = 0; s < kSums; ++s)
#pragma unroll
        for (int j = 0; j < kCols; ++j) sum[s][j] = 0;
      for (int kb = it.kb0; kb < it.kb1 && alive; kb += kChunk) {
#pragma unroll
        for (int s = 0; s < kSums; ++s) {
          const int at = KIND == kI8One ? acc : s;
          if (!(alive = warp_wait(&dfull[at], ph[at], a, abort_flag))) break;
          ph[at] ^= 1u;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < kCols / kPiece; ++c) {
            uint32_t v[kPiece];
            if (kPiece == 8)
              tmem_ld8(tq + at * kAccCols + c * kPiece, v);
            else
              tmem_ld16(tq + at * kAccCols + c * kPiece, v);
            tmem_ld_wait();
            // the read's registers hold their values from here on: the compiler
            // moves no use above the wait
#pragma unroll
            for (int j = 0; j < kPiece; ++j) asm volatile("" : "+r"(v[j]));
#pragma unroll
            for (int j = 0; j < kPiece; ++j)
              sum[s][c * kPiece + j] += __float2int_rn(__uint_as_float(v[j]));
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&dempty[at]);
          if (KIND == kI8One) acc ^= 1;
        }
      }
      if (!alive) break;
      if (a.ksplit > 1) {
        int* p = a.partial +
                 (((size_t)it.split * a.m_tiles * a.n_tiles + it.tile) * kSums * HALF + part * kCols) * kRows + r;
#pragma unroll
        for (int s = 0; s < kSums; ++s)
#pragma unroll
          for (int j = 0; j < kCols; ++j) p[(s * HALF + j) * kRows] = sum[s][j];
        continue;
      }
      const int n = it.nt * kRows + r;
      const bool in = n < a.N;
      const float b0 = in ? a.b_scale0[n] : 0.f;
      const float b1 = KIND == kI8Gated && in ? a.b_scale1[n] : 0.f;
#pragma unroll
      for (int s = 0; s < (KIND == kI8Two ? 2 : 1); ++s) {
        const int m0 = (it.mt * kBlocks + s) * HALF + part * kCols;
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
          const int m = m0 + j;
          if (m >= a.M) break;
          const float sa = __ldg(a.a_scale + m);
          float y = i8_value(sum[s][j], sa, b0);
          if (KIND == kI8Gated) y = siluf_(y) * i8_value(sum[kSums - 1][j], sa, b1);
          if (in) i8_store(a.out, (size_t)m * a.ldo + n, a.out_bf16, y);
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
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols));
  }
}

// Rows of codes as fp16, 16 a thread.
__global__ void __launch_bounds__(256) i8_widen_kernel(I8WidenArgs a) {
  const int pieces = a.pitch / 16;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  pdl_wait();
  pdl_trigger();
  if (i >= (long long)a.rows * pieces) return;
  const long long row = i / pieces;
  const int k = (int)(i - row * pieces) * 16;
  const uint4 w = i8_load16(a.a + row * a.lda, k, a.cols);
  uint32_t v[8];
  i8_to_f16(w.x, v[0], v[1]);
  i8_to_f16(w.y, v[2], v[3]);
  i8_to_f16(w.z, v[4], v[5]);
  i8_to_f16(w.w, v[6], v[7]);
  uint16_t* dst = static_cast<uint16_t*>(a.out) + row * a.pitch + k;
  st_global_v4(dst, v[0], v[1], v[2], v[3]);
  st_global_v4(dst + 8, v[4], v[5], v[6], v[7]);
}

// The splits' sums of one output (two, gated) added and finished; a thread an
// output, a block 128 columns of two rows.
template <int KIND>
__global__ void __launch_bounds__(256) i8_split_sum_kernel(I8TcArgs a, int half) {
  pdl_wait();
  pdl_trigger();
  const int per = half * (KIND == kI8Two ? 2 : 1);  // rows of a tile
  const int r = threadIdx.x & (kRows - 1);
  const int groups = (per + 1) / 2;
  const int tile = blockIdx.x / groups, j = (blockIdx.x % groups) * 2 + (threadIdx.x >> 7);
  int mt, nt;
  tile_at(tile, a.m_tiles, a.n_tiles, mt, nt);
  const int m = mt * per + j, n = nt * kRows + r;
  if (m >= a.M || n >= a.N) return;
  const int sums = KIND == kI8One ? 1 : 2;
  const size_t plane = (size_t)a.m_tiles * a.n_tiles * sums * half * kRows;
  const int* p = a.partial + ((size_t)tile * sums * half + j) * kRows + r;
  int s0 = 0, s1 = 0;
#pragma unroll 8
  for (int z = 0; z < a.ksplit; ++z) {
    s0 += __ldcg(p + z * plane);
    if (KIND == kI8Gated) s1 += __ldcg(p + z * plane + (size_t)half * kRows);
  }
  const float sa = a.a_scale[m];
  float y = i8_value(s0, sa, a.b_scale0[n]);
  if (KIND == kI8Gated) y = siluf_(y) * i8_value(s1, sa, a.b_scale1[n]);
  i8_store(a.out, (size_t)m * a.ldo + n, a.out_bf16, y);
}

template <int KIND, int HALF>
cudaError_t launch_t(const I8TcMaps& m, const I8TcArgs& a, cudaStream_t st) {
  static int attr[64] = {};
  cudaError_t e = ensure_smem_limit(i8_tc_kernel<KIND, HALF>, (int)Plan<HALF>::kBytes, attr);
  if (e != cudaSuccess) return e;
  const int items = a.m_tiles * a.n_tiles * a.ksplit, sms = tc_sm_count();
  return launch_pdl(i8_tc_kernel<KIND, HALF>, dim3(items < sms ? items : sms), kThreads, Plan<HALF>::kBytes, st,
                    m.A, m.B0, m.B1, a);
}
template <int KIND>
cudaError_t launch_half(int half, const I8TcMaps& m, const I8TcArgs& a, cudaStream_t st) {
  if (half == 16) return launch_t<KIND, 16>(m, a, st);
  if (half == 32) return launch_t<KIND, 32>(m, a, st);
  if (half == 64) return launch_t<KIND, 64>(m, a, st);
  return half == 128 ? launch_t<KIND, 128>(m, a, st) : cudaErrorInvalidValue;
}

}  // namespace

bool i8_make_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint64_t pitch,
                 uint32_t box_rows) {
  auto fn = tc_encode_fn();
  if (!fn || !base) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {pitch * 2};
  cuuint32_t box[2] = {64, box_rows};
  cuuint32_t es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_i8_tc(I8Kind kind, int half, const I8TcMaps& m, const I8TcArgs& a, cudaStream_t st) {
  if (kind == kI8One) return launch_half<kI8One>(half, m, a, st);
  if (kind == kI8Gated) return launch_half<kI8Gated>(half, m, a, st);
  return half == 128 ? launch_t<kI8Two, 128>(m, a, st) : cudaErrorInvalidValue;
}

cudaError_t launch_i8_widen(const I8WidenArgs& a, cudaStream_t st) {
  const long long n = (long long)a.rows * (a.pitch / 16);
  return launch_pdl(i8_widen_kernel, dim3((unsigned)((n + 255) / 256)), 256, 0, st, a);
}

cudaError_t launch_i8_split_sum(I8Kind kind, int half, const I8TcArgs& a, cudaStream_t st) {
  const int per = half * (kind == kI8Two ? 2 : 1);
  const dim3 grid((unsigned)(a.m_tiles * a.n_tiles * ((per + 1) / 2)));
  if (kind == kI8One) return launch_pdl(i8_split_sum_kernel<kI8One>, grid, 256, 0, st, a, half);
  if (kind == kI8Two) return launch_pdl(i8_split_sum_kernel<kI8Two>, grid, 256, 0, st, a, half);
  return launch_pdl(i8_split_sum_kernel<kI8Gated>, grid, 256, 0, st, a, half);
}

}  // namespace moe
