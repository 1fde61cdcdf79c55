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
// The weights are the m side of the products (128 rows a tile; gated: 64 rows of
// gate and the same 64 of up, 16 and 16 in turn), the tokens the n side. Weights come by TMA as
// 8-bit codes, 128 x 128 a step; eight warps widen them, a thread half a row,
// and write them to TMEM, from where tcgen05.mma takes its first operand: the
// widened weights cost no shared memory traffic. The tokens are few bytes and
// are widened once, by a launch before this one, into the workspace, and come by
// TMA as fp16.
//
// Two threads issue the MMAs: what an issuer does between two steps (two waits,
// two commits) takes longer than the step's MMAs leave. With one block of tokens
// (kI8One) they take the steps in turn, with two (kI8Two) a block each, and each
// sums on its own. Their sums rotate through three accumulators, so that one is
// read back while two fill (two accumulators left the tensor core idle for the
// read-back, 1400 cycles every 1024 k: the conversion to integers runs at 16 a
// cycle).
//
// Warps: 0 brings weights, 3 tokens, 1 and 2 issue, 4-11 widen, 12-19 read back,
// scale and store. Gated, the two lanes of a warp that hold a column's gate and
// its up sums give each other half of them.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <type_traits>

#include "fp8_common.cuh"
#include "i8_common.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

using namespace tc;

constexpr int kRows = 128;    // weight rows of a tile
constexpr int kStep = 128;    // k of a step
constexpr int kChunk = 8;     // steps whose sums fp32 holds exactly
constexpr int kAccs = 3;      // accumulators
constexpr uint32_t kSlotCols = 64, kTmemCols = 512;
constexpr int kStageW = kRows * kStep;
constexpr int kConvWarp0 = 4, kConvWarps = 8, kEpiWarp0 = 12, kEpiWarps = 8;
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
static_assert(kChunk * kStep * 128 * 128 <= 1 << 24, "a chunk's sums are exact in fp32");

template <int HALF>
struct Plan {
  // TMEM: accumulators, then widened weights (64 columns: 128 k of fp16 pairs)
  static constexpr uint32_t kAccCols = HALF == 128 ? 128 : 64;
  static constexpr uint32_t kSlotCol0 = HALF == 128 ? 384 : 256;
  static constexpr int kSlots = HALF == 128 ? 2 : 4;
  // stages of the two rings, up to about 200 KB
  static constexpr int kStageT = HALF * kStep * 2;
  static constexpr int kT = HALF == 128 ? 4 : HALF == 64 ? 6 : 8;
  static constexpr int kW = HALF == 128 ? 4 : HALF == 64 ? 6 : HALF == 32 ? 8 : 10;
  static constexpr int kCols = HALF / 2;  // columns of an accumulator that an epilogue warp reads
  static constexpr size_t kToken = 0;
  static constexpr size_t kWeight = kToken + (size_t)kT * kStageT;
  static constexpr size_t kScale = kWeight + (size_t)kW * kStageW;  // [epilogue warp][128] scales of rows of A
  static constexpr size_t kBars = kScale + kEpiWarps * 128 * 4;
  static constexpr size_t kBytes = 1024 + kBars + (2 * kT + 2 * kW + 2 * kSlots + 2 * kAccs) * 8 + 16;
  static_assert(kAccs * kAccCols <= kSlotCol0 && kSlotCol0 + kSlots * kSlotCols <= kTmemCols, "TMEM plan");
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

// Asynchronous copy of one fp32 value to shared memory, or of zero; and the wait
// for this thread's copies.
__device__ __forceinline__ void copy4_async(float* dst, const float* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(valid ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

struct Item {
  int mt, nt;     // tile of rows of A, tile of weight rows
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

// Gated: the output that row r of a tile holds the gate or the up sum of, and the
// row of output c's gate sum (up's is 16 rows on).
__device__ __forceinline__ int out_of_row(int r) { return (r >> 5) * 16 + (r & 15); }
__device__ __forceinline__ int row_of_out(int c) { return (c >> 4) * 32 + (c & 15); }

// Accumulators that an item of n steps fills: eight steps each, the two issuers'
// in turn (kI8One: every second step each, so that a lone last step is the
// first issuer's).
template <int KIND>
__device__ __forceinline__ int accs_of(int n) {
  if (KIND == kI8Two) return 2 * ((n + kChunk - 1) / kChunk);
  const int rest = n % (2 * kChunk);
  return 2 * (n / (2 * kChunk)) + (rest < 2 ? rest : 2);
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

template <int KIND, int HALF, bool GATED>
__global__ void __launch_bounds__(kThreads, 1)
    i8_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB0,
                 const __grid_constant__ CUtensorMap tmB1, const I8TcArgs a) {
  using P = Plan<HALF>;
  constexpr int kBlocks = KIND == kI8Two ? 2 : 1;  // token blocks of a tile
  constexpr int kOuts = GATED ? kRows / 2 : kRows;  // columns of the result of a tile
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
  uint64_t* sfull = wempty + P::kW;      // slots of widened weights
  uint64_t* sempty = sfull + P::kSlots;
  uint64_t* dfull = sempty + P::kSlots;  // accumulators
  uint64_t* dempty = dfull + kAccs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(dempty + kAccs);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < P::kT; ++s) {
      mbar_init(&tfull[s], 1);
      mbar_init(&tempty[s], 1);
    }
    for (int s = 0; s < P::kW; ++s) {
      mbar_init(&wfull[s], 1);
      mbar_init(&wempty[s], kConvWarps);
    }
    for (int s = 0; s < P::kSlots; ++s) {
      mbar_init(&sfull[s], kConvWarps);
      mbar_init(&sempty[s], kBlocks);  // one commit per issuer that reads the slot
    }
    for (int b = 0; b < kAccs; ++b) {
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
  const int total = a.m_tiles * a.n_tiles * a.ksplit;

  if (warp < kConvWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp == 0) {
      // --------------------------------------------------------------- weights
      // Before the wait for the kernel before this one: that is the same call's
      // widening of the tokens, and what is older has completed.
      if (lane == 0) {
        Place p;
        bool alive = true;
        for (int t = blockIdx.x; t < total && alive; t += gridDim.x) {
          const Item it = item_at(a, t);
          for (int kb = it.kb0; kb < it.kb1; ++kb) {
            if (!(alive = lane_wait(&wempty[p.at], p.ph ^ 1u, a, abort_flag))) break;
            uint8_t* dst = sW + p.at * kStageW;
            mbar_expect_tx(&wfull[p.at], kStageW);
            if (GATED) {
#pragma unroll
              for (int i = 0; i < kRows / 32; ++i) {
                tma_load_2d(dst + i * 32 * kStep, &tmB0, &wfull[p.at], kb * kStep, it.nt * kOuts + i * 16);
                tma_load_2d(dst + (i * 32 + 16) * kStep, &tmB1, &wfull[p.at], kb * kStep, it.nt * kOuts + i * 16);
              }
            } else {
              tma_load_2d(dst, &tmB0, &wfull[p.at], kb * kStep, it.nt * kOuts);
            }
            p.next(P::kW);
          }
        }
      }
    } else if (warp == 3) {
      // ---------------------------------------------------------------- tokens
      pdl_wait();
      pdl_trigger();
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
    } else if (lane == 0) {
      // --------------------------------------------------------------- issuers
      const int me = warp - 1;
      Place tp, sp;  // token stage and weight slot
      if (KIND == kI8Two && me) tp.next(P::kT);
      int base = 0;  // accumulators filled before this item
      // failure self-test: wait on a barrier that only this warp completes
      bool alive = !a.stall || lane_wait(&dfull[me], 0u, a, abort_flag);
      for (int t = blockIdx.x; t < total && alive; t += gridDim.x) {
        const Item it = item_at(a, t);
        const int n = it.kb1 - it.kb0;
        int in_chunk = 0, use = base + me;
        for (int i = 0; i < n; ++i) {
          if (KIND == kI8Two || (i & 1) == me) {
            const int acc = use % kAccs;
            if (in_chunk == 0 &&
                !(alive = lane_wait(&dempty[acc], ((use / kAccs) & 1u) ^ 1u, a, abort_flag)))
              break;
            if (!(alive = lane_wait(&sfull[sp.at], sp.ph, a, abort_flag) &&
                          lane_wait(&tfull[tp.at], tp.ph, a, abort_flag)))
              break;
            tc_fence_after();
            const uint32_t d = tmem_base + acc * P::kAccCols;
            const uint32_t w = tmem_base + P::kSlotCol0 + sp.at * kSlotCols;
            const uint64_t b = sw128_desc(smem_u32(sT + tp.at * P::kStageT));
            constexpr uint64_t kHalfStage = (P::kStageT / 2) >> 4;
#pragma unroll
            for (int k = 0; k < kStep / 16; ++k)  // 16 k: 8 columns of A, 32 bytes of B's rows
              mma_f16_ta(d, w + 8 * k, b + (k >> 2) * kHalfStage + 2 * (k & 3), kIdesc,
                         in_chunk != 0 || k != 0 ? 1u : 0u);
            mma_commit(&tempty[tp.at]);
            mma_commit(&sempty[sp.at]);
            if (++in_chunk == kChunk || i + (KIND == kI8Two ? 1 : 2) >= n) {
              mma_commit(&dfull[acc]);
              in_chunk = 0;
              use += 2;
            }
          }
          tp.next(P::kT);
          if (KIND == kI8Two) tp.next(P::kT);
          sp.next(P::kSlots);
        }
        base += accs_of<KIND>(n);
      }
    }
    __syncwarp();
  } else if (warp < kEpiWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    // ------------------------------------------------------------------- widen
    const int r = (warp & 3) * 32 + lane;        // this thread's weight row, and TMEM lane
    const int h = (warp - kConvWarp0) >> 2;      // its half of the step's k
    const uint32_t tq = tmem_base + ((uint32_t)((warp & 3) * 32) << 16) + P::kSlotCol0 + h * (kSlotCols / 2);
    Place wp, sp;
    bool alive = true;
    for (int t = blockIdx.x; t < total && alive; t += gridDim.x) {
      const int split = t % a.ksplit;
      const int n = (split + 1) * a.steps / a.ksplit - split * a.steps / a.ksplit;
      for (int i = 0; i < n; ++i) {
        if (!(alive = warp_wait(&wfull[wp.at], wp.ph, a, abort_flag))) break;
        const uint8_t* row = sW + wp.at * kStageW + r * kStep;
        uint32_t v[32];
#pragma unroll
        for (int c = 0; c < 4; ++c) {  // 16-byte pieces, swizzled by the row
          const uint4 w = ld_shared_v4(row + (((h * 4 + c) ^ (r & 7)) << 4));
          i8_to_f16(w.x, v[8 * c], v[8 * c + 1]);
          i8_to_f16(w.y, v[8 * c + 2], v[8 * c + 3]);
          i8_to_f16(w.z, v[8 * c + 4], v[8 * c + 5]);
          i8_to_f16(w.w, v[8 * c + 6], v[8 * c + 7]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&wempty[wp.at]);
        if (!(alive = warp_wait(&sempty[sp.at], sp.ph ^ 1u, a, abort_flag))) break;
        tc_fence_after();
        tmem_st32(tq + sp.at * kSlotCols, v);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sfull[sp.at]);
        wp.next(P::kW);
        sp.next(P::kSlots);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
    // ---------------------------------------------------------------- epilogue
    constexpr int kCols = P::kCols;
    constexpr int kPiece = kCols < 16 ? 8 : 16;
    const int mine = warp - kEpiWarp0, part = mine >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t tq = tmem_base + ((uint32_t)((warp & 3) * 32) << 16) + part * kCols;
    float* scale = reinterpret_cast<float*>(smem + P::kScale) + mine * 128;
    const bool up = GATED && (lane & 16) != 0;  // this lane's row is up's
    int use = 0;
    bool alive = true;
    for (int t = blockIdx.x; t < total && alive; t += gridDim.x) {
      const Item it = item_at(a, t);
      // the scales of this warp's rows of A, in flight during the steps
      constexpr int kMine = kBlocks * kCols;
#pragma unroll
      for (int i = 0; i < (kMine + 31) / 32; ++i) {
        const int j = i * 32 + lane, m = (it.mt * kBlocks + j / kCols) * HALF + part * kCols + j % kCols;
        if (j < kMine) copy4_async(scale + j, a.a_scale + (m < a.M ? m : 0), m < a.M);
      }
      const int n = it.nt * kOuts + (GATED ? out_of_row(r) : r);
      const bool in = n < a.N;
      const float b0 = in ? a.b_scale0[n] : 0.f;
      const float b1 = GATED && in ? a.b_scale1[n] : 0.f;
      int sum[kBlocks][kCols];
#pragma unroll
      for (int s = 0; s < kBlocks; ++s)
#pragma unroll
        for (int j = 0; j < kCols; ++j) sum[s][j] = 0;
      for (int left = accs_of<KIND>(it.kb1 - it.kb0); left > 0 && alive; left -= kBlocks) {
#pragma unroll
        for (int s = 0; s < kBlocks; ++s) {
          const int acc = use % kAccs;
          if (!(alive = warp_wait(&dfull[acc], (use / kAccs) & 1u, a, abort_flag))) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < kCols / kPiece; ++c) {
            uint32_t v[kPiece];
            if (kPiece == 8)
              tmem_ld8(tq + acc * P::kAccCols + c * kPiece, v);
            else
              tmem_ld16(tq + acc * P::kAccCols + c * kPiece, v);
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
          if (lane == 0) mbar_arrive(&dempty[acc]);
          ++use;
        }
      }
      if (!alive) break;
      if (a.ksplit > 1) {
        int* p = a.partial +
                 (((size_t)it.split * a.m_tiles * a.n_tiles + it.tile) * kBlocks * HALF + part * kCols) * kRows + r;
#pragma unroll
        for (int s = 0; s < kBlocks; ++s)
#pragma unroll
          for (int j = 0; j < kCols; ++j) p[(s * HALF + j) * kRows] = sum[s][j];
        continue;
      }
      copies_wait();
      __syncwarp();
      // WHOLE: every row of this warp's blocks exists.
      const auto finish = [&](auto* out, auto whole) {
        constexpr bool WHOLE = decltype(whole)::value;
#pragma unroll
        for (int s = 0; s < kBlocks; ++s) {
          const int m0 = (it.mt * kBlocks + s) * HALF + part * kCols;
          if (!GATED) {
            auto* dst = out + (long long)m0 * a.ldo + n;
            if (in) {
#pragma unroll
              for (int j = 0; j < kCols; j += 8) {
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                  const float4 sa = *reinterpret_cast<const float4*>(scale + s * kCols + j + i);
                  y[i] = i8_value(sum[s][j + i], sa.x, b0);
                  y[i + 1] = i8_value(sum[s][j + i + 1], sa.y, b0);
                  y[i + 2] = i8_value(sum[s][j + i + 2], sa.z, b0);
                  y[i + 3] = i8_value(sum[s][j + i + 3], sa.w, b0);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  if (WHOLE || m0 + j + i < a.M) store_act(dst, 0, y[i]);
                  dst += a.ldo;
                }
              }
            }
          } else {
            // A gate lane finishes the first half of its columns, its up lane the
            // second: each hands on its sums of the other half.
            const int c0 = up ? kCols / 2 : 0;
            auto* dst = out + (long long)(m0 + c0) * a.ldo + n;
            constexpr int kGroup = kCols / 2 < 8 ? kCols / 2 : 8;
#pragma unroll
            for (int p = 0; p < kCols / 2; p += kGroup) {
              float y[kGroup];
#pragma unroll
              for (int j = 0; j < kGroup; ++j) {
                const int lo = sum[s][p + j], hi = sum[s][kCols / 2 + p + j];
                const int own = up ? hi : lo, other = __shfl_xor_sync(0xffffffffu, up ? lo : hi, 16);
                const float sa = scale[s * kCols + c0 + p + j];
                const float g = i8_value(up ? other : own, sa, b0);
                y[j] = siluf_(g) * i8_value(up ? own : other, sa, b1);
              }
#pragma unroll
              for (int j = 0; j < kGroup; ++j) {
                if (in && (WHOLE || m0 + c0 + p + j < a.M)) store_act(dst, 0, y[j]);
                dst += a.ldo;
              }
            }
          }
        }
      };
      const bool whole = (it.mt + 1) * kBlocks * HALF <= a.M;
      const auto finish_as = [&](auto* out) {
        if (whole)
          finish(out, std::true_type{});
        else
          finish(out, std::false_type{});
      };
      if (a.out_bf16)
        finish_as(static_cast<__nv_bfloat16*>(a.out));
      else
        finish_as(static_cast<float*>(a.out));
      __syncwarp();  // the scales are read before the next item's come
    }
  }

  copies_wait();
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
// output, a block the columns of a tile and two (gated: four) of its rows.
template <bool GATED>
__global__ void __launch_bounds__(256) i8_split_sum_kernel(I8TcArgs a, int rows) {
  pdl_wait();
  pdl_trigger();
  constexpr int kOuts = GATED ? kRows / 2 : kRows, kPer = 256 / kOuts;
  const int r = threadIdx.x % kOuts;
  const int groups = (rows + kPer - 1) / kPer;
  const int tile = blockIdx.x / groups, j = (blockIdx.x % groups) * kPer + threadIdx.x / kOuts;
  int mt, nt;
  tile_at(tile, a.m_tiles, a.n_tiles, mt, nt);
  const int m = mt * rows + j, n = nt * kOuts + r;
  if (m >= a.M || n >= a.N) return;
  const size_t plane = (size_t)a.m_tiles * a.n_tiles * rows * kRows;
  const int* p = a.partial + ((size_t)tile * rows + j) * kRows + (GATED ? row_of_out(r) : r);
  int s0 = 0, s1 = 0;
#pragma unroll 8
  for (int z = 0; z < a.ksplit; ++z) {
    s0 += __ldcg(p + z * plane);
    if (GATED) s1 += __ldcg(p + z * plane + 16);
  }
  const float sa = a.a_scale[m];
  float y = i8_value(s0, sa, a.b_scale0[n]);
  if (GATED) y = siluf_(y) * i8_value(s1, sa, a.b_scale1[n]);
  i8_store(a.out, (size_t)m * a.ldo + n, a.out_bf16, y);
}

template <int KIND, int HALF, bool GATED>
cudaError_t launch_t(const I8TcMaps& m, const I8TcArgs& a, cudaStream_t st) {
  static int attr[64] = {};
  cudaError_t e = ensure_smem_limit(i8_tc_kernel<KIND, HALF, GATED>, (int)Plan<HALF>::kBytes, attr);
  if (e != cudaSuccess) return e;
  const int items = a.m_tiles * a.n_tiles * a.ksplit, sms = tc_sm_count();
  return launch_pdl(i8_tc_kernel<KIND, HALF, GATED>, dim3(items < sms ? items : sms), kThreads, Plan<HALF>::kBytes,
                    st, m.A, m.B0, m.B1, a);
}
template <bool GATED>
cudaError_t launch_half(I8Kind kind, int half, const I8TcMaps& m, const I8TcArgs& a, cudaStream_t st) {
  if (kind == kI8Two) return half == 128 ? launch_t<kI8Two, 128, GATED>(m, a, st) : cudaErrorInvalidValue;
  if (half == 16) return launch_t<kI8One, 16, GATED>(m, a, st);
  if (half == 32) return launch_t<kI8One, 32, GATED>(m, a, st);
  if (half == 64) return launch_t<kI8One, 64, GATED>(m, a, st);
  return half == 128 ? launch_t<kI8One, 128, GATED>(m, a, st) : cudaErrorInvalidValue;
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

cudaError_t launch_i8_tc(I8Kind kind, int half, bool gated, const I8TcMaps& m, const I8TcArgs& a,
                         cudaStream_t st) {
  return gated ? launch_half<true>(kind, half, m, a, st) : launch_half<false>(kind, half, m, a, st);
}

cudaError_t launch_i8_widen(const I8WidenArgs& a, cudaStream_t st) {
  const long long n = (long long)a.rows * (a.pitch / 16);
  return launch_pdl(i8_widen_kernel, dim3((unsigned)((n + 255) / 256)), 256, 0, st, a);
}

cudaError_t launch_i8_split_sum(I8Kind kind, int half, bool gated, const I8TcArgs& a, cudaStream_t st) {
  const int rows = half * (kind == kI8Two ? 2 : 1), per = gated ? 4 : 2;
  const dim3 grid((unsigned)(a.m_tiles * a.n_tiles * ((rows + per - 1) / per)));
  return gated ? launch_pdl(i8_split_sum_kernel<true>, grid, 256, 0, st, a, rows)
               : launch_pdl(i8_split_sum_kernel<false>, grid, 256, 0, st, a, rows);
}

}  // namespace moe
