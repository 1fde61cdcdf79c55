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
// gate and the same 64 of up, 16 and 16 in turn in TMEM), the tokens the n side.
// Weights come by TMA as 8-bit codes, 128 x 128 a step; eight warps widen them,
// a thread half a row or a row of every second step, and write them to TMEM, from
// where tcgen05.mma takes its first operand: the widened weights cost no shared
// memory traffic. Up to 16 tokens are few bytes
// beside the weights, and the same warps widen them into shared memory on the
// way; more are widened once, by a launch before this one, into the workspace,
// and come by TMA as fp16 (us, on the way / before: 16 x 4096 x 4096 9.7 / 10.6,
// 32 x 2048 x 2048 7.9 / 8.4, but 32 x 4096 x 14336 20.0 / 18.5, 64 x 4096 x 14336
// 25.4 / 20.6).
//
// Two threads issue the MMAs: what an issuer does between two steps (two waits,
// two commits) takes longer than the step's MMAs leave. With one block of tokens
// (kI8One) they take the steps in turn, with two (kI8Two) a block each, and each
// sums on its own. Their sums rotate through three accumulators, so that one is
// read back while two fill (two accumulators left the tensor core idle for the
// read-back, some 1400 cycles of the 8200 that 1024 k take).
//
// Warps: 0 brings weights, 3 tokens, 1 and 2 issue, 4-11 widen, 12-19 read back,
// scale and store. Gated, the two lanes of a warp that hold a column's gate and
// its up sums give each other half of them.
//
// Bound for few tokens by the weights' stream (5.6 TB/s once it runs, 128 of 152 SMs
// having a share of 4096 weight rows; start and end of the kernel are 7 us: 64 x 4096 x
// 14336 19.5 us, gated 64 x 14336 x 4096 28.9-29.4),
// for many by the hand-overs between widening, issue and read-back: a step's MMAs
// are 1024 cycles, an issuer's waits, issues and commits some 1100 (8192 x 14336 x
// 4096 553-574 us with 18 of widening, 1.68-1.74 PFLOP/s; gated 2048 x 14336 x 4096
// 285-300 us, 1.6-1.7; the tensor pipe busy for 75 % of the cycles), and where sums are
// short by the epilogue's stores, 32 columns of a token an instruction (5632 x 8432 x 384
// in fp32 50 us, 31 without them; 8192 x 14336 x 128 91, floor 35). Between these, 65 to
// about 1000 tokens, by what a tile is: with one block of tokens a slot of widened weights
// serves half the MMAs, and a tile is cut over a whole cluster or not at all (512 x 4096
// x 4096 24.1 us, floor 9.1; 256 x 14336 x 4096 29.6, floor 15.9).
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
// Launched with 96 registers a thread, 61,440 in all, which the warps share out
// anew: kI8Two 128 x 48 + 256 x 56 + 256 x 160 (128 sums a thread of the
// epilogue) = 61,440, kI8One 128 x 64 + 256 x 80 + 256 x 120 = 59,392.
static_assert(kChunk * kStep * 128 * 128 <= 1 << 24, "a chunk's sums are exact in fp32");

template <int HALF>
struct Plan {
  // TMEM: accumulators, then widened weights (64 columns: 128 k of fp16 pairs)
  static constexpr uint32_t kAccCols = HALF == 128 ? 128 : 64;
  static constexpr uint32_t kSlotCol0 = HALF == 128 ? 384 : 256;
  static constexpr int kSlots = HALF == 128 ? 2 : 4;
  // stages of the two rings, up to about 200 KB
  static constexpr int kStageT = HALF * kStep * 2;
  // Few tokens are widened by this kernel, into stages that go with the slots of
  // widened weights.
  static constexpr bool kFused = HALF <= kI8FusedRows;
  static constexpr int kT = kFused || HALF == 128 ? 4 : HALF == 64 ? 6 : 8;
  static constexpr int kW = HALF == 128 ? 4 : HALF == 64 ? 6 : HALF == 32 ? 8 : 10;
  static_assert(!kFused || kT == kSlots, "a stage of tokens per slot");
  static constexpr int kCols = HALF / 2;  // columns of an accumulator that an epilogue warp reads
  static constexpr size_t kToken = 0;
  static constexpr size_t kWeight = kToken + (size_t)kT * kStageT;
  static constexpr size_t kScale = kWeight + (size_t)kW * kStageW;  // [epilogue warp][128] scales of rows of A
  static constexpr size_t kBars = kScale + kEpiWarps * 128 * 4;
  static constexpr size_t kBytes = 1024 + kBars + (2 * kT + 2 * kW + 2 * kSlots + 2 * kAccs) * 8 + 16;
  static_assert(kAccs * kAccCols <= kSlotCol0 && kSlotCol0 + kSlots * kSlotCols <= kTmemCols, "TMEM plan");
  static_assert(kT % 2 == 0 && kW % 2 == 0 && kSlots % 2 == 0, "every second stage is one issuer's, one widening group's");
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

// What a CTA works off: a.waves whole tiles; then, of the a.cut tiles that are
// left, a cluster one, whose CTAs share its steps evenly.
struct Item {
  int mt, nt;     // tile of rows of A, tile of weight rows
  int kb0, kb1;   // steps
  bool part;      // of a tile
};
// Tiles go in bands of 8 token tiles, weight tile by weight tile, so that the
// CTAs in flight share both operands through L2.
constexpr int kBand = 8;
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
struct Walk {
  int i = 0;
  __device__ __forceinline__ bool next(const I8TcArgs& a, Item& it) {
    int tile = i * gridDim.x + blockIdx.x;
    it.kb0 = 0;
    it.kb1 = a.steps;
    it.part = false;
    if (i >= a.waves) {
      const int mine = blockIdx.x / a.ks;
      if (i > a.waves || mine >= a.cut) return false;
      tile = i * gridDim.x + mine;
      const int rank = cluster_rank();
      it.kb0 = rank * a.steps / a.ks;
      it.kb1 = (rank + 1) * a.steps / a.ks;
      it.part = true;
    }
    ++i;
    if (tile >= a.m_tiles * a.n_tiles) return false;  // (the last wave need not be full)
    const int span = kBand * a.n_tiles, band = tile / span, w = tile - band * span;
    const int width = min(kBand, a.m_tiles - band * kBand);
    it.mt = band * kBand + w % width;
    it.nt = w / width;
    return true;
  }
};
constexpr int kMaxCluster = 8;
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Four 32-bit values at this CTA's shared address `addr` in the cluster's CTA `rank`.
__device__ __forceinline__ int4 ld_cluster4(uint32_t addr, int rank) {
  int4 v;
  asm volatile(
      "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %4, %5;\n"
      " ld.shared::cluster.v4.s32 {%0,%1,%2,%3}, [a];\n}"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}

// Gated: the output that row r of a tile holds the gate or the up sum of.
__device__ __forceinline__ int out_of_row(int r) { return (r >> 5) * 16 + (r & 15); }

// Accumulators that an item of n steps fills: eight steps each, the two issuers'
// in turn (kI8One: every second step each, so that a lone last step is that of
// the issuer with the item's first).
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
// A ring's place, of N stages, and its phase's parity, after any number of steps
// of `by` stages (which divides N).
template <int N>
struct Place {
  int at;
  uint32_t ph = 0;
  __device__ __forceinline__ explicit Place(int first = 0) : at(first) {}
  __device__ __forceinline__ void next(int by = 1) {
    at += by;
    const bool round = at >= N;
    at -= round ? N : 0;
    ph ^= round ? 1u : 0u;
  }
};

// 16 codes at column k of N rows, 16 rows apart, of which `rows` exist (zeros
// past them and past column K).
template <int N>
__device__ __forceinline__ void load_codes(uint4 (&c)[N], const uint8_t* row, long long lda, int rows, int k, int K) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    c[i] = make_uint4(0u, 0u, 0u, 0u);
    if (16 * i < rows) {
      if (k + 16 <= K)
        c[i] = __ldg(reinterpret_cast<const uint4*>(row + 16 * i * lda + k));
      else
        c[i] = i8_load16(row + 16 * i * lda, k, K);
    }
  }
}

template <int KIND, int HALF, bool GATED, bool SHORT>
__global__ void __launch_bounds__(kThreads, 1)
    i8_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB0,
                 const __grid_constant__ CUtensorMap tmB1, const I8TcArgs a) {
  using P = Plan<HALF>;
  constexpr int kBlocks = KIND == kI8Two ? 2 : 1;  // token blocks of a tile
  // The eight widening warps share every step where the MMAs of a step take long
  // and a slot has to be filled soon after it came free; else four take every
  // second step, whose waits then overlap.
  constexpr bool kHalves = KIND == kI8Two;
  constexpr int kWideners = kHalves ? kConvWarps : kConvWarps / 2;
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
      mbar_init(&wempty[s], kWideners);
    }
    for (int s = 0; s < P::kSlots; ++s) {
      mbar_init(&sfull[s], kWideners);
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
  if (P::kFused) {
    pdl_wait();
    pdl_trigger();
  }

  if (warp < kConvWarp0) {
    if (KIND == kI8Two)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    else
      asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 0) {
      // --------------------------------------------------------------- weights
      // (Without kFused the weights here and the scales in the epilogue are read before
      // the wait for the kernel before this one: that is the same call's widening of the
      // tokens, which writes neither, and what is older has completed.)
      if (lane == 0) {
        Place<P::kW> p;
        bool alive = true;
        Item it;
        for (Walk walk; alive && walk.next(a, it);) {
          for (int kb = it.kb0; kb < it.kb1; ++kb) {
            if (!(alive = lane_wait(&wempty[p.at], p.ph ^ 1u, a, abort_flag))) break;
            uint8_t* dst = sW + p.at * kStageW;
            mbar_expect_tx(&wfull[p.at], kStageW);
            tma_load_2d(dst, &tmB0, &wfull[p.at], kb * kStep, it.nt * kOuts);
            if (GATED) tma_load_2d(dst + kStageW / 2, &tmB1, &wfull[p.at], kb * kStep, it.nt * kOuts);
            p.next();
          }
        }
      }
    } else if (warp == 3) {
      // ---------------------------------------------------------------- tokens
      if (!P::kFused) {
        pdl_wait();
        pdl_trigger();
        if (lane == 0) {
          Place<P::kT> p;
          bool alive = true;
          Item it;
          for (Walk walk; alive && walk.next(a, it);) {
            for (int kb = it.kb0; kb < it.kb1 && alive; ++kb) {
#pragma unroll
              for (int b = 0; b < kBlocks; ++b) {
                if (!(alive = lane_wait(&tempty[p.at], p.ph ^ 1u, a, abort_flag))) break;
                uint8_t* dst = sT + p.at * P::kStageT;
                const int row = (it.mt * kBlocks + b) * HALF;
                mbar_expect_tx(&tfull[p.at], P::kStageT);
                tma_load_2d(dst, &tmA, &tfull[p.at], kb * kStep, row);
                tma_load_2d(dst + P::kStageT / 2, &tmA, &tfull[p.at], kb * kStep + kStep / 2, row);
                p.next();
              }
            }
          }
        }
      }
    } else if (lane == 0) {
      // --------------------------------------------------------------- issuers
      // An issuer has a block of tokens (kI8Two), or the even or the odd steps of all
      // items together, and so every second stage and slot. (A barrier's parity tells
      // two phases apart: an issuer that came to a stage whose last use was the
      // other's could take the phase before that use for its own.) The issuer
      // with an item's first step has the item's first accumulator.
      const int me = warp - 1;
      constexpr int kBy = KIND == kI8Two ? 1 : 2;  // steps from one of its own to the next
      Place<P::kT> tp(me);
      Place<P::kSlots> sp(KIND == kI8Two ? 0 : me);
      int base = 0, done = 0;  // accumulators filled and steps made before this item
      // failure self-test: wait on a barrier that only this warp completes
      bool alive = !a.stall || lane_wait(&dfull[me], 0u, a, abort_flag);
      const uint64_t b0 = sw128_desc(smem_u32(sT));
      Item it;
      for (Walk walk; alive && walk.next(a, it);) {
        const int n = it.kb1 - it.kb0;
        const int second = KIND == kI8Two ? me : (me + done) & 1;
        int left = KIND == kI8Two ? n : (n + 1 - second) >> 1;  // own steps
        int acc = (base + second) % kAccs;
        uint32_t aph = ((base + second) / kAccs) & 1u;
        while (left > 0) {
          if (!(alive = lane_wait(&dempty[acc], aph ^ 1u, a, abort_flag))) break;
          const uint32_t d = tmem_base + acc * P::kAccCols;
          const int chunk = min(left, kChunk);
          for (int i = 0; i < chunk; ++i) {
            if (!(alive = lane_wait(&sfull[sp.at], sp.ph, a, abort_flag) &&
                          (P::kFused || lane_wait(&tfull[tp.at], tp.ph, a, abort_flag))))
              break;
            tc_fence_after();
            const uint32_t w = tmem_base + P::kSlotCol0 + sp.at * kSlotCols;
            const uint64_t b = b0 + tp.at * (P::kStageT >> 4);
            constexpr uint64_t kHalfStage = (P::kStageT / 2) >> 4;
#pragma unroll
            for (int k = 0; k < kStep / 16; ++k)  // 16 k: 8 columns of A, 32 bytes of B's rows
              mma_f16_ta(d, w + 8 * k, b + (k >> 2) * kHalfStage + 2 * (k & 3), kIdesc,
                         k != 0 ? 1u : (uint32_t)i);
            if (!P::kFused) mma_commit(&tempty[tp.at]);
            mma_commit(&sempty[sp.at]);
            tp.next(2);
            sp.next(kBy);
          }
          if (!alive) break;
          mma_commit(&dfull[acc]);
          left -= chunk;
          // two accumulators on, of three
          aph ^= acc ? 1u : 0u;
          acc = acc ? acc - 1 : 2;
        }
        base += accs_of<KIND>(n);
        done += n;
      }
    }
    __syncwarp();
  } else if (warp < kEpiWarp0) {
    if (KIND == kI8Two)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    else
      asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    // ------------------------------------------------------------------- widen
    // this thread's TMEM lane is 32 (warp % 4) + lane, its weight row as it lies in
    // the stage the same, or gated (gate's rows before up's) as out_of_row says
    const int r = GATED ? out_of_row((warp & 3) * 32 + lane) + (lane & 16) * 4 : (warp & 3) * 32 + lane;
    const int group = (warp - kConvWarp0) >> 2;   // its half of every step's k, or of the steps
    const uint32_t tq = tmem_base + ((uint32_t)((warp & 3) * 32) << 16) + P::kSlotCol0;
    Place<P::kW> wp(kHalves ? 0 : group);
    Place<P::kSlots> sp(kHalves ? 0 : group);
    int done = 0;
    bool alive = true;
    Item it;
    // kFused: 16 codes of a step of every 16th token, eight lanes a token, so that a
    // load touches four lines
    constexpr int kTok = P::kFused ? HALF / 16 : 1;
    const int tok = (threadIdx.x & 127) >> 3, piece = threadIdx.x & 7;
    uint4 codes[kTok];
    for (Walk walk; alive && walk.next(a, it);) {
      const int n = it.kb1 - it.kb0;
      const int first = (group + done) & 1;
      const uint8_t* tokens = nullptr;
      int k = 0, rows = 0;
      if (P::kFused) {
        rows = a.M - it.mt * HALF - tok;
        tokens = a.a + (long long)(it.mt * HALF + tok) * a.lda;
        k = (it.kb0 + first) * kStep + piece * 16;
        if (first < n) load_codes(codes, tokens, a.lda, rows, k, a.K);
      }
      for (int left = kHalves ? n : (n + 1 - first) >> 1; left > 0; --left) {
        if (!(alive = warp_wait(&wfull[wp.at], wp.ph, a, abort_flag))) break;
        const uint8_t* row = sW + wp.at * kStageW + r * kStep;
#pragma unroll
        for (int z = 0; z < (kHalves ? 1 : 2); ++z) {
          const int h = kHalves ? group : z;
          uint32_t v[32];
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // 16-byte pieces, swizzled by the row
            const uint4 w = ld_shared_v4(row + (((h * 4 + c) ^ (r & 7)) << 4));
            i8_to_f16(w.x, v[8 * c], v[8 * c + 1]);
            i8_to_f16(w.y, v[8 * c + 2], v[8 * c + 3]);
            i8_to_f16(w.z, v[8 * c + 4], v[8 * c + 5]);
            i8_to_f16(w.w, v[8 * c + 6], v[8 * c + 7]);
          }
          if (kHalves || z == 1) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&wempty[wp.at]);
          }
          if (z == 0) {
            if (!(alive = warp_wait(&sempty[sp.at], sp.ph ^ 1u, a, abort_flag))) break;
            tc_fence_after();
          }
          tmem_st32(tq + sp.at * kSlotCols + h * (kSlotCols / 2), v);
        }
        if (!alive) break;
        if (P::kFused) {
          // fp16 rows of 128 bytes, their pieces of eight values swizzled by the row;
          // the second 64 k behind the first. Lanes of the one and of the other write
          // their two pieces in opposite order, to different banks.
          const int swap = piece >> 2;
          uint8_t* stage = sT + sp.at * P::kStageT + swap * (P::kStageT / 2) + tok * 128;
          const int at = (piece & 3) * 2;
#pragma unroll
          for (int i = 0; i < kTok; ++i) {
            const uint4 w = codes[i];
            uint32_t v[8];
            i8_to_f16(w.x, v[0], v[1]);
            i8_to_f16(w.y, v[2], v[3]);
            i8_to_f16(w.z, v[4], v[5]);
            i8_to_f16(w.w, v[6], v[7]);
            uint8_t* box = stage + i * 16 * 128;  // (16 rows on the swizzle is the same)
            uint8_t* p0 = box + ((at ^ (tok & 7)) << 4);
            uint8_t* p1 = box + (((at + 1) ^ (tok & 7)) << 4);
            st_shared_v4(swap ? p1 : p0, swap ? v[4] : v[0], swap ? v[5] : v[1], swap ? v[6] : v[2],
                         swap ? v[7] : v[3]);
            st_shared_v4(swap ? p0 : p1, swap ? v[0] : v[4], swap ? v[1] : v[5], swap ? v[2] : v[6],
                         swap ? v[3] : v[7]);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          k += 2 * kStep;
          if (left > 1) load_codes(codes, tokens, a.lda, rows, k, a.K);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sfull[sp.at]);
        wp.next(kHalves ? 1 : 2);
        sp.next(kHalves ? 1 : 2);
      }
      done += n;
    }
  } else {
    if (KIND == kI8Two)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
    else
      asm volatile("setmaxnreg.inc.sync.aligned.u32 120;");
    // ---------------------------------------------------------------- epilogue
    constexpr int kCols = P::kCols;
    constexpr int kPiece = kCols < 16 ? 8 : 16;
    const int mine = warp - kEpiWarp0, part = mine >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t tq = tmem_base + ((uint32_t)((warp & 3) * 32) << 16) + part * kCols;
    float* scale = reinterpret_cast<float*>(smem + P::kScale) + mine * 128;
    const bool up = GATED && (lane & 16) != 0;  // this lane's row is up's
    // What becomes of an accumulator's sums, whole numbers up to 2^24: SHORT (K up to
    // 1024) they are final, for kI8One after the other accumulator's are added, and
    // stay fp32 (bits in `sum`); else they are added as integers.
    const auto value = [](int sum, float sa, float sb) {
      return SHORT ? __int_as_float(sum) * sa * sb : i8_value(sum, sa, sb);
    };
    int use = 0;
    bool alive = true;
    Item it;
    for (Walk walk; alive && walk.next(a, it);) {
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
            if (SHORT) {
#pragma unroll
              for (int j = 0; j < kPiece; ++j) {
                int& to = sum[s][c * kPiece + j];
                to = __float_as_int(__int_as_float(to) + __uint_as_float(v[j]));
              }
            } else {
#pragma unroll
              for (int j = 0; j < kPiece; ++j)
                sum[s][c * kPiece + j] += __float2int_rn(__uint_as_float(v[j]));
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&dempty[acc]);
          ++use;
        }
      }
      if (!alive) break;
      if (it.part) {
        // its sums, for the cluster's CTAs, in the rings' place, which nothing
        // uses any more: [column][row]
        int* dst = reinterpret_cast<int*>(smem) + part * kCols * kRows + r;
#pragma unroll
        for (int s = 0; s < kBlocks; ++s)
#pragma unroll
          for (int j = 0; j < kCols; ++j)
            dst[(s * HALF + j) * kRows] = SHORT ? __float2int_rn(__int_as_float(sum[s][j])) : sum[s][j];
        break;
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
                  y[i] = value(sum[s][j + i], sa.x, b0);
                  y[i + 1] = value(sum[s][j + i + 1], sa.y, b0);
                  y[i + 2] = value(sum[s][j + i + 2], sa.z, b0);
                  y[i + 3] = value(sum[s][j + i + 3], sa.w, b0);
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
                const float g = value(up ? other : own, sa, b0);
                y[j] = siluf_(g) * value(up ? own : other, sa, b1);
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
  __syncwarp();
  // A cut tile: each of the cluster's CTAs adds and finishes its share of the
  // tokens. (Every thread of the cluster comes here, after a wait that ran out
  // too.) A warp takes a token at a time, a lane four rows of the tile.
  if ((int)(blockIdx.x / a.ks) < a.cut) {
    const int rank = cluster_rank(), r = lane * 4;
    const int tile = a.waves * gridDim.x + blockIdx.x / a.ks;
    const int span = kBand * a.n_tiles, band = tile / span, w = tile - band * span;
    const int width = min(kBand, a.m_tiles - band * kBand);
    const int m0 = (band * kBand + w % width) * kBlocks * HALF;
    // gated, the lane with a column's gate sums finishes the first two of the four,
    // the lane with its up sums the others
    const bool up = GATED && (lane & 4) != 0;
    constexpr int kMine = GATED ? 2 : 4;
    const int n = w / width * kOuts + (GATED ? out_of_row(r) + (up ? 2 : 0) : r);
    const int cols = min(kBlocks * HALF, a.M - m0);  // tokens of the tile that exist
    const int c0 = rank * cols / a.ks, c1 = (rank + 1) * cols / a.ks;
    float b0[kMine], b1[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const bool in = warp >= kEpiWarp0 && n + i < a.N;
      b0[i] = in ? a.b_scale0[n + i] : 0.f;
      b1[i] = GATED && in ? a.b_scale1[n + i] : 0.f;
    }
    cluster_sync();
    for (int c = c0 + warp - kEpiWarp0; warp >= kEpiWarp0 && c < c1; c += kEpiWarps) {
      const float sa = a.a_scale[m0 + c];
      const uint32_t at = smem_u32(smem) + (uint32_t)(c * kRows + r) * 4;
      int4 v[kMaxCluster];
#pragma unroll
      for (int z = 0; z < kMaxCluster; ++z)
        v[z] = z < a.ks ? ld_cluster4(at, z) : make_int4(0, 0, 0, 0);
      int sum[4] = {0, 0, 0, 0};
#pragma unroll
      for (int z = 0; z < kMaxCluster; ++z) {
        sum[0] += v[z].x;
        sum[1] += v[z].y;
        sum[2] += v[z].z;
        sum[3] += v[z].w;
      }
      const size_t at_out = (size_t)(m0 + c) * a.ldo + n;
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        float y;
        if (GATED) {
          const int other = __shfl_xor_sync(0xffffffffu, up ? sum[i] : sum[i + 2], 4), own = up ? sum[i + 2] : sum[i];
          y = siluf_(i8_value(up ? other : own, sa, b0[i])) * i8_value(up ? own : other, sa, b1[i]);
        } else {
          y = i8_value(sum[i], sa, b0[i]);
        }
        if (n + i < a.N) i8_store(a.out, at_out + i, a.out_bf16, y);
      }
    }
    cluster_sync();
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

// Rows of codes as fp16, 16 a thread. i8_tc reads weights and scales before it waits for
// this kernel: its trigger stays behind its own wait, and it writes the widened rows only.
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

constexpr int kCutCost = 5;  // of a cut tile's end, in steps

// Clusters of ks CTAs that fit the device at a time.
template <int KIND, int HALF, bool GATED, bool SHORT>
int clusters_of(int dev, int ks) {
  static int known[64][kMaxCluster + 1] = {};
  if (known[dev][ks] == 0) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(tc_sm_count() / ks * ks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Plan<HALF>::kBytes;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, i8_tc_kernel<KIND, HALF, GATED, SHORT>, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();
      n = -1;  // none
    }
    known[dev][ks] = n;
  }
  return known[dev][ks];
}

template <int KIND, int HALF, bool GATED, bool SHORT>
cudaError_t launch_t(const I8TcMaps& m, I8TcArgs a, cudaStream_t st) {
  static int attr[64] = {};
  const auto kernel = i8_tc_kernel<KIND, HALF, GATED, SHORT>;
  cudaError_t e = ensure_smem_limit(kernel, (int)Plan<HALF>::kBytes, attr);
  if (e != cudaSuccess) return e;
  // Whole tiles in waves over the SMs; or clusters of ks CTAs, and what is left after
  // the full waves cut over a cluster each, where that ends sooner.
  const int tiles = a.m_tiles * a.n_tiles, sms = tc_sm_count();
  int dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;  // (below 64: ensure_smem_limit)
  a.ks = 1;
  a.cut = 0;
  a.waves = (tiles + sms - 1) / sms;
  int grid = tiles < sms ? tiles : sms;
  long long best = (long long)a.waves * a.steps;
  for (int ks = 2; ks <= kMaxCluster && 2 * ks <= a.steps && a.waves <= 3; ++ks) {
    const int fit = clusters_of<KIND, HALF, GATED, SHORT>(dev, ks);
    if (fit < 1) continue;
    const int waves = tiles / (fit * ks), rest = tiles - waves * fit * ks;
    if (rest == 0 || rest > fit) continue;
    const long long t = (long long)waves * a.steps + (a.steps + ks - 1) / ks + kCutCost;
    if (t < best) {
      best = t;
      a.ks = ks;
      a.cut = rest;
      grid = (waves ? fit : rest) * ks;
    }
  }
  if (a.cut) a.waves = (tiles - a.cut) / grid;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = a.ks;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Plan<HALF>::kBytes;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, m.A, m.B0, m.B1, a);
}
// A kernel of its own for K of up to 1024, where blocks are large and the
// epilogue is what takes the time (8192 x 14336 x 128 112 -> 92 us, 2048 x 14336 x
// 512 gated 83 -> 75; asked at run time, it slowed long sums by 2.6 %).
template <int KIND, bool GATED>
cudaError_t launch_128(const I8TcMaps& m, const I8TcArgs& a, cudaStream_t st) {
  return a.steps <= kChunk ? launch_t<KIND, 128, GATED, true>(m, a, st) : launch_t<KIND, 128, GATED, false>(m, a, st);
}
template <bool GATED>
cudaError_t launch_half(I8Kind kind, int half, const I8TcMaps& m, const I8TcArgs& a, cudaStream_t st) {
  if (kind == kI8Two) return half == 128 ? launch_128<kI8Two, GATED>(m, a, st) : cudaErrorInvalidValue;
  if (half == 16) return launch_t<kI8One, 16, GATED, false>(m, a, st);
  if (half == 32) return launch_t<kI8One, 32, GATED, false>(m, a, st);
  if (half == 64) return launch_t<kI8One, 64, GATED, false>(m, a, st);
  return half == 128 ? launch_128<kI8One, GATED>(m, a, st) : cudaErrorInvalidValue;
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

}  // namespace moe
