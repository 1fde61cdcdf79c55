// The 8-bit layer for a few tokens, and the 8-bit product for a few rows:
// weight streams on mma.sync (e4m3 x e4m3 -> fp32).
//
// A few tokens meet every weight byte once, so these kernels are bound by
// HBM and, for one token, by latency. mma.sync m16n8k32 takes 16 weight rows
// as its m side and up to 8 tokens as its n side. A contraction does not care
// in which order k is visited as long as both operands agree, so a lane's
// fragment registers are simply 16-byte pieces of the rows: no conversion, no
// shuffles. Every warp owns a ring of slots that its lane 0 fills by TMA
// (128-byte swizzle). Such a stream loses to the latencies of a warp's walk
// through a slot and to instruction issue before it loses to HBM (an SM has
// some 350 issue slots for every 2 KB that HBM brings it). So a slot holds two
// blocks of k, a gate/up item two m16 tiles, and the loops exist once, compact:
// at one token a kernel fetches each of its instructions for a use or two.
// (Single blocks and tiles, whether loaded into registers, by cp.async or by
// TMA, took 280 instructions per 2 KB, 3 TB/s at 8 tokens of the 256-expert
// shape.)
//
// Measured, weights rotated beyond L2: 256 experts, one token 15.3 us (28 MB;
// latency of two dependent kernels, 5 us of them before the first weight
// lands), 8 tokens 48.4 us (3.8 TB/s), 16 tokens 78.6 us; 8 wide experts, 4 tokens
// 182 us (5.3 TB/s); products 1 x 5632 x 2048 5.5 us, 8 x 4096 x 14336 16.6 us.
//
// The products of one 128-wide block are summed by the tensor core and then
// scaled by the block's two scales into fp32 sums held in registers.
//
// The layer takes two kernels:
//  1. f8_few_gateup: every CTA groups the (token, slot) pairs by expert into
//     chunks of at most 8 (ranking by counting), quantises the tokens into
//     shared memory, then takes items of 16 gate and 16 up rows of a chunk's
//     expert (eight and eight make an m16 tile, so that a lane holds a row's
//     gate and up sums). The warps split k; their sums are added in warp order.
//     h needs one scale per 128 columns, which 8 items share: the item that
//     finishes a block last (a counter that it also resets) quantises it.
//  2. f8_few_down: a CTA owns 16 output columns of every chunk and adds the
//     slots, the shared expert and the residual in a fixed order.
#include "fp8_common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr int kFewMaxPairs = 512;  // 16 tokens of at most 32 slots

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// One block of 128 k: rows g and g + 8 of the m16 tile, two 16-byte pieces
// each (k 16 t.. and k 64 + 16 t.. for t = lane % 4).
struct WeightBlock {
  uint4 lo[2], hi[2];
};

// The four steps of 32 k, from zero each and added afterwards: a chain through
// the accumulator waits 73 cycles a step, independent ones follow every 14.
struct BlockSum {
  float d[4][4];
  __device__ __forceinline__ void mma(const WeightBlock& w, const uint4& b0, const uint4& b1) {
    mma_e4m3(d[0], w.lo[0].x, w.hi[0].x, w.lo[0].y, w.hi[0].y, b0.x, b0.y);
    mma_e4m3(d[1], w.lo[0].z, w.hi[0].z, w.lo[0].w, w.hi[0].w, b0.z, b0.w);
    mma_e4m3(d[2], w.lo[1].x, w.hi[1].x, w.lo[1].y, w.hi[1].y, b1.x, b1.y);
    mma_e4m3(d[3], w.lo[1].z, w.hi[1].z, w.lo[1].w, w.hi[1].w, b1.z, b1.w);
  }
  __device__ __forceinline__ float of(int i) const { return (d[0][i] + d[1][i]) + (d[2][i] + d[3][i]); }
};

__device__ __forceinline__ uint4 zero4() { return make_uint4(0u, 0u, 0u, 0u); }

// Scales come by 4-byte asynchronous copies (or as zero); each copying lane
// arrives on the slot's barrier once its copy has landed.
__device__ __forceinline__ void copy4(float* dst, const float* src, uint64_t* bar, bool valid = true) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(tc::smem_u32(dst)), "l"(src),
               "r"(valid ? 4 : 0)
               : "memory");
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}
template <int OFF>
__device__ __forceinline__ uint4 lds16(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4 + %5];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(src), "n"(OFF)
               : "memory");
  return v;
}
template <int OFF>
__device__ __forceinline__ float lds4(uint32_t src) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1 + %2];" : "=f"(v) : "r"(src), "n"(OFF) : "memory");
  return v;
}
// The generic reads of a slot come before the copies that refill it.
__device__ __forceinline__ void reads_before_refill() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Arrivals that complete slot i's barrier. Failure self-test: the first slot of
// the first warp waits for one that never comes.
__device__ __forceinline__ uint32_t few_arrivals(uint32_t n, int i, int stall) {
  return n + (stall && i == 0 ? 1u : 0u);
}

// A box of rows of 128 bytes, 1024-byte aligned; TMA puts piece p (16 bytes) of
// row r at p ^ (r % 8).
constexpr int kBox8 = 1024, kBox16 = 2048;
// A lane's pieces t and t + 4 of row g lie at get and get ^ 64.
__device__ __forceinline__ uint32_t get_at(int g, int t) { return (uint32_t)(g * 128 + ((t ^ g) << 4)); }

// The m16 tile of eight rows at `lo` and eight at `hi` (box rows, shared memory).
__device__ __forceinline__ WeightBlock weights_of(uint32_t lo, uint32_t hi, uint32_t get) {
  WeightBlock w;
  w.lo[0] = lds16<0>(lo + get);
  w.lo[1] = lds16<0>(lo + (get ^ 64u));
  w.hi[0] = lds16<0>(hi + get);
  w.hi[1] = lds16<0>(hi + (get ^ 64u));
  return w;
}

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~static_cast<uintptr_t>(1023));
}

// ---------------------------------------------------------------------------
// chunks of at most 8 pairs of one expert, then of 8 tokens for the shared one
// ---------------------------------------------------------------------------
struct FewLists {
  alignas(16) short ids[kFewMaxPairs];
  short sorted[kFewMaxPairs];          // position -> pair
  short pos[kFewMaxPairs];             // pair -> position
  short token[kFewMaxPairs];           // position -> token
  short start[kFewMaxPairs + 8];       // chunk -> first position (shared: first token)
  short expert[kFewMaxPairs + 8];      // chunk -> expert (E: shared)
  short count[kFewMaxPairs + 8];       // chunk -> pairs in it
  unsigned char first[kFewMaxPairs];   // position starts a chunk
  int n_routed, n_chunks;
};

// Positions order the pairs by (expert, pair). The first N threads of the CTA
// call it; it ends with a barrier of them.
template <int N>
__device__ __forceinline__ void lists_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory");
}
// The shared expert's chunks, after the n routed ones (one warp calls it).
__device__ __forceinline__ void finish_lists(const F8ExpertsArgs& a, FewLists& L, int n, int lane) {
  const int ns = a.Is > 0 ? (a.T + 7) / 8 : 0;
  if (lane < ns) {
    L.start[n + lane] = (short)(8 * lane);
    L.expert[n + lane] = (short)a.E;
    L.count[n + lane] = (short)min(8, a.T - 8 * lane);
  }
  if (lane == 0) {
    L.n_routed = n;
    L.n_chunks = n + ns;
  }
}
template <int N>
__device__ __forceinline__ void build_lists(const F8ExpertsArgs& a, FewLists& L) {
  const int P = a.T * a.k, tid = threadIdx.x, lane = tid & 31;
  bool bad = false;
  for (int i = tid; i < ((P + 7) & ~7); i += N) {
    int e = i < P ? __ldcg(a.ids + i) : 0x7FFF;
    if (i < P && (e < 0 || e >= a.E)) {
      bad = true;
      e = a.E - 1;
    }
    L.ids[i] = (short)e;
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) report(a.ctrl, kDevBadId, kSiteFewFp8);
  lists_sync<N>();
  for (int i = tid; i < P; i += N) {
    const int e = L.ids[i];
    int below = 0, same = 0;
    for (int j = 0; j < P; j += 8) {
      const uint4 o = *reinterpret_cast<const uint4*>(L.ids + j);
      const uint32_t v[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int id = (int)((v[q >> 1] >> (16 * (q & 1))) & 0xFFFFu);
        below += id < e;
        same += id == e && j + q < i;
      }
    }
    L.sorted[below + same] = (short)i;
    L.pos[i] = (short)(below + same);
    L.token[below + same] = (short)(i / a.k);
    L.first[below + same] = (same & 7) == 0;
  }
  lists_sync<N>();
  if (tid < 32) {
    int n = 0;
    for (int r0 = 0; r0 < P; r0 += 32) {
      const bool f = r0 + lane < P && L.first[r0 + lane];
      const unsigned m = __ballot_sync(0xffffffffu, f);
      if (f) {
        const int c = n + __popc(m & ((1u << lane) - 1u));
        L.start[c] = (short)(r0 + lane);
        L.expert[c] = L.ids[L.sorted[r0 + lane]];
      }
      n += __popc(m);
    }
    __syncwarp();
    for (int c = lane; c < n; c += 32) L.count[c] = (short)((c + 1 < n ? L.start[c + 1] : P) - L.start[c]);
    finish_lists(a, L, n, lane);
  }
  lists_sync<N>();
}

// ---------------------------------------------------------------------------
// 1. gate/up
// ---------------------------------------------------------------------------
// Eight streaming warps share an item (16 gate and 16 up rows of a chunk's
// expert) along k, two blocks of 128 each: whole rows are in flight at a time,
// which DRAM's pages want. Rows shorter than sixteen blocks are shared by fewer
// warps, and more items are in flight. Four finishing warps take the items in
// turn: one adds an item's partial sums, applies SwiGLU, stores h and counts
// the block's items, so that the streaming warps never wait for a store, a
// fence or an atomic (with a streaming warp finishing each item behind a CTA
// barrier, 8 tokens of the 256-expert shape took 102 us here).
constexpr int kGuWarps = 8, kGuFinish = 4;
constexpr int kGuThreads = 32 * (kGuWarps + kGuFinish);
constexpr int kGuRows = 16;                   // rows of gate, and of up, in an item
constexpr int kGuAhead = 2;                   // slots per warp: 128 KB per SM
constexpr int kGuSlot = 4 * kBox16;           // gate and up of two blocks
constexpr int kGuArrivals = 5;                // the boxes' bytes, four scales

// SLOTS: items of a group between its warps and the finishers; four where
// shared memory has room beside the tokens' codes, else two.
template <int SLOTS>
struct GuShared {
  uint8_t ring[kGuWarps][kGuAhead][kGuSlot];
  float4 part[SLOTS][kGuWarps][2][32];
  uint64_t landed[kGuWarps][kGuAhead];
  uint64_t full[SLOTS][kGuWarps], empty[SLOTS][kGuWarps];  // by group
  float scale[kGuWarps][kGuAhead][4];                      // gate, up of two blocks
  FewLists lists;
  alignas(16) float xs[1];  // [T][KB], then the codes
};

template <int SLOTS>
__global__ void __launch_bounds__(kGuThreads, 1)
    f8_few_gateup_kernel(const __grid_constant__ CUtensorMap tmG, const __grid_constant__ CUtensorMap tmU,
                         const __grid_constant__ CUtensorMap tmSG, const __grid_constant__ CUtensorMap tmSU,
                         const F8ExpertsArgs a) {
  extern __shared__ uint8_t smem_raw[];
  GuShared<SLOTS>& S = *reinterpret_cast<GuShared<SLOTS>*>(align1024(smem_raw));
  FewLists& L = S.lists;
  const int KB = f8_blocks(a.d);
  float* xs = S.xs;                        // [T][KB]
  const int xstride = KB * kF8Block + 64;  // rows 64 B apart modulo the banks' 128 B
  uint8_t* xq = reinterpret_cast<uint8_t*>(xs) + ((a.T * KB * 4 + 15) & ~15);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int pairs = (KB + 1) / 2;
  const int nsplit = pairs >= 8 ? 8 : (pairs >= 4 ? 4 : 2);  // warps of an item
  const int groups = kGuWarps / nsplit;
  if (tid == 0) {
    for (int i = 0; i < kGuWarps * SLOTS; ++i) {
      tc::mbar_init(&S.full[0][0] + i, nsplit);
      tc::mbar_init(&S.empty[0][0] + i, 1);
    }
    for (int i = 0; i < kGuWarps * kGuAhead; ++i)
      tc::mbar_init(&S.landed[0][0] + i, few_arrivals(kGuArrivals, i, a.stall));
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();
  pdl_trigger();  // (not before the wait: f8_few_down relies on it)

  // item i: 16 rows `rb` of chunk `c`; a group's items are `stride` apart
  const int RB = a.I / kGuRows, RBs = a.Is / kGuRows;
  const int stride = (int)gridDim.x * groups;
  struct Walk {
    int i, c, rb;
  };
  auto settle = [&](Walk& k) {  // chunk and rows of item k.i
    const int routed = L.n_routed * RB;
    if (k.i < routed) {
      k.c = k.i / RB;
      k.rb = k.i - k.c * RB;
    } else if (RBs) {
      const int j = k.i - routed;
      k.c = L.n_routed + j / RBs;
      k.rb = j - j / RBs * RBs;
    }
  };
  const int step_c = stride / RB, step_rb = stride - step_c * RB;
  auto advance = [&](Walk& k) {
    k.i += stride;
    k.c += step_c;
    k.rb += step_rb;
    if (k.rb >= RB) {
      k.rb -= RB;
      ++k.c;
    }
    if (k.c >= L.n_routed) settle(k);  // among or past the shared expert's
  };
  auto item_count = [&]() { return L.n_routed * RB + (L.n_chunks - L.n_routed) * RBs; };

  if (warp < kGuWarps) {
    const int group = warp / nsplit, w = warp % nsplit;
    build_lists<kGuWarps * 32>(a, L);
    const int items = item_count();
    Walk now{group * (int)gridDim.x + (int)blockIdx.x, 0, 0};
    settle(now);
    // One loop fills slots and works them off, so that every piece of its code
    // exists once: a call of one token runs each instruction once or twice, and
    // fetching them is much of its time.
    Walk ahead = now;  // the loads' walk, kGuAhead slots ahead of the arithmetic's
    const int steps = (pairs - w + nsplit - 1) / nsplit;  // pairs of blocks of an item for this warp
    const CUtensorMap *mg = &tmG, *mu = &tmU;
    const float* ps = a.Sg;  // lanes 0, 1: gate's scales, lanes 2, 3: up's
    int todo = 0, row = 0, kb = 0, filled = 0, jf = 0;
    uint8_t* ring = S.ring[warp][0];
    float acc[2][4] = {};
    const uint32_t get = get_at(g, t);
    const uint32_t xq32 = tc::smem_u32(xq) + 2 * w * kF8Block + 16 * t, xs32 = tc::smem_u32(xs) + 8 * w;
    const uint32_t ring32 = tc::smem_u32(ring), sc32 = tc::smem_u32(S.scale[warp]);
    uint32_t xr = 0, x0 = 0, x1 = 0, ph = 0;
    int left = 0, r = 0, j = 0, kx = 0;
    bool codes = false;
    while (true) {
      if (filled < kGuAhead && ahead.i < items && steps) {
        if (todo == 0) {  // a new item
          const int e = L.expert[ahead.c];
          const bool sh = e == a.E;
          const int rows = sh ? a.Is : a.I;
          todo = steps;
          row = (sh ? 0 : e * rows) + ahead.rb * kGuRows;
          kb = 2 * w;
          mg = sh ? &tmSG : &tmG;
          mu = sh ? &tmSU : &tmU;
          const int si = ((sh ? 0 : e * f8_blocks(rows)) + ahead.rb * kGuRows / kF8Block) * KB;
          ps = (sh ? (lane & 2 ? a.Ssu : a.Ssg) : (lane & 2 ? a.Su : a.Sg)) + si;
        }
        uint64_t* bar = &S.landed[warp][jf];
        if (lane == 0) {
          uint8_t* dst = ring + jf * kGuSlot;
          tc::mbar_expect_tx(bar, kGuSlot);
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {  // (zeros past the last block)
            tc::tma_load_2d(dst + 2 * h * kBox16, mg, bar, (kb + h) * kF8Block, row);
            tc::tma_load_2d(dst + (2 * h + 1) * kBox16, mu, bar, (kb + h) * kF8Block, row);
          }
        }
        __syncwarp();
        if (lane < 4) copy4(&S.scale[warp][jf][lane], ps + min(kb + (lane & 1), KB - 1), bar);
        kb += 2 * nsplit;
        if (--todo == 0) advance(ahead);
        if (++jf == kGuAhead) jf = 0;
        if (++filled < kGuAhead) continue;
      }
      if (!codes) {
        codes = true;
        __syncthreads();  // the tokens' codes are there
      }
      if (now.i >= items) break;
      if (left == 0) {  // the chunk's tokens: this lane's column, and its two sums' columns
        const int start = L.start[now.c], last = L.count[now.c] - 1;
        const bool sh = now.c >= L.n_routed;
        auto token = [&](int q) {
          const int p = start + min(q, last);
          return sh ? p : (int)L.token[p];
        };
        xr = xq32 + token(g) * xstride;
        x0 = xs32 + token(2 * t) * KB * 4;
        x1 = xs32 + token(2 * t + 1) * KB * 4;
        left = steps;
        kx = 2 * w;
      }
      if (steps) {
        if (!f8_warp_wait(&S.landed[warp][j], ph, a.wait_ns, a.ctrl, kSiteFewFp8)) break;
        const uint32_t slot = ring32 + j * kGuSlot;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (kx + h >= KB) break;  // the last pair's second block may not exist
          const uint4 b0 = lds16<0>(xr + h * kF8Block), b1 = lds16<64>(xr + h * kF8Block);
          const float sg = lds4<0>(sc32 + 16 * j + 4 * h), su = lds4<8>(sc32 + 16 * j + 4 * h);
          const float s0 = lds4<0>(x0 + 4 * h), s1 = lds4<0>(x1 + 4 * h);
          const float c0 = sg * s0, c1 = sg * s1, c2 = su * s0, c3 = su * s1;
          BlockSum d[2];
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const uint32_t box = slot + 2 * h * kBox16 + m * kBox8;
            d[m].mma(weights_of(box, box + kBox16, get), b0, b1);
          }
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            acc[m][0] = fmaf(d[m].of(0), c0, acc[m][0]);
            acc[m][1] = fmaf(d[m].of(1), c1, acc[m][1]);
            acc[m][2] = fmaf(d[m].of(2), c2, acc[m][2]);
            acc[m][3] = fmaf(d[m].of(3), c3, acc[m][3]);
          }
        }
        xr += 2 * nsplit * kF8Block;
        x0 += 8 * nsplit;
        x1 += 8 * nsplit;
        kx += 2 * nsplit;
        reads_before_refill();
        __syncwarp();
        --filled;
        if (++j == kGuAhead) {
          j = 0;
          ph ^= 1u;
        }
        if (--left) continue;
      }
      // the item's partial sums go to a finisher
      const int at = r % SLOTS;
      if (!f8_warp_wait(&S.empty[at][group], (r / SLOTS & 1) ^ 1, a.wait_ns, a.ctrl, kSiteFewFp8)) break;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        S.part[at][warp][m][lane] = make_float4(acc[m][0], acc[m][1], acc[m][2], acc[m][3]);
        acc[m][0] = acc[m][1] = acc[m][2] = acc[m][3] = 0.f;
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&S.full[at][group]);
      advance(now);
      ++r;
    }
  } else {
    // While the others group the pairs and wait for their first weights, this
    // warpgroup quantises the tokens: sixteen lanes per block of 128, several
    // blocks in flight. (The streaming warps' own loads of x came back behind
    // their loads of cold weights: 20,000 cycles before the first product at 8
    // tokens.)
    const int blocks = a.T * KB;
    constexpr int kHalves = 8, kFlight = 4;
    for (int b0 = (tid >> 4) & (kHalves - 1); b0 - ((tid >> 4) & 1) < blocks; b0 += kHalves * kFlight) {
      uint4 raw[kFlight];
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const int b = b0 + u * kHalves, tok = b / KB, c = (b - tok * KB) * kF8Block + (lane & 15) * 8;
        raw[u] = b < blocks && c < a.d
                     ? *reinterpret_cast<const uint4*>(a.x + (size_t)tok * a.d + c) : zero4();
      }
#pragma unroll
      for (int u = 0; u < kFlight; ++u) {
        const int b = b0 + u * kHalves, tok = b / KB, c = (b - tok * KB) * kF8Block + (lane & 15) * 8;
        float v[8];
        Chunk<__nv_bfloat16>::unpack(raw[u], v);
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, f8_mag(v[j]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const uint32_t sb = f8_scale_bits(m);
        const float inv = f8_inverse(sb);
        if (b < blocks) {
          *reinterpret_cast<uint2*>(xq + tok * xstride + c) =
              make_uint2(f8_pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                         f8_pack4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
          if ((lane & 15) == 0) xs[b] = __uint_as_float(sb);
        }
      }
    }
    __syncthreads();
    const int items = item_count();
    // a finisher has a slot of its group to itself: no more take turns than
    // there are slots
    const int group = (warp - kGuWarps) % groups, turns = min(kGuFinish / groups, SLOTS);
    int r = 0;
    Walk now{group * (int)gridDim.x + (int)blockIdx.x, 0, 0};
    for (settle(now); now.i < items; advance(now), ++r) {
      if (r % turns != (warp - kGuWarps) / groups) continue;
      const int c = now.c, rb = now.rb, start = L.start[c], cnt = L.count[c];
      const bool sh = L.expert[c] == a.E;
      const int slot = r % SLOTS;
      if (!f8_warp_wait(&S.full[slot][group], r / SLOTS & 1, a.wait_ns, a.ctrl, kSiteFewFp8)) break;
      const float4(*part)[2][32] = S.part[slot] + group * nsplit;
      float4 v[2];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        v[m] = part[0][m][lane];
        for (int q = 1; q < nsplit; ++q) {
          const float4 o = part[q][m][lane];
          v[m].x += o.x;
          v[m].y += o.y;
          v[m].z += o.z;
          v[m].w += o.w;
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&S.empty[slot][group]);
      const int row0 = (sh ? a.T * a.k : 0) + start;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        float* h = a.Hf + (size_t)(row0 + 2 * t) * a.ldh + rb * kGuRows + 8 * m + g;
        if (2 * t < cnt) h[0] = siluf_(v[m].x) * v[m].z;
        if (2 * t + 1 < cnt) h[a.ldh] = siluf_(v[m].y) * v[m].w;
      }
      // the last of a block's items quantises its 128 columns
      const int width = sh ? a.Is : a.I, blk = rb * kGuRows / kF8Block;
      const int need = min(kF8Block / kGuRows, width / kGuRows - blk * (kF8Block / kGuRows));
      __threadfence();
      __syncwarp();
      unsigned prev = 0;
      unsigned* ctr = a.counters + (size_t)c * a.hblocks + blk;
      if (lane == 0) prev = atomicAdd(ctr, 1u);
      prev = __shfl_sync(0xffffffffu, prev, 0);
      if ((int)prev != need - 1) continue;
      if (lane == 0) *ctr = 0u;
      __threadfence();
      const int hc = blk * kF8Block + lane * 4;
#pragma unroll 4
      for (int q = 0; q < cnt; ++q) {
        const size_t at = (size_t)(row0 + q) * a.ldh + hc;
        float4 h = make_float4(0.f, 0.f, 0.f, 0.f);
        if (hc < width) h = __ldcg(reinterpret_cast<const float4*>(a.Hf + at));
        const uint32_t m = __reduce_max_sync(
            0xffffffffu, max(max(f8_mag(h.x), f8_mag(h.y)), max(f8_mag(h.z), f8_mag(h.w))));
        const uint32_t sb = f8_scale_bits(m);
        const float inv = f8_inverse(sb);
        *reinterpret_cast<uint32_t*>(a.Hq + at) = f8_pack4(h.x * inv, h.y * inv, h.z * inv, h.w * inv);
        if (lane == 0) a.Hs[(size_t)(row0 + q) * a.hblocks + blk] = __uint_as_float(sb);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// 2. down + combine
// ---------------------------------------------------------------------------
constexpr int kDnCols = 16;
constexpr int kDnPitch = kDnCols + 1;

constexpr int kDnSlot = 2 * (kBox16 + kBox8);  // weights and activations of two blocks
constexpr int kDnArrivals = 20;  // weights, activations, 18 scales

// WARPS warps with AHEAD slots in flight each. Sixteen warps where every CTA
// has an SM of its own (128 KB of weights in flight), six where there are more
// CTAs than SMs, so that two fit, and where the sums of many slots (more than 356
// pairs and shared tokens) leave no room for sixteen warps' slots. A warp's walk through a slot is a chain of
// latencies, so that warps count more than slots: eight warps of three slots
// took 53.8 us where sixteen of two take 48.4 (8 tokens, 256-expert shape,
// both kernels), four of three 198 where six of two take 182 (4 tokens, 8
// wide experts).
template <int WARPS, int AHEAD>
struct DnShared {
  uint8_t ring[WARPS][AHEAD][kDnSlot];
  uint64_t landed[WARPS][AHEAD];
  float scale[WARPS][AHEAD][20];  // of eight activation rows, two blocks; [16], [17]: weights
  FewLists lists;
  float ysum[1];  // [split][P + T][kDnPitch]
};

template <int WARPS, int AHEAD>
__global__ void __launch_bounds__(WARPS * 32, WARPS <= 8 ? 2 : 1)
    f8_few_down_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmSW,
                       const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmSX,
                       const F8ExpertsArgs a) {
  extern __shared__ uint8_t smem_raw[];
  DnShared<WARPS, AHEAD>& S = *reinterpret_cast<DnShared<WARPS, AHEAD>*>(align1024(smem_raw));
  FewLists& L = S.lists;
  float* ysum = S.ysum;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  if (tid == 0) {
    for (int i = 0; i < WARPS * AHEAD; ++i)
      tc::mbar_init(&S.landed[0][0] + i, few_arrivals(kDnArrivals, i, a.stall));
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  const int P = a.T * a.k, rows_all = P + (a.Is > 0 ? a.T : 0);
  const int col0 = blockIdx.x * kDnCols;
  const int KBr = f8_blocks(a.I), KBs = f8_blocks(a.Is), NB = f8_blocks(a.d);
  const int PRr = (KBr + 1) / 2, PRs = (KBs + 1) / 2;  // pairs of blocks
  // The ids and the weights, read before pdl_wait, are older than the gate/up
  // kernel, which has itself waited for its predecessor before letting this one
  // start (f8_few_gateup triggers after its wait; nothing may be launched between
  // the two).
  build_lists<WARPS * 32>(a, L);
  // k split of a chunk: the one that leaves the busiest warp the fewest pairs
  const int PR = PRr > PRs ? PRr : PRs, room = max(rows_all, 16 * WARPS);
  int lsplit = 0, least = 0x7FFFFFFF;
  for (int l = 0; (1 << l) <= min(PR, WARPS) && (rows_all << l) <= room; ++l) {
    const int n = ((L.n_chunks << l) + WARPS - 1) / WARPS * ((PR + (1 << l) - 1) >> l);
    if (n < least) {
      least = n;
      lsplit = l;
    }
  }
  const int split = 1 << lsplit;
  const int walks = L.n_chunks * split;
  // A warp's walk over (chunk, k split) and the pairs of blocks of each.
  struct Walk {
    int idx, c, left, kb;  // chunk c, pairs of it left for this warp, the first block of the next
  };
  auto settle = [&](Walk& k) {  // to the next part that has a pair, if any
    for (; k.idx < walks; k.idx += WARPS) {
      k.c = k.idx >> lsplit;
      const int n = k.c >= L.n_routed ? PRs : PRr, s = k.idx & (split - 1);
      k.left = (n - s + split - 1) >> lsplit;
      k.kb = 2 * s;
      if (k.left > 0) return;
    }
    k.left = 0;
  };
  auto step = [&](Walk& k) {  // one pair on; true if the chunk's part ends
    k.kb += 2 * split;
    if (--k.left) return false;
    k.idx += WARPS;
    return true;
  };
  Walk now{warp, 0, 0, 0};
  settle(now);
  // The loads' walks, ahead of the arithmetic's: weights from the start, the
  // activations once the gate/up kernel has ended. One loop fills slots and
  // works them off, every piece of its code once.
  Walk aw = now, ax = now;
  uint8_t* ring = S.ring[warp][0];
  const uint32_t ring32 = tc::smem_u32(ring), sc32 = tc::smem_u32(S.scale[warp]);
  const uint32_t get = get_at(g, t);
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  uint32_t ph = 0;
  int j = 0, jw = 0, jx = 0, filled_w = 0, filled_x = 0;
  bool waited = false, new_w = true, new_x = true, shared_w = false, shared_x = false;
  const CUtensorMap *mw = &tmW, *mx = &tmX;
  const float *psw = a.Sd, *psx = a.Hs;  // lanes 16, 17: the weights'; lanes 0-15: the rows'
  int row_w = 0, row_x = 0;
  while (true) {
    if (filled_w < AHEAD && aw.left) {
      if (new_w) {
        const int e = L.expert[aw.c];
        shared_w = e == a.E;
        mw = shared_w ? &tmSW : &tmW;
        row_w = (shared_w ? 0 : e * a.d) + col0;
        psw = (shared_w ? a.Ssd : a.Sd) +
              ((shared_w ? 0 : (size_t)e * NB) + col0 / kF8Block) * (shared_w ? KBs : KBr);
      }
      uint64_t* bar = &S.landed[warp][jw];
      if (lane == 0) {
        uint8_t* dst = ring + jw * kDnSlot;
        tc::mbar_expect_tx(bar, 2 * kBox16);
        tc::tma_load_2d(dst, mw, bar, aw.kb * kF8Block, row_w);
        tc::tma_load_2d(dst + kBox16, mw, bar, (aw.kb + 1) * kF8Block, row_w);  // (zeros past the last)
      }
      __syncwarp();
      if (lane >= 16 && lane < 18)
        copy4(&S.scale[warp][jw][lane], psw + min(aw.kb + (lane & 1), (shared_w ? KBs : KBr) - 1), bar);
      new_w = step(aw);
      if (new_w) settle(aw);
      if (++jw == AHEAD) jw = 0;
      if (++filled_w < AHEAD && !waited) continue;
    }
    if (!waited) {
      waited = true;
      pdl_wait();
      pdl_trigger();
    }
    if (filled_x < AHEAD && ax.left) {
      if (new_x) {
        shared_x = ax.c >= L.n_routed;
        mx = shared_x ? &tmSX : &tmX;
        row_x = (shared_x ? P : 0) + L.start[ax.c];
        psx = a.Hs + (size_t)(row_x + min(lane & 7, L.count[ax.c] - 1)) * a.hblocks;
      }
      uint64_t* bar = &S.landed[warp][jx];
      if (lane == 0) {
        uint8_t* dst = ring + jx * kDnSlot + 2 * kBox16;
        tc::mbar_expect_tx(bar, 2 * kBox8);
        tc::tma_load_2d(dst, mx, bar, ax.kb * kF8Block, row_x);
        tc::tma_load_2d(dst + kBox8, mx, bar, (ax.kb + 1) * kF8Block, row_x);
      }
      __syncwarp();
      if (lane < 16)
        copy4(&S.scale[warp][jx][lane], psx + min(ax.kb + (lane >> 3), (shared_x ? KBs : KBr) - 1), bar);
      new_x = step(ax);
      if (new_x) settle(ax);
      if (++jx == AHEAD) jx = 0;
      if (++filled_x < filled_w) continue;
    }
    if (now.left == 0) break;
    if (!f8_warp_wait(&S.landed[warp][j], ph, a.wait_ns, a.ctrl, kSiteFewFp8)) break;
    const uint32_t slot = ring32 + j * kDnSlot, sc = sc32 + 80 * j;
    // the last pair's second block may not exist; the activations' rows may be
    // longer, and what lies there is nobody's
    const bool second = now.kb + 1 < (now.c >= L.n_routed ? KBs : KBr);
    BlockSum d[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t w = slot + h * kBox16, x = slot + 2 * kBox16 + h * kBox8;
      if (h == 0 || second)
        d[h].mma(weights_of(w, w + kBox8, get), lds16<0>(x + get), lds16<0>(x + (get ^ 64u)));
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == 0 || second) {
        const float sw = lds4<64>(sc + 4 * h);
        const float s0 = sw * lds4<0>(sc + 32 * h + 8 * t), s1 = sw * lds4<4>(sc + 32 * h + 8 * t);
        acc[0] = fmaf(d[h].of(0), s0, acc[0]);
        acc[1] = fmaf(d[h].of(1), s1, acc[1]);
        acc[2] = fmaf(d[h].of(2), s0, acc[2]);
        acc[3] = fmaf(d[h].of(3), s1, acc[3]);
      }
    }
    reads_before_refill();
    __syncwarp();
    --filled_w;
    --filled_x;
    if (++j == AHEAD) {
      j = 0;
      ph ^= 1u;
    }
    const int c = now.c, s = now.idx & (split - 1);
    if (!step(now)) continue;
    // the part's sums; their weights are applied when the slots are added
    const int cnt = L.count[c], row0 = (c >= L.n_routed ? P : 0) + L.start[c];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (2 * t + q < cnt) {
        float* y = ysum + ((size_t)s * rows_all + row0 + 2 * t + q) * kDnPitch;
        y[g] = acc[q];
        y[g + 8] = acc[2 + q];
      }
    }
    acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
    settle(now);
  }
  __syncthreads();
  const int parts_r = min(split, PRr), parts_s = min(split, PRs);
  for (int i = tid; i < a.T * kDnCols; i += WARPS * 32) {
    const int tok = i / kDnCols, c = i - tok * kDnCols;
    const size_t o = (size_t)tok * a.d + col0 + c;
    const float res = a.r_attn ? a.r_attn[o] : 0.f;
    const int plane = rows_all * kDnPitch;
    float y = 0.f;
#pragma unroll 4
    for (int sl = 0; sl < a.k; ++sl) {
      const float* p = ysum + L.pos[tok * a.k + sl] * kDnPitch + c;
      float v = p[0];
      for (int s = 1; s < parts_r; ++s) v += p[s * plane];
      y = fmaf(a.alpha[tok * a.k + sl], v, y);
    }
    if (parts_s) {
      const float* p = ysum + (P + tok) * kDnPitch + c;
      float v = p[0];
      for (int s = 1; s < parts_s; ++s) v += p[s * plane];
      y = fmaf(a.s_shared[tok], v, y);
    }
    y += res;
    if (a.out_bf16)
      static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(y);
    else
      static_cast<float*>(a.out)[o] = y;
  }
}

// ---------------------------------------------------------------------------
// product for a few rows
// ---------------------------------------------------------------------------
constexpr int kMmWarps = 8;

// out[m][n] for M <= 8 NT rows: items of 16 output columns, k split over the
// `wpi` warps of an item, two blocks each, whose sums are added in warp order.
template <int NT>
constexpr int mm_slot() { return 2 * (kBox16 + NT * kBox8); }
template <int NT, int AHEAD>
struct MmShared {
  uint8_t ring[kMmWarps][AHEAD][mm_slot<NT>()];
  float4 part[2][NT][kMmWarps][32];
  uint64_t landed[kMmWarps][AHEAD];
  float scale[kMmWarps][AHEAD][36];  // of the activation rows, two blocks; [32], [33]: weights
};
template <int NT, int AHEAD>
__global__ void __launch_bounds__(kMmWarps * 32, 1)
    f8_few_matmul_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                         const F8MatmulArgs a) {
  extern __shared__ uint8_t smem_raw[];
  MmShared<NT, AHEAD>& S = *reinterpret_cast<MmShared<NT, AHEAD>*>(align1024(smem_raw));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  // arrivals: the boxes' bytes, 16 NT scales of the rows, two of the weights
  if (tid == 0) {
    for (int i = 0; i < kMmWarps * AHEAD; ++i)
      tc::mbar_init(&S.landed[0][0] + i, few_arrivals(3 + 16 * NT, i, a.stall));
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  const int KB = f8_blocks(a.K), pairs = (KB + 1) / 2;
  pdl_wait();
  pdl_trigger();
  int wpi = 1;
  while (wpi * 2 <= pairs && wpi < kMmWarps) wpi *= 2;
  const int teams = kMmWarps / wpi, team = warp / wpi, w = warp % wpi;
  const int items = (a.N + 15) / 16;
  const int stride = (int)gridDim.x * teams, rounds = (items + stride - 1) / stride;
  const int first = team * (int)gridDim.x + (int)blockIdx.x;
  const uint32_t get = get_at(g, t);
  // the lane's scale: row lane % (8 NT), block lane / (8 NT) of the two
  const float* xsc = a.a_scale + (size_t)min(lane & (8 * NT - 1), a.M - 1) * KB;
  uint8_t* ring = S.ring[warp][0];
  int li = first, lp = w;  // the loads' item and pair of blocks
  auto load = [&](int j) {
    if (li >= items) return;
    uint64_t* bar = &S.landed[warp][j];
    uint8_t* dst = ring + j * mm_slot<NT>();
    const int kb = 2 * lp;
    if (lane == 0) {
      // rows and columns past the ends, a second block among them, come as zeros,
      // and so do that block's scales (zero codes with infinite ones were NaN)
      tc::mbar_expect_tx(bar, mm_slot<NT>());
      tc::tma_load_2d(dst, &tmB, bar, kb * kF8Block, li * 16);
      tc::tma_load_2d(dst + kBox16, &tmB, bar, (kb + 1) * kF8Block, li * 16);
      tc::tma_load_2d(dst + 2 * kBox16, &tmA, bar, kb * kF8Block, 0);
      tc::tma_load_2d(dst + 2 * kBox16 + NT * kBox8, &tmA, bar, (kb + 1) * kF8Block, 0);
    }
    const int kx = kb + lane / (8 * NT);
    if (lane < 16 * NT) copy4(&S.scale[warp][j][lane], xsc + min(kx, KB - 1), bar, kx < KB);
    if (lane < 2)
      copy4(&S.scale[warp][j][32 + lane],
            a.b_scale + (size_t)(li * 16 / kF8Block) * KB + min(kb + lane, KB - 1), bar, kb + lane < KB);
    lp += wpi;
    if (lp >= pairs) {
      lp = w;
      li += stride;
    }
  };
  for (int j = 0; j < AHEAD; ++j) load(j);
  float acc[NT][4] = {};
  const uint32_t ring32 = tc::smem_u32(ring), sc32 = tc::smem_u32(S.scale[warp]);
  uint32_t ph = 0;
  int r = 0, pr = w, j = 0;
  bool alive = true;
  while (r < rounds) {
    const int i = first + r * stride;
    if (alive && i < items && pr < pairs)
      alive = f8_warp_wait(&S.landed[warp][j], ph, a.wait_ns, a.ctrl, kSiteFewFp8);
    // (a warp whose wait gave up loads nothing more and goes along to the barriers)
    if (alive && i < items && pr < pairs) {
      const uint32_t slot = ring32 + j * mm_slot<NT>(), sc = sc32 + 144 * j;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t wb = slot + h * kBox16;
        const WeightBlock wgt = weights_of(wb, wb + kBox8, get);
        const float sw = lds4<128>(sc + 4 * h);
#pragma unroll
        for (int q = 0; q < NT; ++q) {
          const uint32_t x = slot + 2 * kBox16 + (h * NT + q) * kBox8;
          const uint32_t sx = sc + 4 * (8 * NT * h + 8 * q + 2 * t);
          BlockSum d;
          d.mma(wgt, lds16<0>(x + get), lds16<0>(x + (get ^ 64u)));
          const float c0 = sw * lds4<0>(sx), c1 = sw * lds4<4>(sx);
          acc[q][0] = fmaf(d.of(0), c0, acc[q][0]);
          acc[q][1] = fmaf(d.of(1), c1, acc[q][1]);
          acc[q][2] = fmaf(d.of(2), c0, acc[q][2]);
          acc[q][3] = fmaf(d.of(3), c1, acc[q][3]);
        }
      }
      reads_before_refill();
      __syncwarp();
      load(j);
      if (++j == AHEAD) {
        j = 0;
        ph ^= 1u;
      }
    }
    pr += wpi;
    if (pr - w < pairs) continue;
    pr = w;
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      S.part[r & 1][q][warp][lane] = make_float4(acc[q][0], acc[q][1], acc[q][2], acc[q][3]);
      acc[q][0] = acc[q][1] = acc[q][2] = acc[q][3] = 0.f;
    }
    __syncthreads();
    const int round = r++;
    if (i >= items || w != round % wpi) continue;
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      float4 v = S.part[round & 1][q][team * wpi][lane];
      for (int p = 1; p < wpi; ++p) {
        const float4 o = S.part[round & 1][q][team * wpi + p][lane];
        v.x += o.x;
        v.y += o.y;
        v.z += o.z;
        v.w += o.w;
      }
      const float y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const int m = 8 * q + 2 * t + (z & 1), col = i * 16 + g + 8 * (z >> 1);
        if (m < a.M && col < a.N) {
          if (a.out_bf16)
            static_cast<__nv_bfloat16*>(a.out)[(size_t)m * a.ldo + col] = __float2bfloat16_rn(y[z]);
          else
            static_cast<float*>(a.out)[(size_t)m * a.ldo + col] = y[z];
        }
      }
    }
  }
}

template <int SLOTS>
size_t gateup_smem(int T, int d) {
  const int KB = f8_blocks(d);
  return 1024 + sizeof(GuShared<SLOTS>) + (((size_t)T * KB * 4 + 15) & ~15) +
         (size_t)T * (KB * kF8Block + 64);
}
constexpr size_t kSmemLimit = 227 * 1024;

template <int SLOTS>
cudaError_t launch_gateup(const F8FewMaps& m, const F8ExpertsArgs& a, cudaStream_t st) {
  static int attr[64] = {};
  const size_t smem = gateup_smem<SLOTS>(a.T, a.d);
  cudaError_t e = ensure_smem_limit(f8_few_gateup_kernel<SLOTS>, (int)smem, attr);
  if (e != cudaSuccess) return e;
  return launch_pdl(f8_few_gateup_kernel<SLOTS>, dim3(tc_sm_count()), kGuThreads, smem, st, m.g, m.u, m.sg,
                    m.su, a);
}

// Rows of partial sums: all pairs and shared tokens once, or as many splits of
// them as 16 WARPS rows hold.
template <int WARPS, int AHEAD>
constexpr size_t down_smem(int T, int k) {
  const int rows = T * k + T;
  return 1024 + sizeof(DnShared<WARPS, AHEAD>) +
         (size_t)(rows > 16 * WARPS ? rows : 16 * WARPS) * kDnPitch * 4;
}
// six warps take whatever f8_few_ok lets through
static_assert(down_smem<6, 2>(kF8FewTokens, kFewMaxPairs / kF8FewTokens) <= kSmemLimit, "down's plan exceeds 227 KB");

template <int WARPS, int AHEAD>
cudaError_t launch_down(const F8FewMaps& m, const F8ExpertsArgs& a, cudaStream_t st) {
  static int attr[64] = {};
  const size_t smem = down_smem<WARPS, AHEAD>(a.T, a.k);
  cudaError_t e = ensure_smem_limit(f8_few_down_kernel<WARPS, AHEAD>, (int)smem, attr);
  if (e != cudaSuccess) return e;
  return launch_pdl(f8_few_down_kernel<WARPS, AHEAD>, dim3(a.d / kDnCols), WARPS * 32, smem, st, m.w, m.sw,
                    m.x, m.sx, a);
}

template <int NT, int AHEAD>
cudaError_t launch_matmul(const F8MatmulArgs& a, cudaStream_t st) {
  static int attr[64] = {};
  const size_t smem = 1024 + sizeof(MmShared<NT, AHEAD>);
  cudaError_t e = ensure_smem_limit(f8_few_matmul_kernel<NT, AHEAD>, (int)smem, attr);
  if (e != cudaSuccess) return e;
  CUtensorMap A, B;
  if (!f8_make_map(&A, a.a, a.M, a.K, a.lda, 8 * NT) || !f8_make_map(&B, a.b, a.N, a.K, a.ldb, 16))
    return cudaErrorInvalidValue;
  const int items = (a.N + 15) / 16;
  const int grid = items < tc_sm_count() ? items : tc_sm_count();
  return launch_pdl(f8_few_matmul_kernel<NT, AHEAD>, dim3(grid), kMmWarps * 32, smem, st, A, B, a);
}

}  // namespace

bool f8_few_ok(int T, int d, int k) {
  return T <= kF8FewTokens && T * k <= kFewMaxPairs && gateup_smem<2>(T, d) <= kSmemLimit;
}

cudaError_t launch_f8_few_gateup(const F8FewMaps& m, const F8ExpertsArgs& a, cudaStream_t st) {
  return gateup_smem<4>(a.T, a.d) <= kSmemLimit ? launch_gateup<4>(m, a, st) : launch_gateup<2>(m, a, st);
}

cudaError_t launch_f8_few_down(const F8FewMaps& m, const F8ExpertsArgs& a, cudaStream_t st) {
  const bool sixteen = a.d / kDnCols <= tc_sm_count() && down_smem<16, 2>(a.T, a.k) <= kSmemLimit;
  return sixteen ? launch_down<16, 2>(m, a, st) : launch_down<6, 2>(m, a, st);
}

cudaError_t launch_f8_few_matmul(const F8MatmulArgs& a, cudaStream_t st) {
  return a.M <= 8 ? launch_matmul<1, 3>(a, st) : launch_matmul<2, 2>(a, st);
}

}  // namespace moe
