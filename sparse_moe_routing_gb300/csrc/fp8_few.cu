// The 8-bit layer for a few tokens, and the 8-bit product for a few rows:
// weight streams on mma.sync (e4m3 x e4m3 -> fp32).
//
// A few tokens meet every weight byte once, so these kernels are bound by
// HBM and, for one token, by latency. mma.sync m16n8k32 takes 16 weight rows
// as its m side and up to 8 tokens as its n side. A contraction does not care
// in which order k is visited as long as both operands agree, so a lane's
// fragment registers are simply the 16-byte pieces that it loads from memory:
// no shared-memory staging, no conversion, no shuffles. A warp keeps
// kAhead blocks of 16 rows x 128 k in flight in registers.
//
// The products of one 128-wide block are summed by the tensor core and then
// scaled by the block's two scales into fp32 sums held in registers.
//
// The layer takes two kernels:
//  1. f8_few_gateup: every CTA groups the (token, slot) pairs by expert into
//     chunks of at most 8 (ranking by counting), quantises the tokens into
//     shared memory, then takes items of 8 gate and 8 up rows of a chunk's
//     expert (one m16 tile, so a lane holds a row's gate and up sums). The
//     warps split k; their sums meet in shared memory and are added in warp
//     order. h needs one scale per 128 columns, which 16 items share: the item
//     that finishes a block last (a counter that it also resets) quantises it.
//  2. f8_few_down: a CTA owns 16 output columns of every chunk and adds the
//     slots, the shared expert and the residual in a fixed order.
#include "fp8_common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kFewMaxPairs = 512;  // 16 tokens of at most 32 slots

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One block of 128 k: rows g and g + 8 of the m16 tile, two 16-byte pieces
// each (k 16 t.. and k 64 + 16 t.. for t = lane % 4).
struct WeightBlock {
  uint4 lo[2], hi[2];
};
struct ActBlock {
  uint4 v[2];
};

__device__ __forceinline__ void block_mma(float (&d)[4], const WeightBlock& w, const uint4& b0,
                                          const uint4& b1) {
  d[0] = d[1] = d[2] = d[3] = 0.f;
  mma_e4m3(d, w.lo[0].x, w.hi[0].x, w.lo[0].y, w.hi[0].y, b0.x, b0.y);
  mma_e4m3(d, w.lo[0].z, w.hi[0].z, w.lo[0].w, w.hi[0].w, b0.z, b0.w);
  mma_e4m3(d, w.lo[1].x, w.hi[1].x, w.lo[1].y, w.hi[1].y, b1.x, b1.y);
  mma_e4m3(d, w.lo[1].z, w.hi[1].z, w.lo[1].w, w.hi[1].w, b1.z, b1.w);
}

__device__ __forceinline__ uint4 zero4() { return make_uint4(0u, 0u, 0u, 0u); }

// Bytes of a 16-byte piece past the first n zeroed (n <= 0: all of them). A
// code past the end of a row may be NaN, and NaN times zero is NaN, so both
// operands are cut.
__device__ __forceinline__ uint4 keep_bytes(uint4 v, int n) {
  if (n >= 16) return v;
  auto cut = [](uint32_t w, int m) { return m >= 4 ? w : (m <= 0 ? 0u : w & ((1u << (8 * m)) - 1u)); };
  return make_uint4(cut(v.x, n), cut(v.y, n - 4), cut(v.z, n - 8), cut(v.w, n - 12));
}

// ---------------------------------------------------------------------------
// chunks of at most 8 pairs of one expert, then of 8 tokens for the shared one
// ---------------------------------------------------------------------------
struct FewLists {
  alignas(16) int ids[kFewMaxPairs + 4];
  int n_routed, n_chunks;
  int sorted[kFewMaxPairs];          // position -> pair
  int pos[kFewMaxPairs];             // pair -> position
  int start[kFewMaxPairs + 8];       // chunk -> first position (shared: first token)
  int expert[kFewMaxPairs + 8];      // chunk -> expert (E: shared)
  int count[kFewMaxPairs + 8];       // chunk -> pairs in it
  unsigned char first[kFewMaxPairs]; // position starts a chunk
};

// Positions order the pairs by (expert, pair). All threads of the CTA call it.
__device__ __forceinline__ void build_lists(const F8ExpertsArgs& a, FewLists& L) {
  const int P = a.T * a.k, tid = threadIdx.x, lane = tid & 31;
  bool bad = false;
  for (int i = tid; i < ((P + 3) & ~3); i += blockDim.x) {
    int e = i < P ? __ldcg(a.ids + i) : 0x7FFFFFFF;
    if (i < P && (e < 0 || e >= a.E)) {
      bad = true;
      e = a.E - 1;
    }
    L.ids[i] = e;
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) report(a.ctrl, kDevBadId, kSiteFewFp8);
  __syncthreads();
  for (int i = tid; i < P; i += blockDim.x) {
    const int e = L.ids[i];
    int below = 0, same = 0;
    for (int j = 0; j < P; j += 4) {
      const int4 o = *reinterpret_cast<const int4*>(L.ids + j);
      below += (o.x < e) + (o.y < e) + (o.z < e) + (o.w < e);
      same += (o.x == e && j < i) + (o.y == e && j + 1 < i) + (o.z == e && j + 2 < i) +
              (o.w == e && j + 3 < i);
    }
    L.sorted[below + same] = i;
    L.pos[i] = below + same;
    L.first[below + same] = (same & 7) == 0;
  }
  __syncthreads();
  if (tid < 32) {
    int n = 0;
    for (int r0 = 0; r0 < P; r0 += 32) {
      const bool f = r0 + lane < P && L.first[r0 + lane];
      const unsigned m = __ballot_sync(0xffffffffu, f);
      if (f) {
        const int c = n + __popc(m & ((1u << lane) - 1u));
        L.start[c] = r0 + lane;
        L.expert[c] = L.ids[L.sorted[r0 + lane]];
      }
      n += __popc(m);
    }
    __syncwarp();
    for (int c = lane; c < n; c += 32) L.count[c] = (c + 1 < n ? L.start[c + 1] : P) - L.start[c];
    const int ns = a.Is > 0 ? (a.T + 7) / 8 : 0;
    if (lane < ns) {
      L.start[n + lane] = 8 * lane;
      L.expert[n + lane] = a.E;
      L.count[n + lane] = min(8, a.T - 8 * lane);
    }
    if (lane == 0) {
      L.n_routed = n;
      L.n_chunks = n + ns;
    }
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------
// 1. gate/up
// ---------------------------------------------------------------------------
constexpr int kGuWarps = 16;
constexpr int kGuAhead = 4;

struct GuItem {
  int chunk, rb;  // chunk and block of 8 rows
};

struct GuUnit {
  WeightBlock w;
  float sg, su;
};

__global__ void __launch_bounds__(kGuWarps * 32, 1) f8_few_gateup_kernel(F8ExpertsArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  FewLists& L = *reinterpret_cast<FewLists*>(smem);
  float4* part = reinterpret_cast<float4*>(smem + few_lists_bytes());  // [2][kGuWarps][32]
  const int KB = f8_blocks(a.d);
  float* xs = reinterpret_cast<float*>(part + 2 * kGuWarps * 32);     // [T][KB]
  const int xstride = KB * kF8Block + 64;  // rows 64 B apart modulo the banks' 128 B
  uint8_t* xq = reinterpret_cast<uint8_t*>(xs) + ((a.T * KB * 4 + 15) & ~15);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  pdl_wait();
  pdl_trigger();
  build_lists(a, L);

  // wpi warps share an item along k, the others take other items
  int wpi = 1;
  while (wpi * 2 <= KB && wpi < kGuWarps) wpi *= 2;
  const int slots = kGuWarps / wpi, slot = warp / wpi, w = warp % wpi;
  const int RB = a.I / 8, RBs = a.Is / 8;
  const int routed_items = L.n_routed * RB;
  const int items = routed_items + (L.n_chunks - L.n_routed) * RBs;
  const int stride = (int)gridDim.x * slots;
  const int rounds = (items + stride - 1) / stride;
  const int steps = (KB + wpi - 1) / wpi;  // blocks of an item per warp
  const int units = rounds * steps;
  auto item_at = [&](int i) {
    GuItem it;
    if (i < routed_items) {
      it.chunk = i / RB;
      it.rb = i - it.chunk * RB;
    } else {
      const int j = i - routed_items;
      it.chunk = L.n_routed + j / RBs;
      it.rb = j - (j / RBs) * RBs;
    }
    return it;
  };
  const int first = slot * (int)gridDim.x + (int)blockIdx.x;
  auto load = [&](GuUnit& u, int n) {
    const int r = n / steps, kb = (n - r * steps) * wpi + w;
    const int i = first + r * stride;
    u.w.lo[0] = u.w.lo[1] = u.w.hi[0] = u.w.hi[1] = zero4();
    u.sg = u.su = 0.f;
    if (n >= units || i >= items || kb >= KB) return;
    const GuItem it = item_at(i);
    const int e = L.expert[it.chunk];
    const bool sh = e == a.E;
    const int rows = sh ? a.Is : a.I;
    const size_t row = (sh ? 0 : (size_t)e * rows) + (size_t)it.rb * 8 + g;
    const int k0 = kb * kF8Block + 16 * t;
    const uint8_t* pg = (sh ? a.Wsg : a.Wg) + row * a.d + k0;
    const uint8_t* pu = (sh ? a.Wsu : a.Wu) + row * a.d + k0;
    if (k0 < a.d) {  // d is a multiple of 16
      u.w.lo[0] = ldg_stream(pg);
      u.w.hi[0] = ldg_stream(pu);
    }
    if (k0 + 64 < a.d) {
      u.w.lo[1] = ldg_stream(pg + 64);
      u.w.hi[1] = ldg_stream(pu + 64);
    }
    const size_t si = ((sh ? 0 : (size_t)e * f8_blocks(rows)) + it.rb / 16) * KB + kb;
    u.sg = __ldg((sh ? a.Ssg : a.Sg) + si);
    u.su = __ldg((sh ? a.Ssu : a.Su) + si);
  };
  GuUnit ring[kGuAhead];
#pragma unroll
  for (int j = 0; j < kGuAhead; ++j) load(ring[j], j);

  // the tokens' codes, sixteen lanes per block of 128
  for (int b = tid >> 4; b - ((tid >> 4) & 1) < a.T * KB; b += kGuWarps * 2) {
    const int tok = b / KB, kb = b - tok * KB, c = kb * kF8Block + (lane & 15) * 8;
    float v[8];
    uint4 raw = zero4();
    if (b < a.T * KB && c < a.d)
      raw = *reinterpret_cast<const uint4*>(a.x + (size_t)tok * a.d + c);
    Chunk<__nv_bfloat16>::unpack(raw, v);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, f8_mag(v[j]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const uint32_t sb = f8_scale_bits(m);
    const float inv = f8_inverse(sb);
    if (b < a.T * KB) {
      *reinterpret_cast<uint2*>(xq + (size_t)tok * xstride + c) =
          make_uint2(f8_pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                     f8_pack4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
      if ((lane & 15) == 0) xs[b] = __uint_as_float(sb);
    }
  }
  __syncthreads();

  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int n0 = 0; n0 < units; n0 += kGuAhead) {
#pragma unroll
    for (int j = 0; j < kGuAhead; ++j) {
      const int n = n0 + j;
      if (n >= units) break;
      const int r = n / steps, st = n - r * steps, kb = st * wpi + w;
      const int i = first + r * stride;
      const bool live = i < items;
      const GuItem it = live ? item_at(i) : GuItem{0, 0};
      const int start = L.start[it.chunk], cnt = L.count[it.chunk];
      const bool sh = L.expert[it.chunk] == a.E;
      if (live && kb < KB) {
        auto token = [&](int s) {
          const int p = start + min(s, cnt - 1);
          return sh ? p : L.sorted[p] / a.k;
        };
        const uint8_t* xr = xq + (size_t)token(g) * xstride + kb * kF8Block + 16 * t;
        float d[4];
        block_mma(d, ring[j].w, *reinterpret_cast<const uint4*>(xr),
                  *reinterpret_cast<const uint4*>(xr + 64));
        const float s0 = xs[token(2 * t) * KB + kb], s1 = xs[token(2 * t + 1) * KB + kb];
        acc[0] = fmaf(d[0], ring[j].sg * s0, acc[0]);
        acc[1] = fmaf(d[1], ring[j].sg * s1, acc[1]);
        acc[2] = fmaf(d[2], ring[j].su * s0, acc[2]);
        acc[3] = fmaf(d[3], ring[j].su * s1, acc[3]);
      }
      load(ring[j], n + kGuAhead);
      if (st != steps - 1) continue;
      // the item's sums: all warps write, one warp of the slot adds
      float4* buf = part + (r & 1) * kGuWarps * 32;
      buf[warp * 32 + lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
      __syncthreads();
      if (!live || w != r % wpi) continue;
      float4 v = buf[slot * wpi * 32 + lane];
      for (int q = 1; q < wpi; ++q) {
        const float4 o = buf[(slot * wpi + q) * 32 + lane];
        v.x += o.x;
        v.y += o.y;
        v.z += o.z;
        v.w += o.w;
      }
      const int row0 = (sh ? a.T * a.k : 0) + start;
      const int col = it.rb * 8 + g;
      if (2 * t < cnt) a.Hf[(size_t)(row0 + 2 * t) * a.ldh + col] = siluf_(v.x) * v.z;
      if (2 * t + 1 < cnt) a.Hf[(size_t)(row0 + 2 * t + 1) * a.ldh + col] = siluf_(v.y) * v.w;
      // the last of a block's items quantises its 128 columns
      const int width = sh ? a.Is : a.I, blk = it.rb / 16;
      const int need = min(16, width / 8 - blk * 16);
      __threadfence();
      __syncwarp();
      unsigned prev = 0;
      unsigned* ctr = a.counters + (size_t)it.chunk * a.hblocks + blk;
      if (lane == 0) prev = atomicAdd(ctr, 1u);
      prev = __shfl_sync(0xffffffffu, prev, 0);
      if ((int)prev != need - 1) continue;
      if (lane == 0) *ctr = 0u;
      __threadfence();
      const int c = blk * kF8Block + lane * 4;
#pragma unroll 1
      for (int s = 0; s < cnt; ++s) {
        const size_t at = (size_t)(row0 + s) * a.ldh + c;
        float4 h = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c < width) h = __ldcg(reinterpret_cast<const float4*>(a.Hf + at));
        const uint32_t m = __reduce_max_sync(
            0xffffffffu, max(max(f8_mag(h.x), f8_mag(h.y)), max(f8_mag(h.z), f8_mag(h.w))));
        const uint32_t sb = f8_scale_bits(m);
        const float inv = f8_inverse(sb);
        *reinterpret_cast<uint32_t*>(a.Hq + at) = f8_pack4(h.x * inv, h.y * inv, h.z * inv, h.w * inv);
        if (lane == 0) a.Hs[(size_t)(row0 + s) * a.hblocks + blk] = __uint_as_float(sb);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// 2. down + combine
// ---------------------------------------------------------------------------
constexpr int kDnWarps = 8;
constexpr int kDnAhead = 4;
constexpr int kDnCols = 16;
constexpr int kDnPitch = kDnCols + 1;

// A warp's walk over (chunk, k split) and the blocks of each.
struct DnWalk {
  int idx, kb;
};
struct DnUnit {
  WeightBlock w;
  float sw;
  ActBlock x;
  float s0, s1;
};

__global__ void __launch_bounds__(kDnWarps * 32) f8_few_down_kernel(F8ExpertsArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  FewLists& L = *reinterpret_cast<FewLists*>(smem);
  float* ysum = reinterpret_cast<float*>(smem + few_lists_bytes());  // [split][P + T][kDnPitch]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int P = a.T * a.k, rows_all = P + (a.Is > 0 ? a.T : 0);
  const int col0 = blockIdx.x * kDnCols;
  const int KBr = f8_blocks(a.I), KBs = f8_blocks(a.Is), NB = f8_blocks(a.d);
  // The ids and the weights are older than the gate/up kernel, which has
  // itself waited for its predecessor before letting this one start.
  build_lists(a, L);
  int split = 1;
  while (L.n_chunks * split < kDnWarps && split * 2 <= (KBr > KBs ? KBr : KBs)) split *= 2;
  const int walks = L.n_chunks * split;
  auto blocks_of = [&](int idx) { return L.expert[idx / split] == a.E ? KBs : KBr; };
  auto settle = [&](DnWalk& k) {  // to the next block that exists, if any
    while (k.idx < walks && k.kb >= blocks_of(k.idx)) {
      k.idx += kDnWarps;
      k.kb = k.idx % split;
    }
  };
  auto load_w = [&](DnUnit& u, const DnWalk& k) {
    u.w.lo[0] = u.w.lo[1] = u.w.hi[0] = u.w.hi[1] = zero4();
    u.sw = 0.f;
    if (k.idx >= walks) return;
    const int e = L.expert[k.idx / split];
    const bool sh = e == a.E;
    const int K = sh ? a.Is : a.I;
    const int k0 = k.kb * kF8Block + 16 * t;
    const uint8_t* p = (sh ? a.Wsd : a.Wd) + ((sh ? 0 : (size_t)e * a.d) + col0 + g) * K + k0;
    const size_t eight = (size_t)8 * K;
    if (k0 < K) {
      u.w.lo[0] = ldg_stream(p);
      u.w.hi[0] = ldg_stream(p + eight);
    }
    if (k0 + 64 < K) {
      u.w.lo[1] = ldg_stream(p + 64);
      u.w.hi[1] = ldg_stream(p + eight + 64);
    }
    u.sw = __ldg((sh ? a.Ssd : a.Sd) +
                 ((sh ? 0 : (size_t)e * NB) + col0 / kF8Block) * (sh ? KBs : KBr) + k.kb);
  };
  auto load_x = [&](DnUnit& u, const DnWalk& k) {
    u.x.v[0] = u.x.v[1] = zero4();
    u.s0 = u.s1 = 0.f;
    if (k.idx >= walks) return;
    const int c = k.idx / split;
    const int row0 = (L.expert[c] == a.E ? P : 0) + L.start[c], last = L.count[c] - 1;
    const uint8_t* p = a.Hq + (size_t)(row0 + min(g, last)) * a.ldh + k.kb * kF8Block + 16 * t;
    u.x.v[0] = __ldcg(reinterpret_cast<const uint4*>(p));
    u.x.v[1] = __ldcg(reinterpret_cast<const uint4*>(p + 64));
    u.s0 = __ldcg(a.Hs + (size_t)(row0 + min(2 * t, last)) * a.hblocks + k.kb);
    u.s1 = __ldcg(a.Hs + (size_t)(row0 + min(2 * t + 1, last)) * a.hblocks + k.kb);
  };
  DnUnit ring[kDnAhead];
  DnWalk at[kDnAhead];  // the block that each ring entry holds
  DnWalk next{warp, warp % split};
  settle(next);
#pragma unroll
  for (int j = 0; j < kDnAhead; ++j) {
    at[j] = next;
    load_w(ring[j], next);
    next.kb += split;
    settle(next);
  }
  pdl_wait();
  pdl_trigger();
#pragma unroll
  for (int j = 0; j < kDnAhead; ++j) load_x(ring[j], at[j]);

  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  bool more = at[0].idx < walks;
  while (more) {
#pragma unroll
    for (int j = 0; j < kDnAhead; ++j) {
      if (at[j].idx >= walks) {
        more = false;
        break;
      }
      float d[4];
      block_mma(d, ring[j].w, ring[j].x.v[0], ring[j].x.v[1]);
      acc[0] = fmaf(d[0], ring[j].sw * ring[j].s0, acc[0]);
      acc[1] = fmaf(d[1], ring[j].sw * ring[j].s1, acc[1]);
      acc[2] = fmaf(d[2], ring[j].sw * ring[j].s0, acc[2]);
      acc[3] = fmaf(d[3], ring[j].sw * ring[j].s1, acc[3]);
      const int idx = at[j].idx;
      if (at[j].kb + split >= blocks_of(idx)) {  // the walk's sums, weighted
        const int c = idx / split, s = idx - c * split;
        const bool sh = L.expert[c] == a.E;
        const int start = L.start[c], cnt = L.count[c];
#pragma unroll
        for (int j2 = 0; j2 < 2; ++j2) {
          if (2 * t + j2 < cnt) {
            const int p = start + 2 * t + j2;
            const float al = sh ? a.s_shared[p] : a.alpha[L.sorted[p]];
            float* y = ysum + ((size_t)s * rows_all + (sh ? P : 0) + p) * kDnPitch;
            y[g] = al * acc[j2];
            y[g + 8] = al * acc[2 + j2];
          }
        }
        acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
      }
      at[j] = next;
      load_w(ring[j], next);
      load_x(ring[j], next);
      next.kb += split;
      settle(next);
    }
  }
  __syncthreads();
  for (int i = tid; i < a.T * kDnCols; i += kDnWarps * 32) {
    const int tok = i / kDnCols, c = i - tok * kDnCols;
    float y = 0.f;
    for (int sl = 0; sl < a.k; ++sl) {
      const int p = L.pos[tok * a.k + sl];
      for (int s = 0; s < min(split, KBr); ++s) y += ysum[((size_t)s * rows_all + p) * kDnPitch + c];
    }
    for (int s = 0; s < min(split, KBs); ++s)
      y += ysum[((size_t)s * rows_all + P + tok) * kDnPitch + c];
    const size_t o = (size_t)tok * a.d + col0 + c;
    if (a.r_attn) y += a.r_attn[o];
    if (a.out_bf16)
      static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(y);
    else
      static_cast<float*>(a.out)[o] = y;
  }
}

// ---------------------------------------------------------------------------
// product for a few rows
// ---------------------------------------------------------------------------
constexpr int kMmWarps = 16;
constexpr int kMmAhead = 3;

template <int NT>
struct MmUnit {
  WeightBlock w;
  float sw;
  ActBlock x[NT];
  float s0[NT], s1[NT];
};

// out[m][n] for M <= 8 NT rows: items of 16 output columns, k split over the
// warps of an item.
template <int NT>
__global__ void __launch_bounds__(kMmWarps * 32, 1) f8_few_matmul_kernel(F8MatmulArgs a) {
  __shared__ float4 part[2][NT][kMmWarps][32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int KB = f8_blocks(a.K);
  pdl_wait();
  pdl_trigger();
  int wpi = 1;
  while (wpi * 2 <= KB && wpi < kMmWarps) wpi *= 2;
  const int slots = kMmWarps / wpi, slot = warp / wpi, w = warp % wpi;
  const int items = (a.N + 15) / 16;
  const int stride = (int)gridDim.x * slots, rounds = (items + stride - 1) / stride;
  const int steps = (KB + wpi - 1) / wpi, units = rounds * steps;
  const int first = slot * (int)gridDim.x + (int)blockIdx.x;
  auto load = [&](MmUnit<NT>& u, int n) {
    const int r = n / steps, kb = (n - r * steps) * wpi + w;
    const int i = first + r * stride;
    u.w.lo[0] = u.w.lo[1] = u.w.hi[0] = u.w.hi[1] = zero4();
    u.sw = 0.f;
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      u.x[q].v[0] = u.x[q].v[1] = zero4();
      u.s0[q] = u.s1[q] = 0.f;
    }
    if (n >= units || i >= items || kb >= KB) return;
    const int k0 = kb * kF8Block + 16 * t;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = k0 + 64 * h, left = a.K - k;
      if (left <= 0) continue;
      const int lo = i * 16 + g, hi = lo + 8;
      if (lo < a.N) u.w.lo[h] = keep_bytes(ldg_stream(a.b + (size_t)lo * a.ldb + k), left);
      if (hi < a.N) u.w.hi[h] = keep_bytes(ldg_stream(a.b + (size_t)hi * a.ldb + k), left);
#pragma unroll
      for (int q = 0; q < NT; ++q)
        u.x[q].v[h] = keep_bytes(
            *reinterpret_cast<const uint4*>(a.a + (size_t)min(8 * q + g, a.M - 1) * a.lda + k),
            left);
    }
    u.sw = __ldg(a.b_scale + (size_t)(i * 16 / kF8Block) * KB + kb);
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      u.s0[q] = a.a_scale[(size_t)min(8 * q + 2 * t, a.M - 1) * KB + kb];
      u.s1[q] = a.a_scale[(size_t)min(8 * q + 2 * t + 1, a.M - 1) * KB + kb];
    }
  };
  MmUnit<NT> ring[kMmAhead];
#pragma unroll
  for (int j = 0; j < kMmAhead; ++j) load(ring[j], j);
  float acc[NT][4] = {};
  for (int n0 = 0; n0 < units; n0 += kMmAhead) {
#pragma unroll
    for (int j = 0; j < kMmAhead; ++j) {
      const int n = n0 + j;
      if (n >= units) break;
      const int r = n / steps, st = n - r * steps;
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        float d[4];
        block_mma(d, ring[j].w, ring[j].x[q].v[0], ring[j].x[q].v[1]);
        const float c0 = ring[j].sw * ring[j].s0[q], c1 = ring[j].sw * ring[j].s1[q];
        acc[q][0] = fmaf(d[0], c0, acc[q][0]);
        acc[q][1] = fmaf(d[1], c1, acc[q][1]);
        acc[q][2] = fmaf(d[2], c0, acc[q][2]);
        acc[q][3] = fmaf(d[3], c1, acc[q][3]);
      }
      load(ring[j], n + kMmAhead);
      if (st != steps - 1) continue;
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        part[r & 1][q][warp][lane] = make_float4(acc[q][0], acc[q][1], acc[q][2], acc[q][3]);
        acc[q][0] = acc[q][1] = acc[q][2] = acc[q][3] = 0.f;
      }
      __syncthreads();
      const int i = first + r * stride;
      if (i >= items || w != r % wpi) continue;
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        float4 v = part[r & 1][q][slot * wpi][lane];
        for (int p = 1; p < wpi; ++p) {
          const float4 o = part[r & 1][q][slot * wpi + p][lane];
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
}

size_t gateup_smem(int T, int d) {
  const int KB = f8_blocks(d);
  return few_lists_bytes() + 2 * kGuWarps * 32 * sizeof(float4) + (((size_t)T * KB * 4 + 15) & ~15) +
         (size_t)T * (KB * kF8Block + 64);
}
// Rows of partial sums: all pairs and shared tokens once, or fewer of them
// split up to kDnWarps ways (split x chunks stays below 2 kDnWarps, of 8 rows).
size_t down_smem(int T, int k) {
  const int rows = T * k + T;
  return few_lists_bytes() + (size_t)(rows > 16 * kDnWarps ? rows : 16 * kDnWarps) * kDnPitch * 4;
}

}  // namespace

static_assert(sizeof(FewLists) <= few_lists_bytes(), "few_lists_bytes covers the lists");

bool f8_few_ok(int T, int d, int k) {
  return T <= kF8FewTokens && T * k <= kFewMaxPairs && gateup_smem(T, d) <= 220 * 1024;
}

cudaError_t launch_f8_few_gateup(const F8ExpertsArgs& a, cudaStream_t st) {
  static int attr[64] = {};
  const size_t smem = gateup_smem(a.T, a.d);
  cudaError_t e = ensure_smem_limit(f8_few_gateup_kernel, (int)smem, attr);
  if (e != cudaSuccess) return e;
  return launch_pdl(f8_few_gateup_kernel, dim3(tc_sm_count()), kGuWarps * 32, smem, st, a);
}

cudaError_t launch_f8_few_down(const F8ExpertsArgs& a, cudaStream_t st) {
  static int attr[64] = {};
  const size_t smem = down_smem(a.T, a.k);
  cudaError_t e = ensure_smem_limit(f8_few_down_kernel, (int)smem, attr);
  if (e != cudaSuccess) return e;
  return launch_pdl(f8_few_down_kernel, dim3(a.d / kDnCols), kDnWarps * 32, smem, st, a);
}

cudaError_t launch_f8_few_matmul(const F8MatmulArgs& a, cudaStream_t st) {
  const int items = (a.N + 15) / 16;
  const int grid = items < tc_sm_count() ? items : tc_sm_count();
  return a.M <= 8 ? launch_pdl(f8_few_matmul_kernel<1>, dim3(grid), kMmWarps * 32, 0, st, a)
                  : launch_pdl(f8_few_matmul_kernel<2>, dim3(grid), kMmWarps * 32, 0, st, a);
}

}  // namespace moe
