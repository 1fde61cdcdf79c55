// Entry points of the 8-bit calls: argument checks, workspace plans and launch
// sequences. See include/moe_route.h.
#include "moe_route.h"

#include <stdint.h>

#include "common.cuh"
#include "fp8_common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kBm = 128, kBn = 256;  // tile of the tensor-core products
constexpr int kSms = 152;            // SMs that a split product is laid out for

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }
bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

moe_status_t cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  set_last_cuda_error(e);
  return MOE_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// product
// ---------------------------------------------------------------------------
moe_status_t validate_mm(const moe_fp8_matmul_t* m) {
  if (!m || m->M < 0 || m->N < 0 || m->K < 1) return MOE_ERR_INVALID_ARG;
  if (m->out_dtype != MOE_BF16 && m->out_dtype != MOE_F32) return MOE_ERR_INVALID_ARG;
  if (m->lda < m->K || m->ldb < m->K || m->ldo < m->N) return MOE_ERR_INVALID_ARG;
  if (m->lda % 16 || m->ldb % 16) return MOE_ERR_INVALID_ARG;
  // a tensor map's row pitch is below 2^40 bytes
  if (m->lda >= (1ll << 40) || m->ldb >= (1ll << 40) || m->ldo >= (1ll << 40))
    return MOE_ERR_UNSUPPORTED;
  // the kernels count 16-column items and 128 x 256 tiles in 32 bits
  if (m->K > (1 << 30) || m->N > (1 << 30) || m->M > (1 << 30) ||
      ((long long)m->M / kBm + 1) * ((long long)m->N / kBn + 1) > (1ll << 26))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

struct MmPlan {
  int tiles, ksplit;
  size_t partial, total;
};
// Fewer tiles than half the SMs: k is split over CTAs, at least three blocks
// each.
MmPlan mm_plan(const moe_fp8_matmul_t& m) {
  MmPlan p{};
  p.tiles = ((m.M + kBm - 1) / kBm) * ((m.N + kBn - 1) / kBn);
  p.ksplit = 1;
  p.partial = p.total = align256(sizeof(Ctrl));
  if (m.M <= kF8FewTokens) return p;
  const int KB = f8_blocks(m.K);
  if (p.tiles > 0 && 2 * p.tiles <= kSms) {
    int s = kSms / p.tiles;
    if (s > KB / 3) s = KB / 3;
    if (s > 1) p.ksplit = s;
  }
  if (p.ksplit > 1) p.total = p.partial + (size_t)p.ksplit * p.tiles * kBm * kBn * 4;
  return p;
}

// ---------------------------------------------------------------------------
// layer
// ---------------------------------------------------------------------------
// The checks' view of an 8-bit layer's routing half: bf16, the separate kernels.
moe_cfg_t route_cfg(const moe_cfg_t& c) {
  moe_cfg_t r = c;
  r.expert_dtype = MOE_BF16;
  r.path = MOE_PATH_AUTO;
  return r;
}

// The two kernels for a few tokens, unless wide experts average three pairs or
// more each: mma.sync then meets every weight with several chunks' worth of
// columns, and the tensor-core products are faster. us, few / tensor cores (one
// call, L2 flushed before it): 256 experts T=8 58 / 75, T=16 92 / 100; 60 experts
// T=16 121 / 139; 8 wide experts T=4 189 / 194, T=8 253 / 251, T=12 287 / 251, T=16
// 329 / 253; the tiny shape T=16 (4 pairs each) 17 / 26. Between them the rule
// takes the slower side at one measured place: 64 experts of width 1408, T=12
// 104 / 112 but T=16 (1.5 pairs each) 122 / 114.
bool use_few(const moe_cfg_t& c) {
  if (c.path == MOE_PATH_TC || !f8_few_ok(c.T, c.d_model, c.top_k)) return false;
  if (c.path == MOE_PATH_GEMV) return true;
  const bool wide = (long long)c.d_model * c.d_ff >= (4ll << 20);
  return !(wide && c.T * c.top_k >= 3 * c.n_experts);
}

moe_status_t validate_f8(const moe_cfg_t* c) {
  if (!c) return MOE_ERR_INVALID_ARG;
  if (c->expert_dtype != MOE_F8_E4M3_B128) return MOE_ERR_INVALID_ARG;
  if (c->path < MOE_PATH_AUTO || c->path > MOE_PATH_FUSED) return MOE_ERR_INVALID_ARG;
  const moe_cfg_t r = route_cfg(*c);
  const moe_status_t s = validate_route_cfg(&r);
  if (s != MOE_OK) return s;
  if (c->act_dtype != MOE_BF16 || c->path == MOE_PATH_FUSED) return MOE_ERR_UNSUPPORTED;
  if (c->d_model % 16 || c->d_ff % 16 || c->d_ff_shared % 16) return MOE_ERR_UNSUPPORTED;
  if (c->path == MOE_PATH_GEMV && !f8_few_ok(c->T, c->d_model, c->top_k)) return MOE_ERR_UNSUPPORTED;
  // rows and row blocks are counted in 32 bits, tensor maps in 2^31 rows
  const long long widest = c->d_model > c->d_ff ? c->d_model : c->d_ff;
  if (((long long)c->T + 1) * (c->top_k + 1) > (1ll << 28) || widest * c->n_experts >= (1ll << 31))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Scales of a row of h, routed or shared.
int h_blocks(const moe_cfg_t& c) { return f8_blocks(c.d_ff > c.d_ff_shared ? c.d_ff : c.d_ff_shared); }

struct F8Plan {
  RoutePlan r;
  int hblocks;
  size_t xq, xs, Hf, Hq, Hs, Y, total;
};
F8Plan f8_plan(const moe_cfg_t& c) {
  F8Plan p{};
  p.r = route_plan(c);
  size_t off = p.r.end;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += align256(bytes);
    return o;
  };
  const size_t T = c.T, P = T * c.top_k, d = c.d_model;
  p.hblocks = h_blocks(c);
  const size_t ldh = (size_t)p.hblocks * kF8Block;
  const bool few = c.T <= kF8FewTokens;
  p.xq = take((P + T) * d);
  p.xs = take((P + T) * f8_blocks(c.d_model) * 4);
  p.Hf = take(few ? (P + T) * ldh * 4 : 0);
  p.Hq = take((P + T) * ldh);
  p.Hs = take((P + T) * p.hblocks * 4);
  p.Y = take((P + T) * d * 4);
  p.total = off;
  return p;
}

template <typename T>
T* at(const moe_cfg_t* c, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(c->workspace) + off);
}

moe_status_t check_workspace(const moe_cfg_t* c) {
  if (!c->workspace || !aligned(c->workspace, 256)) return MOE_ERR_WORKSPACE;
  return c->workspace_bytes < f8_plan(*c).total ? MOE_ERR_WORKSPACE : MOE_OK;
}

bool bank_ok(const moe_bank_t& b) {
  return b.w && b.scale && aligned(b.w, 16) && aligned(b.scale, 16);
}

struct Banks {
  moe_bank_t gate, up, down, s_gate, s_up, s_down;
};

moe_status_t check_tensors(const void* x, const float* r_attn, const int32_t* ids, const float* w,
                           const Banks& b, const moe_cfg_t* c, const void* out, int out_dtype) {
  if (out_dtype != MOE_BF16 && out_dtype != MOE_F32) return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {x, ids, w, out};
  for (const void* q : ptrs)
    if (!q || !aligned(q, 16)) return MOE_ERR_INVALID_ARG;
  if (r_attn && !aligned(r_attn, 16)) return MOE_ERR_INVALID_ARG;
  if (!bank_ok(b.gate) || !bank_ok(b.up) || !bank_ok(b.down)) return MOE_ERR_INVALID_ARG;
  if (c->d_ff_shared > 0 && (!bank_ok(b.s_gate) || !bank_ok(b.s_up) || !bank_ok(b.s_down)))
    return MOE_ERR_INVALID_ARG;
  if (out == x || (out == (const void*)r_attn && out_dtype != MOE_F32)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

const uint8_t* codes(const moe_bank_t& b) { return static_cast<const uint8_t*>(b.w); }
const float* scales(const moe_bank_t& b) { return static_cast<const float*>(b.scale); }

moe_status_t enqueue_few(const void* x, const float* r_attn, const int32_t* ids, const float* w,
                         const float* s_shared, const Banks& b, const moe_cfg_t* c, void* out,
                         int out_dtype, cudaStream_t st) {
  const F8Plan p = f8_plan(*c);
  F8ExpertsArgs a{};
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.ids = ids;
  a.alpha = w;
  a.s_shared = s_shared;
  a.r_attn = r_attn;
  a.Wg = codes(b.gate); a.Wu = codes(b.up); a.Wd = codes(b.down);
  a.Sg = scales(b.gate); a.Su = scales(b.up); a.Sd = scales(b.down);
  a.Wsg = codes(b.s_gate); a.Wsu = codes(b.s_up); a.Wsd = codes(b.s_down);
  a.Ssg = scales(b.s_gate); a.Ssu = scales(b.s_up); a.Ssd = scales(b.s_down);
  a.Hf = at<float>(c, p.Hf);
  a.Hq = at<uint8_t>(c, p.Hq);
  a.Hs = at<float>(c, p.Hs);
  a.counters = at<unsigned>(c, p.r.f8_counters);
  a.out = out;
  a.ctrl = at<Ctrl>(c, 0);
  a.T = c->T; a.d = c->d_model; a.E = c->n_experts; a.k = c->top_k;
  a.I = c->d_ff; a.Is = c->d_ff_shared;
  a.hblocks = p.hblocks;
  a.ldh = p.hblocks * kF8Block;
  a.out_bf16 = out_dtype == MOE_BF16;
  const uint64_t E = a.E, d = a.d, I = a.I, Is = a.Is, rows = (uint64_t)a.T * a.k + a.T;
  F8FewMaps m;
  bool ok = f8_make_map(&m.g, a.Wg, E * I, d, d, 16) && f8_make_map(&m.u, a.Wu, E * I, d, d, 16) &&
            f8_make_map(&m.w, a.Wd, E * d, I, I, 16) && f8_make_map(&m.x, a.Hq, rows, a.ldh, a.ldh, 8);
  if (ok && Is)
    ok = f8_make_map(&m.sg, a.Wsg, Is, d, d, 16) && f8_make_map(&m.su, a.Wsu, Is, d, d, 16) &&
         f8_make_map(&m.sw, a.Wsd, d, Is, Is, 16);
  if (!ok) return MOE_ERR_CUDA;
  if (!Is) {
    m.sg = m.g;
    m.su = m.u;
    m.sw = m.w;
  }
  m.sx = m.x;
  // (armed as the layer's gate/up and down, whichever kernels run them)
  a.wait_ns = launch_wait_limit(MOE_KERNEL_F8_TC_GATEUP, &a.stall);
  cudaError_t e =
      run_kernel(MOE_KERNEL_F8_FEW_GATEUP, st, [&] { return launch_f8_few_gateup(m, a, st); });
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  a.wait_ns = launch_wait_limit(MOE_KERNEL_F8_TC_DOWN, &a.stall);
  return cuda_status(run_kernel(MOE_KERNEL_F8_FEW_DOWN, st, [&] { return launch_f8_few_down(m, a, st); }));
}

moe_status_t enqueue_bucket(const int32_t* ids, const moe_cfg_t* c, const RoutePlan& r,
                            int shared_rows, cudaStream_t st) {
  BucketArgs b{};
  b.ids = ids;
  b.counts = at<int32_t>(c, r.counts);
  b.offsets = at<int32_t>(c, r.offsets);
  b.active = at<int32_t>(c, r.active);
  b.n_active = &at<Ctrl>(c, 0)->n_active;
  b.perm = at<int32_t>(c, r.perm);
  b.pos = at<int32_t>(c, r.pos);
  b.ctrl = at<Ctrl>(c, 0);
  b.P = c->T * c->top_k;
  b.E = c->n_experts;
  b.rowblocks = at<int2>(c, r.rowblocks);
  b.n_rowblocks = &at<Ctrl>(c, 0)->n_rowblocks;
  b.bm = kBm;
  b.shared_rows = shared_rows;
  if (bucket_ctas(b.P) == 1)
    return cuda_status(run_kernel(MOE_KERNEL_BUCKET, st, [&] { return launch_bucket(b, st); }));
  int* hist = at<int>(c, r.cta_hist);
  cudaError_t e = run_kernel(MOE_KERNEL_BUCKET, st, [&] { return launch_bucket_hist(b, hist, st); });
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  return cuda_status(run_kernel(MOE_KERNEL_BUCKET, st, [&] { return launch_bucket_pack(b, hist, st); }));
}

// Bucketing, quantised rows in packed order, grouped gate/up and down, combine.
// A shared expert as wide as the routed ones is one more group of the grouped
// products; one of another width runs as its own launches of the same kernels.
moe_status_t enqueue_tc(const void* x, const float* r_attn, const int32_t* ids, const float* w,
                        const float* s_shared, const Banks& b, const moe_cfg_t* c, void* out,
                        int out_dtype, cudaStream_t st) {
  const F8Plan p = f8_plan(*c);
  const int T = c->T, d = c->d_model, E = c->n_experts, k = c->top_k, P = T * k;
  const int I = c->d_ff, Is = c->d_ff_shared, ldh = p.hblocks * kF8Block;
  const bool apart = Is > 0 && Is != I, with = Is > 0 && !apart;
  moe_status_t s = enqueue_bucket(ids, c, p.r, with ? T : 0, st);
  if (s != MOE_OK) return s;
  uint8_t* xq = at<uint8_t>(c, p.xq);
  uint8_t* Hq = at<uint8_t>(c, p.Hq);
  float* Y = at<float>(c, p.Y);
  const F8PackArgs pk{static_cast<const __nv_bfloat16*>(x), at<int32_t>(c, p.r.pos), xq,
                      at<float>(c, p.xs), T, d, k, Is > 0 ? 1 : 0};
  cudaError_t e = run_kernel(MOE_KERNEL_F8_QUANT, st, [&] { return launch_f8_pack(pk, st); });
  if (e != cudaSuccess) return MOE_ERR_CUDA;

  const int t_rb = (T + kBm - 1) / kBm;
  const int max_rb = P / kBm + (P < E ? P : E) + 1 + (with ? t_rb : 0);
  F8TcArgs a{};
  a.rowblocks = at<int2>(c, p.r.rowblocks);
  a.n_rowblocks = &at<Ctrl>(c, 0)->n_rowblocks;
  a.offsets = at<int32_t>(c, p.r.offsets);
  a.perm = at<int32_t>(c, p.r.perm);
  a.alpha = w;
  a.s_shared = s_shared;
  a.ctrl = at<Ctrl>(c, 0);
  a.E = E;
  a.T = T;
  a.P = P;
  a.ksplit = 1;
  const uint64_t rows = (uint64_t)P + T;
  const auto map = [&](CUtensorMap* m, const moe_bank_t& bk, uint64_t n, int K, uint32_t box) {
    return f8_make_map(m, bk.w, n, K, K, box);
  };

  // gate/up over the routed groups (and the shared one), or over the shared
  // expert alone
  auto gateup = [&](bool alone) -> moe_status_t {
    const int width = alone ? Is : I;
    F8TcMaps m{};
    bool ok = f8_make_map(&m.A, xq, rows, d, d, kBm);
    if (!alone)
      ok = ok && map(&m.B0, b.gate, (uint64_t)E * I, d, kBn / 2) &&
           map(&m.B1, b.up, (uint64_t)E * I, d, kBn / 2);
    if (alone || with)
      ok = ok && map(&m.B2, b.s_gate, Is, d, kBn / 2) && map(&m.B3, b.s_up, Is, d, kBn / 2);
    if (!ok) return MOE_ERR_CUDA;
    if (alone) {
      m.B0 = m.B2;
      m.B1 = m.B3;
    } else if (!with) {
      m.B2 = m.B0;
      m.B3 = m.B1;
    }
    F8TcArgs g = a;
    g.shared_only = alone ? 1 : 0;
    g.a_scale = at<float>(c, p.xs);
    g.a_blocks = f8_blocks(d);
    g.b_scale0 = scales(b.gate);
    g.b_scale1 = scales(b.up);
    g.b_scale2 = scales(b.s_gate);
    g.b_scale3 = scales(b.s_up);
    g.out = Hq;
    g.ldo = ldh;
    g.out_scale = at<float>(c, p.Hs);
    g.out_blocks = p.hblocks;
    g.K = d;
    g.n_cols = width;
    g.n_tiles = f8_blocks(width);
    g.brows = width;
    g.b_blocks = f8_blocks(width);
    g.wait_ns = launch_wait_limit(MOE_KERNEL_F8_TC_GATEUP, &g.stall);
    const int items = (alone ? t_rb : max_rb) * g.n_tiles;
    return cuda_status(run_kernel(MOE_KERNEL_F8_TC_GATEUP, st,
                                  [&] { return launch_f8_tc(kF8GateUp, m, g, items, st); }));
  };
  auto down = [&](bool alone) -> moe_status_t {
    const int K = alone ? Is : I;
    F8TcMaps m{};
    bool ok = f8_make_map(&m.A, Hq, rows, K, ldh, kBm);
    if (!alone) ok = ok && map(&m.B0, b.down, (uint64_t)E * d, I, kBn);
    if (alone || with) ok = ok && map(&m.B2, b.s_down, d, Is, kBn);
    if (!ok) return MOE_ERR_CUDA;
    if (alone) m.B0 = m.B2;
    if (!alone && !with) m.B2 = m.B0;
    m.B1 = m.B0;
    m.B3 = m.B2;
    F8TcArgs g = a;
    g.shared_only = alone ? 1 : 0;
    g.a_scale = at<float>(c, p.Hs);
    g.a_blocks = p.hblocks;
    g.b_scale0 = g.b_scale1 = scales(b.down);
    g.b_scale2 = g.b_scale3 = scales(b.s_down);
    g.out = Y;
    g.ldo = d;
    g.K = K;
    g.n_cols = d;
    g.n_tiles = (d + kBn - 1) / kBn;
    g.brows = d;
    g.b_blocks = f8_blocks(d);
    g.wait_ns = launch_wait_limit(MOE_KERNEL_F8_TC_DOWN, &g.stall);
    const int items = (alone ? t_rb : max_rb) * g.n_tiles;
    return cuda_status(run_kernel(MOE_KERNEL_F8_TC_DOWN, st,
                                  [&] { return launch_f8_tc(kF8Down, m, g, items, st); }));
  };
  if ((s = gateup(false)) != MOE_OK) return s;
  if (apart && (s = gateup(true)) != MOE_OK) return s;
  if ((s = down(false)) != MOE_OK) return s;
  if (apart && (s = down(true)) != MOE_OK) return s;
  const CombineRowsArgs cb{r_attn, Y, at<int32_t>(c, p.r.pos), out, T, d, k, Is > 0 ? 1 : 0,
                           out_dtype == MOE_BF16};
  return cuda_status(run_kernel(MOE_KERNEL_COMBINE, st, [&] { return launch_combine_rows(cb, st); }));
}

moe_status_t enqueue_experts(const void* x, const float* r_attn, const int32_t* ids, const float* w,
                             const float* s_shared, const Banks& b, const moe_cfg_t* c, void* out,
                             int out_dtype, cudaStream_t st) {
  return use_few(*c) ? enqueue_few(x, r_attn, ids, w, s_shared, b, c, out, out_dtype, st)
                     : enqueue_tc(x, r_attn, ids, w, s_shared, b, c, out, out_dtype, st);
}

}  // namespace

// A count for every chunk (at most one a pair, and two of the shared expert's)
// and block of h that a call of the few-token kernels can have.
size_t f8_counter_bytes(const moe_cfg_t& c) {
  return ((size_t)kF8FewTokens * c.top_k + 2) * h_blocks(c) * sizeof(unsigned);
}

cudaError_t f8_reset_counters(const moe_cfg_t& c, cudaStream_t st) {
  if (c.expert_dtype != MOE_F8_E4M3_B128 || validate_f8(&c) != MOE_OK || check_workspace(&c) != MOE_OK)
    return cudaSuccess;
  const RoutePlan r = route_plan(c);
  return cudaMemsetAsync(at<char>(&c, r.f8_counters), 0, r.f8_counters_bytes, st);
}

}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_fp8_quantize(const void* x, int32_t x_dtype, int64_t ldx, int32_t count,
                              int32_t rows, int32_t cols, int32_t block_rows, void* codes,
                              int64_t ldq, float* scales, void* stream) {
  if (x_dtype != MOE_BF16 && x_dtype != MOE_F32) return MOE_ERR_INVALID_ARG;
  if (count < 0 || rows < 0 || cols < 0 || ldx < cols || ldq < cols) return MOE_ERR_INVALID_ARG;
  if (block_rows != 1 && block_rows != kF8Block) return MOE_ERR_INVALID_ARG;
  if (count == 0 || rows == 0 || cols == 0) return MOE_OK;
  if (!x || !codes || !scales) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, x_dtype == MOE_BF16 ? 2 : 4) || !aligned(scales, 4)) return MOE_ERR_INVALID_ARG;
  if ((long long)count * rows > 0x7FFFFFFFll || cols > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  if (block_rows == kF8Block &&
      (long long)count * f8_blocks(rows) * f8_blocks(cols) > 0x7FFFFFFFll)
    return MOE_ERR_UNSUPPORTED;
  const F8QuantArgs a{x, static_cast<uint8_t*>(codes), scales, rows, cols, count, ldx, ldq};
  cudaStream_t st = (cudaStream_t)stream;
  return cuda_status(run_kernel(MOE_KERNEL_F8_QUANT, st, [&] {
    return launch_f8_quant(a, x_dtype == MOE_BF16, block_rows != 1, st);
  }));
}

size_t moe_fp8_matmul_workspace_bytes(const moe_fp8_matmul_t* mm) {
  return validate_mm(mm) == MOE_OK ? mm_plan(*mm).total : 0;
}

moe_status_t moe_fp8_matmul_init(const moe_fp8_matmul_t* mm, void* stream) {
  const moe_status_t s = validate_mm(mm);
  if (s != MOE_OK) return s;
  const MmPlan p = mm_plan(*mm);
  if (!mm->workspace || !aligned(mm->workspace, 256) || mm->workspace_bytes < p.total)
    return MOE_ERR_WORKSPACE;
  return cuda_status(cudaMemsetAsync(mm->workspace, 0, sizeof(Ctrl), (cudaStream_t)stream));
}

moe_status_t moe_fp8_matmul(const void* a, const float* a_scale, const void* b, const float* b_scale,
                            const moe_fp8_matmul_t* mm, void* out, void* stream) {
  moe_status_t s = validate_mm(mm);
  if (s != MOE_OK) return s;
  const MmPlan p = mm_plan(*mm);
  if (!mm->workspace || !aligned(mm->workspace, 256) || mm->workspace_bytes < p.total)
    return MOE_ERR_WORKSPACE;
  if (mm->M == 0 || mm->N == 0) return MOE_OK;
  const bool bf16 = mm->out_dtype == MOE_BF16;
  if (!a || !a_scale || !b || !b_scale || !out) return MOE_ERR_INVALID_ARG;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(a_scale, 4) || !aligned(b_scale, 4) ||
      !aligned(out, bf16 ? 2 : 4))
    return MOE_ERR_INVALID_ARG;
  if (out == a || out == b || out == (const void*)a_scale || out == (const void*)b_scale)
    return MOE_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  if (mm->M <= kF8FewTokens) {
    F8MatmulArgs f{static_cast<const uint8_t*>(a), a_scale, static_cast<const uint8_t*>(b),
                   b_scale, out, static_cast<Ctrl*>(mm->workspace), mm->M, mm->N, mm->K, bf16 ? 1 : 0,
                   mm->lda, mm->ldb, mm->ldo, 0, 0};
    f.wait_ns = launch_wait_limit(MOE_KERNEL_F8_MATMUL, &f.stall);
    return cuda_status(run_kernel(MOE_KERNEL_F8_MATMUL, st, [&] { return launch_f8_few_matmul(f, st); }));
  }
  F8TcMaps m{};
  if (!f8_make_map(&m.A, a, mm->M, mm->K, mm->lda, kBm) ||
      !f8_make_map(&m.B0, b, mm->N, mm->K, mm->ldb, kBn))
    return MOE_ERR_CUDA;
  m.B1 = m.B2 = m.B3 = m.B0;
  char* ws = static_cast<char*>(mm->workspace);
  F8TcArgs g{};
  g.a_scale = a_scale;
  g.b_scale0 = g.b_scale1 = g.b_scale2 = g.b_scale3 = b_scale;
  g.out = out;
  g.partial = reinterpret_cast<float*>(ws + p.partial);
  g.ctrl = reinterpret_cast<Ctrl*>(ws);
  g.K = mm->K;
  g.rows = mm->M;
  g.n_cols = mm->N;
  g.n_tiles = (mm->N + kBn - 1) / kBn;
  g.b_blocks = f8_blocks(mm->N);
  g.a_blocks = f8_blocks(mm->K);
  g.ldo = mm->ldo;
  g.ksplit = p.ksplit;
  g.out_bf16 = bf16 ? 1 : 0;
  g.out_vec = aligned(out, 16) && (mm->ldo * (bf16 ? 2 : 4)) % 16 == 0 ? 1 : 0;
  g.wait_ns = launch_wait_limit(MOE_KERNEL_F8_MATMUL, &g.stall);
  cudaError_t e = run_kernel(MOE_KERNEL_F8_MATMUL, st, [&] {
    return launch_f8_tc(kF8Dense, m, g, p.tiles * p.ksplit, st);
  });
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  if (p.ksplit == 1) return MOE_OK;
  return cuda_status(run_kernel(MOE_KERNEL_F8_MATMUL, st, [&] { return launch_f8_split_sum(g, st); }));
}

size_t moe_fp8_workspace_bytes(const moe_cfg_t* cfg) {
  const moe_status_t s = validate_f8(cfg);
  return s == MOE_OK ? f8_plan(*cfg).total : 0;
}

moe_status_t moe_fp8_workspace_init(const moe_cfg_t* cfg, void* stream) {
  const moe_status_t s = validate_f8(cfg);
  if (s != MOE_OK) return s;
  const moe_status_t e = check_workspace(cfg);
  if (e != MOE_OK) return e;
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t c = cudaMemsetAsync(cfg->workspace, 0, sizeof(Ctrl), st);
  return cuda_status(c == cudaSuccess ? f8_reset_counters(*cfg, st) : c);
}

moe_status_t moe_fp8_experts_forward(const void* x, const float* r_attn, const int32_t* topk_ids,
                                     const float* weights, const float* s_shared, moe_bank_t W_gate,
                                     moe_bank_t W_up, moe_bank_t W_down, moe_bank_t Ws_gate,
                                     moe_bank_t Ws_up, moe_bank_t Ws_down, const void* w_shared,
                                     const moe_cfg_t* cfg, void* out, int32_t out_dtype,
                                     void* stream) {
  moe_status_t s = validate_f8(cfg);
  if (s != MOE_OK) return s;
  if ((s = check_workspace(cfg)) != MOE_OK) return s;
  if (cfg->T == 0) return MOE_OK;
  const Banks b{W_gate, W_up, W_down, Ws_gate, Ws_up, Ws_down};
  if ((s = check_tensors(x, r_attn, topk_ids, weights, b, cfg, out, out_dtype)) != MOE_OK) return s;
  cudaStream_t st = (cudaStream_t)stream;
  if (cfg->d_ff_shared > 0) {
    if (!s_shared && !w_shared) return MOE_ERR_INVALID_ARG;
    if ((s_shared && !aligned(s_shared, 16)) || (w_shared && !aligned(w_shared, 16)))
      return MOE_ERR_INVALID_ARG;
    if (!s_shared) {
      float* gate = at<float>(cfg, f8_plan(*cfg).r.s_shared);
      const RouterArgs ra{x, nullptr, w_shared, nullptr, cfg->T, cfg->d_model, 0};
      cudaError_t e = run_kernel(MOE_KERNEL_SHARED_GATE, st,
                                 [&] { return launch_shared_gate(ra, gate, true, st); });
      if (e != cudaSuccess) return MOE_ERR_CUDA;
      s_shared = gate;
    }
  }
  return enqueue_experts(x, r_attn, topk_ids, weights, s_shared, b, cfg, out, out_dtype, st);
}

moe_status_t moe_fp8_layer_forward(const void* x, const float* r_attn, const void* W_router,
                                   const float* expert_bias, moe_bank_t W_gate, moe_bank_t W_up,
                                   moe_bank_t W_down, moe_bank_t Ws_gate, moe_bank_t Ws_up,
                                   moe_bank_t Ws_down, const void* w_shared, const moe_cfg_t* cfg,
                                   void* out, int32_t out_dtype, int32_t* topk_ids, float* weights,
                                   void* stream) {
  moe_status_t s = validate_f8(cfg);
  if (s != MOE_OK) return s;
  if ((s = check_workspace(cfg)) != MOE_OK) return s;
  if (cfg->T == 0) return MOE_OK;
  const Banks b{W_gate, W_up, W_down, Ws_gate, Ws_up, Ws_down};
  if ((s = check_tensors(x, r_attn, topk_ids, weights, b, cfg, out, out_dtype)) != MOE_OK) return s;
  if (!W_router || !aligned(W_router, 16)) return MOE_ERR_INVALID_ARG;
  if (expert_bias && !aligned(expert_bias, 16)) return MOE_ERR_INVALID_ARG;
  const bool shared = cfg->d_ff_shared > 0;
  if (shared && (!w_shared || !aligned(w_shared, 16))) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  float* gate = shared ? at<float>(cfg, f8_plan(*cfg).r.s_shared) : nullptr;
  s = route_chain(x, W_router, expert_bias, shared ? w_shared : nullptr, cfg, topk_ids, weights, gate,
                  st);
  if (s != MOE_OK) return s;
  return enqueue_experts(x, r_attn, topk_ids, weights, gate, b, cfg, out, out_dtype, st);
}

}  // extern "C"
