// Entry points of the norm in front of a layer and of the 8-bit integer calls:
// argument checks, workspace plans and launch sequences. See
// include/moe_route.h.
#include "moe_route.h"

#include <stdint.h>

#include "common.cuh"
#include "fp8_common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kTileRows = 128;  // weight rows of a tile
constexpr int kStepK = 128;
constexpr int kSms = 152;       // SMs that a product is laid out for

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }
bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
int elem(int dtype) { return dtype == MOE_BF16 ? 2 : 4; }
bool value_type(int dtype) { return dtype == MOE_BF16 || dtype == MOE_F32; }

moe_status_t cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  set_last_cuda_error(e);
  return MOE_ERR_CUDA;
}

moe_status_t validate_mm(const moe_i8_matmul_t* m) {
  if (!m || m->M < 0 || m->N < 0 || m->K < 1) return MOE_ERR_INVALID_ARG;
  if (!value_type(m->out_dtype) || (m->gated != 0 && m->gated != 1)) return MOE_ERR_INVALID_ARG;
  if (m->lda < m->K || m->ldb < m->K || m->ldo < m->N) return MOE_ERR_INVALID_ARG;
  if (m->lda % 16 || m->ldb % 16) return MOE_ERR_INVALID_ARG;
  // a sum of more products could pass 2^31
  if (m->K > kI8MaxK) return MOE_ERR_UNSUPPORTED;
  // a tensor map's row pitch is below 2^40 bytes
  if (m->lda >= (1ll << 40) || m->ldb >= (1ll << 40) || m->ldo >= (1ll << 40)) return MOE_ERR_UNSUPPORTED;
  // the kernels count rows, columns and tiles (of 256 rows where there are more than a
  // wave: below 2^30) in 32 bits, and the widening launch its pieces
  if (m->N >= (1 << 30) || m->M >= (1 << 30) || (long long)m->M * m->N > (1ll << (m->gated ? 43 : 44)) ||
      (long long)m->M * m->K > (1ll << 40))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

struct MmPlan {
  I8Kind kind;
  int half, m_tiles, n_tiles;
  int pitch;  // of the widened rows
  size_t wide, total;
};
MmPlan mm_plan(const moe_i8_matmul_t& m) {
  MmPlan p{};
  p.wide = p.total = align256(sizeof(Ctrl));
  if (m.M <= kI8FewRows || m.N == 0) return p;
  p.half = m.M <= 16 ? 16 : m.M <= 32 ? 32 : m.M <= 64 ? 64 : 128;
  p.kind = kI8One;
  const int cols = m.gated ? kTileRows / 2 : kTileRows;
  p.n_tiles = (m.N + cols - 1) / cols;
  const auto tiles_of = [&](int rows) { return (long long)((m.M + rows - 1) / rows) * p.n_tiles; };
  // two blocks a tile where that leaves a tile for every second SM
  if (m.M > 128 && 2 * tiles_of(256) >= kSms) {
    p.kind = kI8Two;
  } else if (m.M > 32) {
    // Else the block of tokens that ends soonest by this estimate, in steps, among
    // those of one wave of tiles: the steps of a CTA, after cutting over a
    // cluster, and the read-back and sums behind them. us with blocks of 128 / 64 / 32:
    // 256 x 240 x 4608 12.3 / 10.3 / 9.8, 333 x 1001 x 1400 11.2 / 9.3 / 8.7, 128 x 4911 x
    // 1858 13.3 / 11.1 / 14.6, 4571 x 64 x 1328 15.0 / 12.8 / 14.6, 1536 x 1044 x 465 8.0 /
    // 10.2 / 11.1, 64 x 4096 x 4096 - / 12.1 / 13.2. It takes the slower of two at 333 x
    // 1001 x 1400.
    const int steps = (m.K + kStepK - 1) / kStepK;
    double best = 1e30;
    for (int half = p.half, h = half; h >= 32; h /= 2) {
      const long long tiles = tiles_of(h);
      if (tiles > kSms && h < half) break;
      int ks = tiles > 0 && tiles <= kSms ? (int)(kSms / tiles) : 1;
      if (ks > 8) ks = 8;
      if (ks > steps / 2) ks = steps / 2;
      const int end = h == 32 ? 3 : h == 64 ? 5 : steps <= 8 ? 6 : 15;  // (128: sums of up to 1024 stay fp32)
      double cost = steps + end;
      if (ks > 1 && (double)steps / ks + end + 3 < cost) cost = (double)steps / ks + end + 3;
      if (cost < best) {
        best = cost;
        p.half = h;
      }
    }
  }
  const int rows = p.half * (p.kind == kI8Two ? 2 : 1);
  p.m_tiles = (m.M + rows - 1) / rows;
  p.pitch = (m.K + 15) / 16 * 16;
  if (m.M > kI8FusedRows) p.total += align256((size_t)m.M * p.pitch * 2);
  return p;
}

moe_status_t check_workspace(const moe_i8_matmul_t* m, const MmPlan& p) {
  return !m->workspace || !aligned(m->workspace, 256) || m->workspace_bytes < p.total ? MOE_ERR_WORKSPACE : MOE_OK;
}

moe_status_t product(const void* a, const float* a_scale, const void* b0, const float* s0, const void* b1,
                     const float* s1, const moe_i8_matmul_t* mm, void* out, int gated, void* stream) {
  moe_status_t s = validate_mm(mm);
  if (s != MOE_OK) return s;
  if (mm->gated != gated) return MOE_ERR_INVALID_ARG;
  const MmPlan p = mm_plan(*mm);
  if ((s = check_workspace(mm, p)) != MOE_OK) return s;
  if (mm->M == 0 || mm->N == 0) return MOE_OK;
  const bool bf16 = mm->out_dtype == MOE_BF16;
  const void* codes[] = {a, b0, gated ? b1 : b0};
  const void* scales[] = {a_scale, s0, gated ? s1 : s0};
  for (int i = 0; i < 3; ++i) {
    if (!codes[i] || !aligned(codes[i], 16) || !scales[i] || !aligned(scales[i], 4)) return MOE_ERR_INVALID_ARG;
    if (out == codes[i] || out == scales[i]) return MOE_ERR_INVALID_ARG;
  }
  if (!out || !aligned(out, elem(mm->out_dtype))) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  if (mm->M <= kI8FewRows) {
    const I8FewArgs f{static_cast<const uint8_t*>(a), static_cast<const uint8_t*>(b0),
                      static_cast<const uint8_t*>(b1), a_scale, s0, s1, out, mm->M, mm->N, mm->K, bf16 ? 1 : 0,
                      mm->lda, mm->ldb, mm->ldo, 0};
    return cuda_status(run_kernel(MOE_KERNEL_I8_MATMUL, st, [&] { return launch_i8_few(f, gated != 0, st); }));
  }
  char* ws = static_cast<char*>(mm->workspace);
  const bool fused = mm->M <= kI8FusedRows;
  I8TcMaps m{};
  if ((!fused && !i8_make_map(&m.A, ws + p.wide, mm->M, mm->K, p.pitch, p.half)) ||
      !f8_make_map(&m.B0, b0, mm->N, mm->K, mm->ldb, gated ? kTileRows / 2 : kTileRows) ||
      (gated && !f8_make_map(&m.B1, b1, mm->N, mm->K, mm->ldb, kTileRows / 2))) {
    const cudaError_t e = cudaGetLastError();  // (set where the driver has no encoder)
    return cuda_status(e != cudaSuccess ? e : cudaErrorInvalidValue);
  }
  if (!gated) m.B1 = m.B0;  // (not read)
  if (fused) {
    m.A = m.B0;  // (not read)
  } else {
    const I8WidenArgs w{static_cast<const uint8_t*>(a), ws + p.wide, mm->M, mm->K, p.pitch, mm->lda};
    const cudaError_t e = run_kernel(MOE_KERNEL_I8_MATMUL, st, [&] { return launch_i8_widen(w, st); });
    if (e != cudaSuccess) return cuda_status(e);
  }
  I8TcArgs g{};
  g.a = static_cast<const uint8_t*>(a);
  g.lda = mm->lda;
  g.K = mm->K;
  g.a_scale = a_scale;
  g.b_scale0 = s0;
  g.b_scale1 = s1;
  g.out = out;
  g.ctrl = reinterpret_cast<Ctrl*>(ws);
  g.M = mm->M;
  g.N = mm->N;
  g.steps = (mm->K + kStepK - 1) / kStepK;
  g.m_tiles = p.m_tiles;
  g.n_tiles = p.n_tiles;
  g.out_bf16 = bf16 ? 1 : 0;
  g.ldo = mm->ldo;
  g.wait_ns = launch_wait_limit(MOE_KERNEL_I8_MATMUL, &g.stall);
  return cuda_status(run_kernel(MOE_KERNEL_I8_MATMUL, st,
                                [&] { return launch_i8_tc(p.kind, p.half, gated != 0, m, g, st); }));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_add_rmsnorm(const moe_rmsnorm_t* n, const void* x, const void* residual, const void* gain,
                             void* sum_out, void* out, void* codes, float* scales, void* stream) {
  if (!n || n->T < 0 || n->d < 1 || !(n->eps >= 0.f)) return MOE_ERR_INVALID_ARG;
  const int T = n->T, d = n->d;
  if (!value_type(n->x_dtype) || n->ldx < d) return MOE_ERR_INVALID_ARG;
  if (residual && (!value_type(n->residual_dtype) || n->ldr < d)) return MOE_ERR_INVALID_ARG;
  if (gain && !value_type(n->gain_dtype)) return MOE_ERR_INVALID_ARG;
  if (sum_out && (!value_type(n->sum_dtype) || n->lds < d)) return MOE_ERR_INVALID_ARG;
  if (out && (!value_type(n->out_dtype) || n->ldo < d)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;  // (tensors without rows may have no address)
  if (!codes != !scales) return MOE_ERR_INVALID_ARG;
  if (codes && ((n->codes_dtype != MOE_I8_ROW && n->codes_dtype != MOE_F8_E4M3_B128) || n->ldq < d))
    return MOE_ERR_INVALID_ARG;
  if (!sum_out && !out && !codes) return MOE_ERR_INVALID_ARG;
  if (d > kRowsMaxCols) return MOE_ERR_UNSUPPORTED;
  if (!x || !aligned(x, elem(n->x_dtype)) || (residual && !aligned(residual, elem(n->residual_dtype))) ||
      (gain && !aligned(gain, elem(n->gain_dtype))) || (sum_out && !aligned(sum_out, elem(n->sum_dtype))) ||
      (out && !aligned(out, elem(n->out_dtype))) || !aligned(scales, 4))
    return MOE_ERR_INVALID_ARG;
  // An output may take an input's place, value by value; nothing else may meet.
  const auto place = [&](const void* o, int dtype, int64_t ld) {
    return (o != x || (dtype == n->x_dtype && ld == n->ldx)) &&
           (o != residual || (dtype == n->residual_dtype && ld == n->ldr)) && o != gain;
  };
  if (sum_out && !place(sum_out, n->sum_dtype, n->lds)) return MOE_ERR_INVALID_ARG;
  if (out && (!place(out, n->out_dtype, n->ldo) || out == sum_out)) return MOE_ERR_INVALID_ARG;
  if (codes) {
    const void* other[] = {x, residual, gain, sum_out, out};
    for (const void* o : other)
      if (o && (o == codes || o == (const void*)scales)) return MOE_ERR_INVALID_ARG;
    if (codes == (void*)scales) return MOE_ERR_INVALID_ARG;
  }
  RowsArgs a{};
  a.x = x;
  a.residual = residual;
  a.gain = gain;
  a.sum = sum_out;
  a.out = out;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = scales;
  a.ldx = n->ldx;
  a.ldr = n->ldr;
  a.lds = n->lds;
  a.ldo = n->ldo;
  a.ldq = n->ldq;
  a.rows = T;
  a.cols = d;
  a.norm = 1;
  a.kind = !codes ? kRowsNone : n->codes_dtype == MOE_I8_ROW ? kRowsInt8 : kRowsE4m3;
  a.x_bf16 = n->x_dtype == MOE_BF16;
  a.res_bf16 = n->residual_dtype == MOE_BF16;
  a.gain_bf16 = n->gain_dtype == MOE_BF16;
  a.sum_bf16 = n->sum_dtype == MOE_BF16;
  a.out_bf16 = n->out_dtype == MOE_BF16;
  a.eps = n->eps;
  cudaStream_t st = (cudaStream_t)stream;
  return cuda_status(run_kernel(MOE_KERNEL_ADD_RMSNORM, st, [&] { return launch_rows(a, st); }));
}

moe_status_t moe_i8_quantize(const void* x, int32_t x_dtype, int64_t ldx, int32_t rows, int32_t cols, void* codes,
                             int64_t ldq, float* scales, void* stream) {
  if (!value_type(x_dtype) || rows < 0 || cols < 1 || ldx < cols || ldq < cols) return MOE_ERR_INVALID_ARG;
  if (cols > kRowsMaxCols) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  if (!x || !codes || !scales || !aligned(x, elem(x_dtype)) || !aligned(scales, 4)) return MOE_ERR_INVALID_ARG;
  if (codes == x || x == (const void*)scales || codes == (void*)scales) return MOE_ERR_INVALID_ARG;
  RowsArgs a{};
  a.x = x;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = scales;
  a.ldx = ldx;
  a.ldq = ldq;
  a.rows = rows;
  a.cols = cols;
  a.kind = kRowsInt8;
  a.x_bf16 = x_dtype == MOE_BF16;
  cudaStream_t st = (cudaStream_t)stream;
  return cuda_status(run_kernel(MOE_KERNEL_I8_QUANT, st, [&] { return launch_rows(a, st); }));
}

size_t moe_i8_matmul_workspace_bytes(const moe_i8_matmul_t* mm) {
  return validate_mm(mm) == MOE_OK ? mm_plan(*mm).total : 0;
}

int32_t moe_i8_matmul_form(const moe_i8_matmul_t* mm) {
  if (validate_mm(mm) != MOE_OK) return -1;
  const MmPlan p = mm_plan(*mm);
  return p.kind == kI8Two ? 2 * p.half : p.half;
}

moe_status_t moe_i8_matmul_init(const moe_i8_matmul_t* mm, void* stream) {
  moe_status_t s = validate_mm(mm);
  if (s != MOE_OK) return s;
  if ((s = check_workspace(mm, mm_plan(*mm))) != MOE_OK) return s;
  return cuda_status(cudaMemsetAsync(mm->workspace, 0, sizeof(Ctrl), (cudaStream_t)stream));
}

moe_status_t moe_i8_matmul(const void* a, const float* a_scale, const void* b, const float* b_scale,
                           const moe_i8_matmul_t* mm, void* out, void* stream) {
  return product(a, a_scale, b, b_scale, nullptr, nullptr, mm, out, 0, stream);
}

moe_status_t moe_i8_gated_matmul(const void* a, const float* a_scale, const void* gate, const float* gate_scale,
                                 const void* up, const float* up_scale, const moe_i8_matmul_t* mm, void* out,
                                 void* stream) {
  return product(a, a_scale, gate, gate_scale, up, up_scale, mm, out, 1, stream);
}

}  // extern "C"
