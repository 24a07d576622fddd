// C ABI of the feed-forward operators: argument checks, workspace layout and
// launches.  See include/mpopt.h for the contract of every entry point.

#include <cmath>

#include "../../include/mpopt.h"
#include "checks.h"
#include "internal.h"

namespace mpopt {
namespace {

// ------------------------------------------------------------ linear plan --

// Elements between rows of a copy whose rows start on 16 bytes.
int64_t packed_ld(int64_t cols, int es) { return static_cast<int64_t>(round_up(static_cast<size_t>(cols * es), 16)) / es; }

size_t packed_bytes(int64_t rows, int64_t cols, int es) {
  return round_up(static_cast<size_t>(rows) * static_cast<size_t>(packed_ld(cols, es)) * es, 256);
}

bool tma_readable(const void* p, int64_t ld, int64_t rows, int es) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (rows <= 1 || (ld * es) % 16 == 0);
}

// Hands out the workspace behind the header to operand copies; launch() makes
// them all at once.
struct Repacker {
  uint8_t* next;
  size_t left;
  int es;
  RepackBatch batch{};
  int64_t rows = 0, cols = 0;      // of the largest copy, for the launch record

  // `o` <- an operand of [rows][cols] elements that the TMA can read: the
  // caller's own, or a copy with 16-byte aligned rows.
  opt_status operand(const void* p, int64_t ld, int64_t n_rows, int64_t n_cols, int mn_major, LinearOperand* o) {
    if (tma_readable(p, ld, n_rows, es)) {
      *o = LinearOperand{p, n_rows > 1 ? ld : packed_ld(n_cols, es), mn_major};
      return OPT_OK;
    }
    const size_t bytes = packed_bytes(n_rows, n_cols, es);
    if (bytes > left) return OPT_ERR_WORKSPACE;
    const int64_t dst_ld = packed_ld(n_cols, es);
    batch.m[batch.n++] = RepackMatrix{p, next, ld, dst_ld, n_cols, n_rows * dst_ld * es / 16};
    if (n_rows * n_cols > rows * cols) {
      rows = n_rows;
      cols = n_cols;
    }
    *o = LinearOperand{next, dst_ld, mn_major};
    next += bytes;
    left -= bytes;
    return OPT_OK;
  }

  opt_status launch(cudaStream_t stream) {
    if (batch.n == 0) return OPT_OK;
    prof_begin(OPT_KERNEL_LINEAR_REPACK, batch.n, rows, cols, stream);
    const cudaError_t e = launch_repack(batch, es, stream);
    prof_end(stream);
    return cuda_status(e, "linear operand copies");
  }
};

// Bytes of the copies that operands with these bases and distances need.
size_t repack_need(const void* p, int64_t ld, int64_t rows, int64_t cols, int es) {
  return tma_readable(p, ld, rows, es) ? 0 : packed_bytes(rows, cols, es);
}

opt_status run_product(const LinearArgs& g, int kernel, int64_t m, int64_t n, cudaStream_t stream, const char* where) {
  prof_begin(kernel, 1, m, n, stream);
  const cudaError_t e = launch_linear(g, stream);
  prof_end(stream);
  return cuda_status(e, where);
}

bool extents_ok(int64_t m, int64_t n, int64_t k) {
  return m >= 0 && n >= 1 && k >= 1 && m <= kMaxExtent && n <= kMaxExtent && k <= kMaxExtent;
}

}  // namespace
}  // namespace mpopt

using namespace mpopt;

extern "C" {

opt_status opt_rmsnorm_forward(const opt_rmsnorm_args* a, void* stream) {
  if (!a || a->rows < 0 || a->cols < 1 || a->rows > kMaxExtent) return OPT_ERR_INVALID_ARG;
  if (!float_dtype(a->dtype) || !float_dtype(a->gamma_dtype)) return OPT_ERR_INVALID_ARG;
  if (!std::isfinite(a->eps) || a->eps < 0.f) return OPT_ERR_INVALID_ARG;
  if (!a->q != !a->q_scale) return OPT_ERR_INVALID_ARG;
  if (a->cols > kNormMaxCols) return OPT_ERR_UNSUPPORTED;
  if (a->rows == 0) return OPT_OK;
  const int es = elem_size(a->dtype);
  MPOPT_TRY(check_matrix(a->x, false, a->x_ld, a->rows, a->cols, es));
  MPOPT_TRY(check_matrix(a->residual, true, a->residual_ld, a->rows, a->cols, es));
  MPOPT_TRY(check_matrix(a->h, true, a->h_ld, a->rows, a->cols, es));
  MPOPT_TRY(check_matrix(a->y, true, a->y_ld, a->rows, a->cols, 2));
  MPOPT_TRY(check_matrix(a->q, true, a->q_ld, a->rows, a->cols, 1));
  MPOPT_TRY(check_vector(a->gamma, false, elem_size(a->gamma_dtype)));
  MPOPT_TRY(check_vector(a->q_scale, true, 4));
  MPOPT_TRY(check_vector(a->rstd, true, 4));
  const RmsnormArgs k{a->x,    a->residual, a->gamma, a->h,    a->y,     a->q,           a->q_scale,
                      a->rstd, a->rows,     a->cols,  a->x_ld, a->residual_ld, a->h_ld,  a->y_ld,
                      a->q_ld, a->dtype,    a->gamma_dtype, a->eps, 1};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  prof_begin(OPT_KERNEL_RMSNORM, 1, a->rows, a->cols, st);
  const cudaError_t e = launch_rmsnorm(k, st);
  prof_end(st);
  return cuda_status(e, "rmsnorm launch");
}

opt_status opt_quantize_rows(const void* x, int64_t x_ld, int32_t dtype, int64_t rows, int64_t cols, uint8_t* q,
                             int64_t q_ld, float* scale, void* stream) {
  if (rows < 0 || cols < 1 || rows > kMaxExtent || !float_dtype(dtype)) return OPT_ERR_INVALID_ARG;
  if (cols > kNormMaxCols) return OPT_ERR_UNSUPPORTED;
  if (rows == 0) return OPT_OK;
  MPOPT_TRY(check_matrix(x, false, x_ld, rows, cols, elem_size(dtype)));
  MPOPT_TRY(check_matrix(q, false, q_ld, rows, cols, 1));
  MPOPT_TRY(check_vector(scale, false, 4));
  RmsnormArgs k{};
  k.x = x;
  k.q = q;
  k.q_scale = scale;
  k.rows = rows;
  k.cols = cols;
  k.x_ld = x_ld;
  k.q_ld = q_ld;
  k.dtype = dtype;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  prof_begin(OPT_KERNEL_QUANTIZE, 1, rows, cols, st);
  const cudaError_t e = launch_rmsnorm(k, st);
  prof_end(st);
  return cuda_status(e, "quantize launch");
}

size_t opt_rmsnorm_workspace_size(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols < 1) return 0;
  return round_up(static_cast<size_t>(rows < kNormPartialRows ? rows : kNormPartialRows) * cols * 4, 256);
}

opt_status opt_rmsnorm_backward(const opt_rmsnorm_grad_args* a, void* workspace, size_t workspace_bytes,
                                void* stream) {
  if (!a || a->rows < 0 || a->cols < 1 || a->rows > kMaxExtent) return OPT_ERR_INVALID_ARG;
  if (!float_dtype(a->dtype) || !float_dtype(a->gamma_dtype)) return OPT_ERR_INVALID_ARG;
  if (a->cols > kNormGradMaxCols) return OPT_ERR_UNSUPPORTED;
  MPOPT_TRY(check_vector(a->dgamma, true, 4));
  if (a->rows > 0) {
    const int es = elem_size(a->dtype);
    MPOPT_TRY(check_matrix(a->dy, false, a->dy_ld, a->rows, a->cols, 2));
    MPOPT_TRY(check_matrix(a->h, false, a->h_ld, a->rows, a->cols, es));
    MPOPT_TRY(check_matrix(a->dh, true, a->dh_ld, a->rows, a->cols, es));
    MPOPT_TRY(check_matrix(a->dx, true, a->dx_ld, a->rows, a->cols, es));
    MPOPT_TRY(check_vector(a->gamma, false, elem_size(a->gamma_dtype)));
    MPOPT_TRY(check_vector(a->rstd, false, 4));
    if (a->dgamma) MPOPT_TRY(check_workspace(workspace, workspace_bytes, opt_rmsnorm_workspace_size(a->rows, a->cols)));
  }
  if (!a->dx && !a->dgamma) return OPT_OK;
  RmsnormGradArgs k{a->dy,   a->h,    a->gamma, a->rstd, a->dh,    a->dx,    a->dgamma, static_cast<float*>(workspace),
                    a->rows, a->cols, a->dy_ld, a->h_ld, a->dh_ld, a->dx_ld, a->dtype,  a->gamma_dtype,
                    a->accumulate};
  return cuda_status(launch_rmsnorm_grad(k, static_cast<cudaStream_t>(stream)), "rmsnorm gradient launch");
}

// Bytes of the bias gradient's partial sums.
static size_t column_sum_bytes(int64_t m, int64_t n) {
  const int64_t s = column_sum_slices(m, n);
  return s > 1 ? round_up(static_cast<size_t>(s) * static_cast<size_t>(n) * 4, 256) : 0;
}

size_t opt_linear_workspace_size(int64_t m, int64_t n, int64_t k, int32_t flags) {
  if (!extents_ok(m, n, k)) return 0;
  const bool any = (flags & OPT_LINEAR_ANY_LAYOUT) != 0;
  // 16-byte rows: k a multiple of 16 also serves 8-bit operands
  const size_t x_w = any || k % 16 ? packed_bytes(m, k, 2) + packed_bytes(n, k, 2) : 0;
  const size_t dz = any || n % 8 ? packed_bytes(m, n, 2) : 0;
  return kLinearHeaderBytes + x_w + dz + round_up(static_cast<size_t>(column_sum_most(m, n)) * 4, 256);
}

opt_status opt_linear_forward(const opt_linear_args* a, void* workspace, size_t workspace_bytes, void* stream) {
  if (!a || !extents_ok(a->m, a->n, a->k)) return OPT_ERR_INVALID_ARG;
  if (a->dtype != OPT_DTYPE_BF16 && a->dtype != OPT_DTYPE_E4M3) return OPT_ERR_INVALID_ARG;
  if (a->bias && !float_dtype(a->bias_dtype)) return OPT_ERR_INVALID_ARG;
  if (a->act < OPT_ACT_NONE || a->act > OPT_ACT_SILU) return OPT_ERR_INVALID_ARG;
  const bool fp8 = a->dtype == OPT_DTYPE_E4M3;
  if (!fp8 && (a->x_scale || a->w_scale)) return OPT_ERR_INVALID_ARG;
  if (a->m == 0) return OPT_OK;
  const int es = fp8 ? 1 : 2;
  MPOPT_TRY(check_matrix(a->x, false, a->x_ld, a->m, a->k, es));
  MPOPT_TRY(check_matrix(a->w, false, a->w_ld, a->n, a->k, es));
  MPOPT_TRY(check_vector(a->x_scale, !fp8, 4));
  MPOPT_TRY(check_vector(a->w_scale, !fp8, 4));
  MPOPT_TRY(check_vector(a->bias, true, elem_size(a->bias_dtype)));
  MPOPT_TRY(check_matrix(a->residual, true, a->residual_ld, a->m, a->n, 2));
  MPOPT_TRY(check_matrix(a->y, false, a->y_ld, a->m, a->n, 2));
  MPOPT_TRY(check_matrix(a->z, true, a->z_ld, a->m, a->n, 2));
  const size_t need = kLinearHeaderBytes + repack_need(a->x, a->x_ld, a->m, a->k, es) +
                      repack_need(a->w, a->w_ld, a->n, a->k, es);
  MPOPT_TRY(check_workspace(workspace, workspace_bytes, need));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  Repacker rp{static_cast<uint8_t*>(workspace) + kLinearHeaderBytes, workspace_bytes - kLinearHeaderBytes, es};
  LinearArgs g{};
  g.mode = kLinearForward;
  g.fp8 = fp8;
  MPOPT_TRY(rp.operand(a->w, a->w_ld, a->n, a->k, 0, &g.A));
  MPOPT_TRY(rp.operand(a->x, a->x_ld, a->m, a->k, 0, &g.B));
  MPOPT_TRY(rp.launch(st));
  g.na = a->n;
  g.nb = a->m;
  g.nk = a->k;
  g.a_scale = a->w_scale;
  g.b_scale = a->x_scale;
  g.bias = a->bias;
  g.bias_dtype = a->bias_dtype;
  g.act = a->act;
  g.residual = a->residual;
  g.residual_ld = a->residual_ld;
  g.y = a->y;
  g.y_ld = a->y_ld;
  g.z_out = a->z;
  g.z_ld = a->z_ld;
  g.header = static_cast<uint32_t*>(workspace);
  return run_product(g, OPT_KERNEL_LINEAR, a->m, a->n, st, "linear launch");
}

opt_status opt_linear_backward(const opt_linear_grad_args* a, void* workspace, size_t workspace_bytes, void* stream) {
  if (!a || !extents_ok(a->m, a->n, a->k)) return OPT_ERR_INVALID_ARG;
  if (a->act_prev < OPT_ACT_NONE || a->act_prev > OPT_ACT_SILU) return OPT_ERR_INVALID_ARG;
  if (a->dx && a->act_prev != OPT_ACT_NONE && !a->z_prev && a->m > 0) return OPT_ERR_INVALID_ARG;
  MPOPT_TRY(check_vector(a->dw, true, 4));
  MPOPT_TRY(check_vector(a->dbias, true, 4));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a->m == 0) {
    if (a->accumulate) return OPT_OK;
    if (a->dw) {
      const size_t bytes = static_cast<size_t>(a->n) * static_cast<size_t>(a->k) * 4;
      MPOPT_TRY(cuda_status(cudaMemsetAsync(a->dw, 0, bytes, st), "linear gradient clear"));
    }
    if (a->dbias)
      MPOPT_TRY(cuda_status(cudaMemsetAsync(a->dbias, 0, static_cast<size_t>(a->n) * 4, st), "linear gradient clear"));
    return OPT_OK;
  }
  if (!a->dx && !a->dw && !a->dbias) return OPT_OK;
  MPOPT_TRY(check_matrix(a->dz, false, a->dz_ld, a->m, a->n, 2));
  MPOPT_TRY(check_matrix(a->x, !a->dw, a->x_ld, a->m, a->k, 2));
  MPOPT_TRY(check_matrix(a->w, !a->dx, a->w_ld, a->n, a->k, 2));
  MPOPT_TRY(check_matrix(a->z_prev, true, a->z_prev_ld, a->m, a->k, 2));
  MPOPT_TRY(check_matrix(a->dx, true, a->dx_ld, a->m, a->k, 2));
  const size_t sums = a->dbias ? column_sum_bytes(a->m, a->n) : 0;
  const size_t products = a->dx || a->dw ? repack_need(a->dz, a->dz_ld, a->m, a->n, 2) +
                                               (a->dx ? repack_need(a->w, a->w_ld, a->n, a->k, 2) : 0) +
                                               (a->dw ? repack_need(a->x, a->x_ld, a->m, a->k, 2) : 0)
                                         : 0;
  if (a->dx || a->dw || sums) MPOPT_TRY(check_workspace(workspace, workspace_bytes, kLinearHeaderBytes + products + sums));
  uint8_t* const scratch = static_cast<uint8_t*>(workspace) + kLinearHeaderBytes;
  const ColumnSumArgs column_sums{a->dz,    a->dz_ld, a->m, a->n, a->dbias, reinterpret_cast<float*>(scratch),
                                  a->accumulate};
  if (a->dx || a->dw) {
    Repacker rp{scratch + sums, workspace_bytes - kLinearHeaderBytes - sums, 2};
    LinearOperand dz{}, w{}, x{};
    MPOPT_TRY(rp.operand(a->dz, a->dz_ld, a->m, a->n, 0, &dz));
    if (a->dx) MPOPT_TRY(rp.operand(a->w, a->w_ld, a->n, a->k, 1, &w));
    if (a->dw) MPOPT_TRY(rp.operand(a->x, a->x_ld, a->m, a->k, 1, &x));
    MPOPT_TRY(rp.launch(st));
    LinearArgs gx{};
    gx.mode = kLinearDx;
    gx.A = w;
    gx.B = dz;
    gx.na = a->k;
    gx.nb = a->m;
    gx.nk = a->n;
    gx.act = a->act_prev;
    gx.z_in = a->z_prev;
    gx.z_ld = a->z_prev_ld;
    gx.y = a->dx;
    gx.y_ld = a->dx_ld;
    gx.header = static_cast<uint32_t*>(workspace);
    LinearArgs gw{};
    gw.mode = kLinearDw;
    gw.A = x;
    gw.B = dz;
    gw.B.mn_major = 1;
    gw.na = a->k;
    gw.nb = a->n;
    gw.nk = a->m;
    gw.dw = a->dw;
    gw.dw_ld = a->k;
    gw.accumulate = a->accumulate;
    gw.header = static_cast<uint32_t*>(workspace);
    if (a->dx && a->dw && linear_grad_fits(gx, gw)) {
      const bool with_sums = a->dbias && column_sum_slices(a->m, a->n) == 1;
      prof_begin(OPT_KERNEL_LINEAR_GRAD, 1, a->m, a->n, st);
      const cudaError_t e = launch_linear_grad(gx, gw, with_sums ? &column_sums : nullptr, st);
      prof_end(st);
      MPOPT_TRY(cuda_status(e, "linear gradient launch"));
      if (with_sums) return OPT_OK;
    } else {
      if (a->dx) MPOPT_TRY(run_product(gx, OPT_KERNEL_LINEAR_DX, a->m, a->k, st, "linear dx launch"));
      if (a->dw) MPOPT_TRY(run_product(gw, OPT_KERNEL_LINEAR_DW, a->n, a->k, st, "linear dw launch"));
    }
  }
  if (a->dbias) {
    prof_begin(OPT_KERNEL_LINEAR_DBIAS, 1, a->m, a->n, st);
    const cudaError_t e = launch_column_sums(column_sums, st);
    prof_end(st);
    MPOPT_TRY(cuda_status(e, "linear bias gradient launch"));
  }
  return OPT_OK;
}

}  // extern "C"
