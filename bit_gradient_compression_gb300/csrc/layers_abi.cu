// Entry points of the layers (declared in include/loco.h): argument checks and
// dispatch.  As in abi.cu, everything is checked on the host before anything is
// launched, so a refused call writes nothing.
#include <math.h>

#include "layers_args.h"
#include "layers_internal.h"
#include "steps_internal.h"

namespace loco {

namespace {

loco_status check_norm(const loco_norm_config* cfg, int64_t rows, int64_t cols) {
  if (cfg == nullptr) return fail(LOCO_ERR_INVALID_ARG, "cfg is NULL");
  if (cfg->kind != LOCO_NORM_LAYER && cfg->kind != LOCO_NORM_RMS)
    return fail(LOCO_ERR_UNSUPPORTED, "kind = %d (LOCO_NORM_LAYER or LOCO_NORM_RMS)", cfg->kind);
  if (!(cfg->eps >= 0.0f) || !isfinite(cfg->eps))
    return fail(LOCO_ERR_INVALID_ARG, "eps = %g must be finite and >= 0", cfg->eps);
  LOCO_TRY(check_dtype(cfg->x_dtype, "x_dtype"));
  LOCO_TRY(check_dtype(cfg->y_dtype, "y_dtype"));
  LOCO_TRY(check_dtype(cfg->param_dtype, "param_dtype"));
  LOCO_TRY(check_dtype(cfg->grad_dtype, "grad_dtype"));
  LOCO_TRY(check_dim(rows, 0, "rows"));
  return check_dim(cols, 1, "cols");
}

loco_status check_linear(const loco_linear_config* cfg, int64_t T, int64_t N, int64_t K) {
  if (cfg == nullptr) return fail(LOCO_ERR_INVALID_ARG, "cfg is NULL");
  LOCO_TRY(check_dtype(cfg->out_dtype, "out_dtype"));
  LOCO_TRY(check_dtype(cfg->param_dtype, "param_dtype"));
  LOCO_TRY(check_dim(T, 0, "T"));
  LOCO_TRY(check_dim(N, 0, "N"));
  return check_dim(K, 0, "K");
}

}  // namespace

}  // namespace loco

using namespace loco;

extern "C" {

int64_t loco_ckpt_code_bytes(int64_t rows, int64_t cols) {
  if (rows < 1 || rows > kMaxDim || cols < 1 || cols > kMaxDim) return 0;
  return rows * ((cols + kCkptBlock - 1) / kCkptBlock) * kCkptBlock;
}

int64_t loco_ckpt_scale_bytes(int64_t rows, int64_t cols) {
  if (rows < 1 || rows > kMaxDim || cols < 1 || cols > kMaxDim) return 0;
  return rows * ((cols + kCkptBlock - 1) / kCkptBlock);
}

int64_t loco_norm_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || rows > kMaxDim || cols < 1 || cols > kMaxDim) return 0;
  const int64_t parts = rows < kNormPartials ? (rows < 1 ? 1 : rows) : kNormPartials;
  return parts * 2 * cols * int64_t(sizeof(float));
}

int64_t loco_linear_workspace_bytes(int64_t N) {
  if (N < 1 || N > kMaxDim) return 0;
  return N * int64_t(sizeof(float));
}

loco_status loco_ckpt_encode(const void* x, int32_t x_dtype, int64_t ldx, int64_t rows, int64_t cols, int8_t* codes,
                             uint8_t* scales, loco_stream_t stream) {
  LOCO_TRY(check_dtype(x_dtype, "x_dtype"));
  LOCO_TRY(check_dim(rows, 0, "rows"));
  LOCO_TRY(check_dim(cols, 0, "cols"));
  if (rows == 0 || cols == 0) return done();
  Args g;
  g.add(x, rows, cols, ldx, elem_size(x_dtype), elem_size(x_dtype), "x");
  g.outputs();
  g.ckpt(codes, scales, rows, cols);
  LOCO_TRY(g.check());
  EncodeArgs a{x, ldx, rows, cols, x_dtype == LOCO_BF16, codes, scales};
  return launch_result(launch_ckpt_encode(a, reinterpret_cast<cudaStream_t>(stream)), "loco_ckpt_encode");
}

loco_status loco_ckpt_decode(const int8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, int32_t act,
                             const void* gamma, const void* beta, int32_t param_dtype, void* out, int32_t out_dtype,
                             int64_t ldo, loco_stream_t stream) {
  LOCO_TRY(check_act(act));
  LOCO_TRY(check_dtype(param_dtype, "param_dtype"));
  LOCO_TRY(check_dtype(out_dtype, "out_dtype"));
  LOCO_TRY(check_dim(rows, 0, "rows"));
  LOCO_TRY(check_dim(cols, 0, "cols"));
  if (rows == 0 || cols == 0) return done();
  Args g;
  g.ckpt(codes, scales, rows, cols);
  g.opt_vec(gamma, cols, elem_size(param_dtype), "gamma");
  g.opt_vec(beta, cols, elem_size(param_dtype), "beta");
  g.outputs();
  g.add(out, rows, cols, ldo, elem_size(out_dtype), elem_size(out_dtype), "out");
  LOCO_TRY(g.check());
  DecodeArgs a{codes, scales, rows, cols, ldo, act, gamma, beta, param_dtype == LOCO_BF16, out, out_dtype == LOCO_BF16};
  return launch_result(launch_ckpt_decode(a, reinterpret_cast<cudaStream_t>(stream)), "loco_ckpt_decode");
}

loco_status loco_norm_forward(const loco_norm_config* cfg, const void* x, int64_t ldx, int64_t rows, int64_t cols,
                              const void* gamma, const void* beta, void* y, int64_t ldy, float* mean, float* rstd,
                              int8_t* codes, uint8_t* scales, loco_stream_t stream) {
  LOCO_TRY(check_norm(cfg, rows, cols));
  LOCO_TRY(both_or_neither(codes, scales));
  if (rows == 0) return done();
  const size_t xe = elem_size(cfg->x_dtype), ye = elem_size(cfg->y_dtype), pe = elem_size(cfg->param_dtype);
  Args g;
  g.add(x, rows, cols, ldx, xe, xe, "x");
  g.opt_vec(gamma, cols, pe, "gamma");
  g.opt_vec(beta, cols, pe, "beta");
  g.outputs();
  g.add(y, rows, cols, ldy, ye, ye, "y");
  if (cfg->kind == LOCO_NORM_LAYER) g.opt_vec(mean, rows, 4, "mean");
  g.opt_vec(rstd, rows, 4, "rstd");
  if (codes != nullptr) g.ckpt(codes, scales, rows, cols);
  LOCO_TRY(g.check());
  NormFwdArgs a{x, gamma, beta, y, mean, rstd, codes, scales, ldx, ldy, rows, cols, cfg->eps,
                cfg->kind == LOCO_NORM_RMS, cfg->x_dtype == LOCO_BF16, cfg->y_dtype == LOCO_BF16,
                cfg->param_dtype == LOCO_BF16};
  return launch_result(launch_norm_forward(a, reinterpret_cast<cudaStream_t>(stream)), "loco_norm_forward");
}

loco_status loco_norm_backward(const loco_norm_config* cfg, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                               const int8_t* codes, const uint8_t* scales, const float* mean, const float* rstd,
                               int64_t rows, int64_t cols, const void* gamma, const void* residual, int64_t ldr,
                               void* dx, int64_t lddx, void* dgamma, void* dbeta, void* workspace, int64_t ws_bytes,
                               loco_stream_t stream) {
  LOCO_TRY(check_norm(cfg, rows, cols));
  const size_t xe = elem_size(cfg->x_dtype), ye = elem_size(cfg->y_dtype), pe = elem_size(cfg->param_dtype),
               ge = elem_size(cfg->grad_dtype);
  const bool params = dgamma != nullptr || dbeta != nullptr;
  const int64_t need = params && rows > 0 ? loco_norm_workspace_bytes(rows, cols) : 0;
  if (need > 0 && workspace == nullptr) return fail(LOCO_ERR_INVALID_ARG, "workspace is NULL");
  if (ws_bytes < need)
    return fail(LOCO_ERR_INVALID_ARG, "workspace holds %lld bytes, %lld are needed", (long long)ws_bytes,
                (long long)need);
  Args g;
  if (rows > 0) {
    if (x == nullptr) {
      if (codes == nullptr || scales == nullptr)
        return fail(LOCO_ERR_INVALID_ARG, "x is NULL and so is its checkpoint (codes, scales)");
      g.ckpt(codes, scales, rows, cols);
    } else {
      g.add(x, rows, cols, ldx, xe, xe, "x");
      if (cfg->kind == LOCO_NORM_LAYER) g.vec(mean, rows, 4, "mean");
    }
    g.add(dy, rows, cols, lddy, ye, ye, "dy");
    g.vec(rstd, rows, 4, "rstd");
    g.opt_vec(gamma, cols, pe, "gamma");
    if (residual != nullptr) {
      g.add(residual, rows, cols, ldr, xe, xe, "residual");
      g.in_place_in = &g.m[g.n - 1];
    }
  }
  g.outputs();
  if (rows > 0) g.add(dx, rows, cols, lddx, xe, xe, "dx");
  g.opt_vec(dgamma, cols, ge, "dgamma");
  g.opt_vec(dbeta, cols, ge, "dbeta");
  if (need > 0) g.add(workspace, 1, need, need, 1, 16, "workspace");
  LOCO_TRY(g.check());
  if (rows == 0 && !params) return done();
  NormBwdArgs a{};
  a.dy = dy, a.x = x, a.codes = codes, a.scales = scales, a.mean = mean, a.rstd = rstd, a.gamma = gamma;
  a.residual = residual, a.dx = dx, a.dgamma = dgamma, a.dbeta = dbeta;
  a.partials = params ? static_cast<float*>(workspace) : nullptr;
  a.lddy = lddy, a.ldx = ldx, a.ldr = ldr, a.lddx = lddx, a.rows = rows, a.cols = cols;
  a.rms = cfg->kind == LOCO_NORM_RMS, a.x_bf16 = cfg->x_dtype == LOCO_BF16, a.y_bf16 = cfg->y_dtype == LOCO_BF16;
  a.param_bf16 = cfg->param_dtype == LOCO_BF16, a.grad_bf16 = cfg->grad_dtype == LOCO_BF16;
  return launch_result(launch_norm_backward(a, reinterpret_cast<cudaStream_t>(stream)), "loco_norm_backward");
}

int32_t loco_matrices_overlap(const void* a, int64_t lda, int64_t rows_a, int64_t cols_a, int32_t bytes_a, const void* b,
                              int64_t ldb, int64_t rows_b, int64_t cols_b, int32_t bytes_b) {
  if (a == nullptr || b == nullptr || rows_a < 1 || cols_a < 1 || rows_b < 1 || cols_b < 1) return 0;
  const Mat x{a, rows_a, cols_a, rows_a == 1 ? cols_a : lda, size_t(bytes_a), 1, ""};
  const Mat y{b, rows_b, cols_b, rows_b == 1 ? cols_b : ldb, size_t(bytes_b), 1, ""};
  for (const Mat* m : {&x, &y}) {
    // what no entry point takes: not known to lie apart
    if (m->elem < 1 || m->elem > 16 || m->cols > LOCO_MAX_N || m->ld < m->cols) return 1;
    if (m->rows > 1 && (m->rows > kMaxDim || m->ld > kMaxDim)) return 1;
  }
  return mats_overlap(x, y);
}

loco_status loco_linear_align(const void* src, int64_t lds, int64_t rows, int64_t cols, void* dst, int64_t ldd,
                              loco_stream_t stream) {
  LOCO_TRY(check_dim(rows, 0, "rows"));
  LOCO_TRY(check_dim(cols, 0, "cols"));
  if (rows == 0 || cols == 0) return done();
  if (ldd < cols || ldd % 8 != 0 || ldd > kMaxDim)
    return fail(LOCO_ERR_INVALID_ARG, "ldd = %lld must be a multiple of 8 in [cols, LOCO_MAX_DIM]", (long long)ldd);
  Args g;
  g.add(src, rows, cols, lds, 2, 2, "src");
  g.outputs();
  g.add(dst, rows, (cols + 7) / 8 * 8, ldd, 2, 16, "dst");
  LOCO_TRY(g.check());
  return launch_result(launch_align(AlignArgs{src, lds, rows, cols, dst, ldd}, reinterpret_cast<cudaStream_t>(stream)),
                       "loco_linear_align");
}

loco_status loco_linear_forward(const loco_linear_config* cfg, const void* x, int64_t ldx, const void* w, int64_t ldw,
                                const void* bias, const void* residual, int64_t ldr, int64_t T, int64_t N, int64_t K,
                                void* y, int64_t ldy, int8_t* codes, uint8_t* scales, loco_stream_t stream) {
  LOCO_TRY(check_linear(cfg, T, N, K));
  LOCO_TRY(check_act(cfg->act));
  LOCO_TRY(both_or_neither(codes, scales));
  if (T == 0 || N == 0) return done();
  const size_t oe = elem_size(cfg->out_dtype);
  Args g;
  if (K > 0) {
    g.add(x, T, K, ldx, 2, 2, "x");
    g.add(w, N, K, ldw, 2, 2, "w");
  }
  g.opt_vec(bias, N, elem_size(cfg->param_dtype), "bias");
  if (residual != nullptr) {
    g.add(residual, T, N, ldr, oe, oe, "residual");
    g.in_place_in = &g.m[g.n - 1];
  }
  g.outputs();
  g.add(y, T, N, ldy, oe, oe, "y");
  if (codes != nullptr) g.ckpt(codes, scales, T, N);
  LOCO_TRY(g.check());
  LinearArgs a{};
  a.a = w, a.lda = ldw, a.b = x, a.ldb = ldx;
  a.M = N, a.N = T, a.K = K;
  a.bias = bias, a.param_bf16 = cfg->param_dtype == LOCO_BF16;
  a.save_codes = codes, a.save_scales = scales;
  a.act = cfg->act;
  a.residual = residual, a.ldr = ldr;
  a.out = y, a.ldo = ldy, a.out_bf16 = cfg->out_dtype == LOCO_BF16;
  return launch_result(launch_linear(a, reinterpret_cast<cudaStream_t>(stream)), "loco_linear_forward");
}

loco_status loco_linear_backward_input(const loco_linear_config* cfg, const void* dy, int64_t lddy, const void* w,
                                       int64_t ldw, const int8_t* codes, const uint8_t* scales, const void* residual,
                                       int64_t ldr, int64_t T, int64_t N, int64_t K, void* dx, int64_t lddx,
                                       loco_stream_t stream) {
  LOCO_TRY(check_linear(cfg, T, N, K));
  LOCO_TRY(check_act(cfg->act));
  if (T == 0 || K == 0) return done();
  const bool slope = cfg->act != LOCO_ACT_NONE;
  const size_t oe = elem_size(cfg->out_dtype);
  Args g;
  if (N > 0) {
    g.add(dy, T, N, lddy, 2, 2, "dy");
    g.add(w, N, K, ldw, 2, 2, "w");
  }
  if (slope) g.ckpt(codes, scales, T, K);
  if (residual != nullptr) {
    g.add(residual, T, K, ldr, oe, oe, "residual");
    g.in_place_in = &g.m[g.n - 1];
  }
  g.outputs();
  g.add(dx, T, K, lddx, oe, oe, "dx");
  LOCO_TRY(g.check());
  LinearArgs a{};
  a.a = w, a.lda = ldw, a.a_mn = 1, a.b = dy, a.ldb = lddy;
  a.M = K, a.N = T, a.K = N;
  a.act = cfg->act;
  a.z_codes = slope ? codes : nullptr, a.z_scales = slope ? scales : nullptr;
  a.residual = residual, a.ldr = ldr;
  a.out = dx, a.ldo = lddx, a.out_bf16 = cfg->out_dtype == LOCO_BF16;
  return launch_result(launch_linear(a, reinterpret_cast<cudaStream_t>(stream)), "loco_linear_backward_input");
}

loco_status loco_linear_backward_weight(const loco_linear_config* cfg, const void* dy, int64_t lddy, const void* x,
                                        int64_t ldx, const int8_t* codes, const uint8_t* scales, const void* gamma,
                                        const void* beta, int64_t T, int64_t N, int64_t K, void* dw, int64_t lddw,
                                        void* db, void* workspace, int64_t ws_bytes, loco_stream_t stream) {
  LOCO_TRY(check_linear(cfg, T, N, K));
  if (N == 0 || (K == 0 && db == nullptr)) return done();
  const size_t oe = elem_size(cfg->out_dtype), pe = elem_size(cfg->param_dtype);
  const bool from_ckpt = x == nullptr && T > 0;  // (an empty x may be NULL; without rows nothing but zeros is written)
  const bool shift = from_ckpt && beta != nullptr && K > 0;
  const int64_t need = shift ? loco_linear_workspace_bytes(N) : 0;
  if (need > 0 && workspace == nullptr) return fail(LOCO_ERR_INVALID_ARG, "workspace is NULL");
  if (ws_bytes < need)
    return fail(LOCO_ERR_INVALID_ARG, "workspace holds %lld bytes, %lld are needed", (long long)ws_bytes,
                (long long)need);
  Args g;
  if (T > 0) {
    g.add(dy, T, N, lddy, 2, 2, "dy");
    if (K > 0) {
      if (!from_ckpt) {
        g.add(x, T, K, ldx, 2, 2, "x");
      } else {
        if (codes == nullptr || scales == nullptr)
          return fail(LOCO_ERR_INVALID_ARG, "x is NULL and so is its checkpoint (codes, scales)");
        g.ckpt(codes, scales, T, K);
      }
    }
  }
  if (from_ckpt && K > 0) {
    g.opt_vec(gamma, K, pe, "gamma");
    g.opt_vec(beta, K, pe, "beta");
  }
  g.outputs();
  if (K > 0) g.add(dw, N, K, lddw, oe, oe, "dw");
  g.opt_vec(db, N, oe, "db");
  if (need > 0) g.add(workspace, 1, need, need, 1, 16, "workspace");
  LOCO_TRY(g.check());
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int out_bf16 = cfg->out_dtype == LOCO_BF16;
  if (db != nullptr || shift) {
    ColSumArgs c{dy, lddy, T, N, shift ? static_cast<float*>(workspace) : nullptr, db, out_bf16};
    const cudaError_t e = launch_col_sum(c, s);
    if (e != cudaSuccess) return launch_result(e, "loco_linear_backward_weight");
  }
  if (K == 0) return done();
  LinearArgs a{};
  a.a = x, a.lda = ldx, a.a_mn = 1, a.b = dy, a.ldb = lddy, a.b_mn = 1;
  if (from_ckpt) a.a_codes = codes, a.a_scales = scales;
  a.M = K, a.N = N, a.K = T;
  a.param_bf16 = cfg->param_dtype == LOCO_BF16;
  if (from_ckpt) a.col_scale = gamma;
  if (shift) a.col_shift = beta, a.row_sum = static_cast<const float*>(workspace);
  a.act = LOCO_ACT_NONE;
  a.out = dw, a.ldo = lddw, a.out_bf16 = out_bf16;
  return launch_result(launch_linear(a, s), "loco_linear_backward_weight");
}

loco_status loco_linear_timeouts(int64_t* count) {
  if (count == nullptr) return fail(LOCO_ERR_INVALID_ARG, "count is NULL");
  int64_t linear = 0, forward = 0, backward = 0;
  cudaError_t e = read_linear_timeouts(&linear);
  if (e == cudaSuccess) e = read_join_forward_timeouts(&forward);
  if (e == cudaSuccess) e = read_join_backward_timeouts(&backward);
  if (e == cudaSuccess) *count = linear + forward + backward;
  return launch_result(e, "loco_linear_timeouts");
}

}  // extern "C"
