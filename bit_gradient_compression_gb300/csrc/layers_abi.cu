// Entry points of the layers (declared in include/loco.h): argument checks and
// dispatch.  As in abi.cu, everything is checked on the host before anything is
// launched, so a refused call writes nothing.
#include <math.h>

#include "abi_checks.h"
#include "layers_internal.h"
#include "loco.h"

namespace loco {

namespace {

constexpr int64_t kMaxDim = LOCO_MAX_DIM;

size_t elem_size(int32_t dtype) { return dtype == LOCO_BF16 ? 2 : 4; }

// A matrix argument: element (i, j) at p + (i*ld + j) * elem bytes.
struct Mat {
  const void* p;
  int64_t rows, cols, ld;
  size_t elem, align;
  const char* name;
  size_t bytes() const { return (size_t(rows - 1) * size_t(ld) + size_t(cols)) * elem; }
};

// Whether two matrices share an element's bytes.  Two of the same pitch that lie beside one
// another in a wider matrix (columns 0..a and b..c of its rows) do not.
bool mats_overlap(const Mat& x, const Mat& y) {
  if (!overlap(x.p, x.bytes(), y.p, y.bytes())) return false;
  const uint64_t pitch = uint64_t(x.ld) * x.elem;
  if (x.rows <= 1 || y.rows <= 1 || pitch != uint64_t(y.ld) * y.elem) {
    // a single row against a pitched matrix: compare with that matrix's rows
    const Mat& one = x.rows <= 1 ? x : y;
    const Mat& many = x.rows <= 1 ? y : x;
    if (one.rows > 1) return true;
    const uint64_t mp = uint64_t(many.ld) * many.elem, mw = uint64_t(many.cols) * many.elem;
    const uintptr_t o = reinterpret_cast<uintptr_t>(one.p), m = reinterpret_cast<uintptr_t>(many.p);
    if (o < m || many.rows <= 1) return true;
    const uint64_t at = (o - m) % mp;
    return at < mw || at + uint64_t(one.cols) * one.elem > mp;
  }
  const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
  const uint64_t wx = uint64_t(x.cols) * x.elem, wy = uint64_t(y.cols) * y.elem;
  const uint64_t at = a <= b ? (b - a) % pitch : (pitch - (a - b) % pitch) % pitch;  // y's column offset in x's rows
  return at < wx || at + wy > pitch;
}

constexpr int kMaxMats = 16;

struct Args {
  Mat m[kMaxMats];
  int n = 0;
  int first_out = -1;  // arguments from here on are written
  const Mat* in_place_in = nullptr;

  void add(const void* p, int64_t rows, int64_t cols, int64_t ld, size_t elem, size_t align, const char* name) {
    m[n++] = Mat{p, rows, cols, ld, elem, align, name};
  }
  void vec(const void* p, int64_t count, size_t elem, const char* name) { add(p, 1, count, count, elem, elem, name); }
  void opt_vec(const void* p, int64_t count, size_t elem, const char* name) {
    if (p != nullptr) vec(p, count, elem, name);
  }
  void ckpt(const void* codes, const void* scales, int64_t rows, int64_t cols) {
    add(codes, 1, loco_ckpt_code_bytes(rows, cols), loco_ckpt_code_bytes(rows, cols), 1, 16, "codes");
    add(scales, 1, loco_ckpt_scale_bytes(rows, cols), loco_ckpt_scale_bytes(rows, cols), 1, 1, "scales");
  }
  void outputs() { first_out = n; }

  loco_status check() const {
    BufCheck b[kMaxMats];
    for (int i = 0; i < n; ++i) {
      // vectors and checkpoints come here as one row, whose length was bounded by their sizes
      if (m[i].ld < m[i].cols || (m[i].rows > 1 && m[i].ld > kMaxDim))
        return fail(LOCO_ERR_INVALID_ARG, "%s: row pitch %lld outside [%lld, LOCO_MAX_DIM]", m[i].name,
                    (long long)m[i].ld, (long long)m[i].cols);
      if (m[i].bytes() > size_t(LOCO_MAX_N))
        return fail(LOCO_ERR_INVALID_ARG, "%s: %zu bytes are more than any device holds", m[i].name, m[i].bytes());
      b[i] = BufCheck{m[i].p, m[i].bytes(), m[i].align, m[i].name};
    }
    const loco_status st = check_buffers(b, n);
    if (st != LOCO_OK) return st;
    for (int i = first_out; i < n; ++i)
      for (int j = 0; j < n; ++j) {
        if (j == i || !mats_overlap(m[i], m[j])) continue;
        // the residual may be the output itself
        const bool same = m[i].p == m[j].p && m[i].ld == m[j].ld && m[i].elem == m[j].elem && m[i].rows == m[j].rows &&
                          m[i].cols == m[j].cols;
        if (same && j < first_out && &m[j] == in_place_in) continue;
        return fail(LOCO_ERR_INVALID_ARG, "%s overlaps %s", m[i].name, m[j].name);
      }
    return LOCO_OK;
  }
};

loco_status check_dtype(int32_t d, const char* name) {
  if (d != LOCO_F32 && d != LOCO_BF16)
    return fail(LOCO_ERR_UNSUPPORTED, "%s = %d (LOCO_F32 or LOCO_BF16)", name, d);
  return LOCO_OK;
}

loco_status check_dim(int64_t v, int64_t least, const char* name) {
  if (v < least || v > kMaxDim)
    return fail(LOCO_ERR_INVALID_ARG, "%s = %lld outside [%lld, LOCO_MAX_DIM]", name, (long long)v, (long long)least);
  return LOCO_OK;
}

loco_status check_act(int32_t act) {
  if (act < LOCO_ACT_NONE || act > LOCO_ACT_SILU) return fail(LOCO_ERR_UNSUPPORTED, "act = %d", act);
  return LOCO_OK;
}

loco_status both_or_neither(const void* codes, const void* scales) {
  if ((codes == nullptr) != (scales == nullptr))
    return fail(LOCO_ERR_INVALID_ARG, "codes and scales go together: one of them is NULL");
  return LOCO_OK;
}

loco_status done() {
  return launch_result(cudaSuccess, "");
}

#define LOCO_TRY(call)                         \
  do {                                         \
    const loco_status st_ = (call);            \
    if (st_ != LOCO_OK) return st_;            \
  } while (0)

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
  return launch_result(read_linear_timeouts(count), "loco_linear_timeouts");
}

}  // extern "C"
