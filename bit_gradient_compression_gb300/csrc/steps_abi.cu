// Entry points of joins, log probabilities and many-tensor optimizer steps (declared in include/loco.h):
// argument checks and dispatch.  As elsewhere everything is checked on the host before anything is
// launched, so a refused call writes nothing.
#include <math.h>
#include <stdio.h>

#include <algorithm>
#include <new>

#include "layers_args.h"
#include "steps_internal.h"

namespace loco {

namespace {

loco_status check_join(const loco_join_config* cfg, int64_t rows, int64_t cols) {
  if (cfg == nullptr) return fail(LOCO_ERR_INVALID_ARG, "cfg is NULL");
  if (cfg->kind != LOCO_NORM_LAYER && cfg->kind != LOCO_NORM_RMS)
    return fail(LOCO_ERR_UNSUPPORTED, "kind = %d (LOCO_NORM_LAYER or LOCO_NORM_RMS)", cfg->kind);
  if (cfg->post != 0 && cfg->post != 1) return fail(LOCO_ERR_UNSUPPORTED, "post = %d (0 or 1)", cfg->post);
  if (!(cfg->eps >= 0.0f) || !isfinite(cfg->eps))
    return fail(LOCO_ERR_INVALID_ARG, "eps = %g must be finite and >= 0", cfg->eps);
  if (!isfinite(cfg->residual_scale) || !isfinite(cfg->block_scale))
    return fail(LOCO_ERR_INVALID_ARG, "residual_scale = %g and block_scale = %g must be finite", cfg->residual_scale,
                cfg->block_scale);
  LOCO_TRY(check_dtype(cfg->x_dtype, "x_dtype"));
  LOCO_TRY(check_dtype(cfg->y_dtype, "y_dtype"));
  LOCO_TRY(check_dtype(cfg->param_dtype, "param_dtype"));
  LOCO_TRY(check_dtype(cfg->grad_dtype, "grad_dtype"));
  LOCO_TRY(check_dim(rows, 0, "rows"));
  return check_dim(cols, 1, "cols");
}

loco_status check_logits(int32_t dtype, int64_t rows, int64_t vocab, float scale) {
  LOCO_TRY(check_dtype(dtype, "dtype"));
  LOCO_TRY(check_dim(rows, 0, "rows"));
  LOCO_TRY(check_dim(vocab, 1, "vocab"));
  constexpr float kLog2E = 1.4426950408889634f;  // (the kernels' exponents are to base 2)
  if (!(scale > 0.0f) || !isfinite(scale * kLog2E))
    return fail(LOCO_ERR_INVALID_ARG, "scale = %g must be > 0 and scale * log2(e) finite", scale);
  return LOCO_OK;
}

// ------------------------------------------------------------------ many tensors

constexpr int kBuffers = 7;  // of one tensor
const char* const kBufferNames[kBuffers] = {"param", "grad", "m", "v", "m_steps", "v_steps", "param_bf16"};

// One buffer of a tensor: [lo, hi), written or only read.
struct Range {
  uintptr_t lo, hi;
  int tensor;
  int8_t buffer;
  bool out;
};

// Buffers of the call on the host: those of a few tensors on the stack, more from the heap.
struct Ranges {
  Range few[kAdamFew * kBuffers + 1];
  Range* r = few;
  int64_t n = 0;
  ~Ranges() {
    if (r != few) delete[] r;
  }
};

loco_status fail_tensor(loco_status st, int i, const char* buffer, const char* what) {
  return fail(st, "tensors[%d].%s %s", i, buffer, what);
}

constexpr int kNameSize = 40;
const char* buffer_name(const Range& r, char (&name)[kNameSize]) {
  if (r.tensor < 0)
    snprintf(name, kNameSize, "grad_scale");
  else
    snprintf(name, kNameSize, "tensors[%d].%s", r.tensor, kBufferNames[int(r.buffer)]);
  return name;
}

// Every buffer of every tensor, one kind after another (tensors of a kind mostly share their allocations):
// null, alignment and extent, then whether anything that is written overlaps anything else.
loco_status check_tensors(const loco_adam_tensors_config& cfg, const loco_adam_tensor* t, int32_t count,
                          const float* grad_scale, Ranges* all) {
  if (count > kAdamFew) {
    all->r = new (std::nothrow) Range[size_t(count) * kBuffers + 1];
    if (all->r == nullptr) {
      all->r = all->few;
      return fail(LOCO_ERR_INVALID_ARG, "no host memory for the buffers of %d tensors", count);
    }
  }
  const bool eight = cfg.state_bits == 8;
  const int64_t pe = int64_t(elem_size(cfg.param_dtype)), ge = int64_t(elem_size(cfg.grad_dtype));
  for (int b = 0; b < kBuffers; ++b) {
    for (int i = 0; i < count; ++i) {
      const loco_adam_tensor& x = t[i];
      if (x.n == 0) continue;
      const int64_t nb = (x.n + LOCO_STATE_BLOCK - 1) / LOCO_STATE_BLOCK;
      const void* p = nullptr;
      int64_t bytes = 0;
      size_t align = 4;
      switch (b) {
        case 0: p = x.param, bytes = x.n * pe, align = size_t(pe); break;
        case 1: p = x.grad, bytes = x.n * ge, align = size_t(ge); break;
        case 2: p = x.m, bytes = eight ? nb * LOCO_STATE_BLOCK : x.n * 4, align = eight ? 16 : 4; break;
        case 3: p = x.v, bytes = eight ? nb * LOCO_STATE_BLOCK : x.n * 4, align = eight ? 16 : 4; break;
        case 4: p = x.m_steps, bytes = eight ? nb * 4 : 0; break;
        case 5: p = x.v_steps, bytes = eight ? nb * 4 : 0; break;
        default: p = x.param_bf16, bytes = p != nullptr ? x.n * 2 : 0, align = 2; break;
      }
      if (bytes == 0) continue;
      if (p == nullptr) return fail_tensor(LOCO_ERR_INVALID_ARG, i, kBufferNames[b], "is NULL");
      if (reinterpret_cast<uintptr_t>(p) % align != 0) {
        return fail(LOCO_ERR_MISALIGNED, "tensors[%d].%s (%p) is not %zu-byte aligned", i, kBufferNames[b], p, align);
      }
      const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
      all->r[all->n++] = Range{lo, lo + uintptr_t(bytes), i, int8_t(b), b != 1};
    }
  }
  if (grad_scale != nullptr) {
    if (reinterpret_cast<uintptr_t>(grad_scale) % 4 != 0)
      return fail(LOCO_ERR_MISALIGNED, "grad_scale (%p) is not 4-byte aligned", static_cast<const void*>(grad_scale));
    const uintptr_t lo = reinterpret_cast<uintptr_t>(grad_scale);
    all->r[all->n++] = Range{lo, lo + 4, -1, 1, false};
  }
  // extents, a few at a time in the order above; the index of one that fails is put to its name afterwards
  constexpr int kAtOnce = 64;
  for (int64_t at = 0; at < all->n; at += kAtOnce) {
    BufCheck c[kAtOnce];
    const int n = int(std::min<int64_t>(kAtOnce, all->n - at));
    for (int k = 0; k < n; ++k) {
      const Range& r = all->r[at + k];
      c[k] = BufCheck{reinterpret_cast<const void*>(r.lo), size_t(r.hi - r.lo), 1, kBufferNames[int(r.buffer)]};
    }
    if (check_buffers(c, n) == LOCO_OK) continue;
    for (int k = 0; k < n; ++k) {
      char name[kNameSize];
      c[k].name = buffer_name(all->r[at + k], name);
      LOCO_TRY(check_buffers(c + k, 1));
    }
  }
  // by their beginnings: what is written must begin after all before it end, what is read after all written before it
  std::sort(all->r, all->r + all->n, [](const Range& a, const Range& b) { return a.lo < b.lo; });
  const Range *last = nullptr, *last_out = nullptr;  // the ones that end last
  for (int64_t i = 0; i < all->n; ++i) {
    const Range& r = all->r[i];
    const Range* other = r.out ? last : last_out;
    if (other != nullptr && r.lo < other->hi) {
      char a[kNameSize], b[kNameSize];
      return fail(LOCO_ERR_INVALID_ARG, "%s overlaps %s", buffer_name(*other, a), buffer_name(r, b));
    }
    if (last == nullptr || r.hi > last->hi) last = &r;
    if (r.out && (last_out == nullptr || r.hi > last_out->hi)) last_out = &r;
  }
  return LOCO_OK;
}

bool on(const void* p, size_t align) { return reinterpret_cast<uintptr_t>(p) % align == 0; }

// Launches tensors [at, at + n) of the call.
template <int MAX>
loco_status launch_some(const loco_adam_tensors_config& cfg, const loco_adam_tensor* tensors, int at, int n,
                        const loco_adam_hparams& hp, int64_t t, const AdamTensorsArgs& args, cudaStream_t s) {
  AdamTensorList<MAX> l;
  l.a = args;
  l.count = 0;
  uint64_t units = 0;
  const double bc1 = hp.bias_correction ? 1.0 - pow(double(hp.beta1), double(t)) : 1.0;
  const uint32_t key = mix32(mix32(cfg.dither) ^ uint32_t(uint64_t(t)));
  const bool eight = cfg.state_bits == 8, pb = cfg.param_dtype == LOCO_BF16, gb = cfg.grad_dtype == LOCO_BF16;
  for (int i = at; i < at + n; ++i) {
    const loco_adam_tensor& x = tensors[i];
    if (x.n == 0) continue;
    const float lr = hp.lr * x.lr_scale, wd = hp.weight_decay * x.decay_scale;
    AdamTensor& o = l.t[l.count];
    o.p = x.param, o.g = x.grad, o.m = x.m, o.v = x.v, o.m_steps = x.m_steps, o.v_steps = x.v_steps, o.copy = x.param_bf16;
    o.n = x.n;
    o.c1 = hp.bias_correction ? float(double(lr) / bc1) : lr;
    o.lr_wd = lr * wd;
    o.key = mix32(key ^ uint32_t(i));
    o.wide = on(x.param, pb ? 8 : 16) && on(x.grad, gb ? 8 : 16) && (eight || (on(x.m, 16) && on(x.v, 16))) &&
             on(x.param_bf16, 8);
    l.first[l.count++] = uint32_t(units);
    units += uint64_t((x.n + LOCO_STATE_BLOCK - 1) / LOCO_STATE_BLOCK);
    if (units > 0x7FFFFFFFu)
      return fail(LOCO_ERR_UNSUPPORTED, "tensors %d to %d have more than 2^39 elements", at, i);
  }
  if (l.count == 0) return done();
  l.first[l.count] = uint32_t(units);
  const AdamTensorsKind kind{cfg.state_bits, pb, gb, cfg.dither != 0};
  return launch_result(launch_adam_tensors<MAX>(l, kind, s), "loco_adam_tensors");
}

}  // namespace

}  // namespace loco

using namespace loco;

extern "C" {

loco_status loco_join_forward(const loco_join_config* cfg, const void* x, int64_t ldx, const void* y, int64_t ldy,
                              int64_t rows, int64_t cols, const void* post_gamma, const void* post_beta,
                              const void* gate, const float* row_gate, const void* gamma, const void* beta, void* h,
                              int64_t ldh, void* u, int64_t ldu, float* stats, loco_stream_t stream) {
  LOCO_TRY(check_join(cfg, rows, cols));
  if (rows == 0) return done();
  const size_t xe = elem_size(cfg->x_dtype), ye = elem_size(cfg->y_dtype), pe = elem_size(cfg->param_dtype);
  Args g;
  g.add(x, rows, cols, ldx, xe, xe, "x");
  g.in_place_in = &g.m[g.n - 1];
  g.add(y, rows, cols, ldy, ye, ye, "y");
  g.opt_vec(post_gamma, cols, pe, "post_gamma");
  g.opt_vec(post_beta, cols, pe, "post_beta");
  g.opt_vec(gate, cols, pe, "gate");
  g.opt_vec(row_gate, rows, 4, "row_gate");
  if (u != nullptr) {
    g.opt_vec(gamma, cols, pe, "gamma");
    g.opt_vec(beta, cols, pe, "beta");
  }
  g.outputs();
  g.add(h, rows, cols, ldh, xe, xe, "h");
  if (u != nullptr) g.add(u, rows, cols, ldu, ye, ye, "u");
  if (stats != nullptr) g.add(stats, 1, 4 * rows, 4 * rows, 4, 4, "stats");
  LOCO_TRY(g.check());
  JoinFwdArgs a{};
  a.x = x, a.y = y, a.post_gamma = post_gamma, a.post_beta = post_beta, a.gate = gate, a.row_gate = row_gate;
  if (u != nullptr) a.gamma = gamma, a.beta = beta;
  a.h = h, a.u = u, a.stats = stats;
  a.ldx = ldx, a.ldy = ldy, a.ldh = ldh, a.ldu = ldu, a.rows = rows, a.cols = cols;
  a.eps = cfg->eps, a.a = cfg->residual_scale, a.s = cfg->block_scale;
  a.rms = cfg->kind == LOCO_NORM_RMS, a.post = cfg->post, a.x_bf16 = cfg->x_dtype == LOCO_BF16;
  a.y_bf16 = cfg->y_dtype == LOCO_BF16, a.param_bf16 = cfg->param_dtype == LOCO_BF16;
  return launch_result(launch_join_forward(a, reinterpret_cast<cudaStream_t>(stream)), "loco_join_forward");
}

int64_t loco_join_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || rows > kMaxDim || cols < 1 || cols > kMaxDim) return 0;
  const int64_t parts = rows < kJoinPartials ? (rows < 1 ? 1 : rows) : kJoinPartials;
  return parts * kJoinSums * cols * int64_t(sizeof(float));
}

loco_status loco_join_backward(const loco_join_config* cfg, const void* dh, int64_t lddh, const void* du, int64_t lddu,
                               const void* h, int64_t ldh, const void* y, int64_t ldy, const float* stats, int64_t rows,
                               int64_t cols, const void* post_gamma, const void* post_beta, const void* gate,
                               const float* row_gate, const void* gamma, void* dx, int64_t lddx, void* dy, int64_t lddy,
                               void* dpost_gamma, void* dpost_beta, void* dgate, float* drow_gate, void* dgamma,
                               void* dbeta, void* workspace, int64_t ws_bytes, loco_stream_t stream) {
  LOCO_TRY(check_join(cfg, rows, cols));
  const size_t xe = elem_size(cfg->x_dtype), ye = elem_size(cfg->y_dtype), pe = elem_size(cfg->param_dtype),
               ge = elem_size(cfg->grad_dtype);
  const bool params = dpost_gamma != nullptr || dpost_beta != nullptr || dgate != nullptr || dgamma != nullptr ||
                      dbeta != nullptr;
  const int64_t need = params && rows > 0 ? loco_join_workspace_bytes(rows, cols) : 0;
  if (need > 0 && workspace == nullptr) return fail(LOCO_ERR_INVALID_ARG, "workspace is NULL");
  if (ws_bytes < need)
    return fail(LOCO_ERR_INVALID_ARG, "workspace holds %lld bytes, %lld are needed", (long long)ws_bytes,
                (long long)need);
  const bool need_y = cfg->post || dgate != nullptr || drow_gate != nullptr || dpost_gamma != nullptr;
  Args g;
  if (rows > 0) {
    if (dh != nullptr) {
      g.add(dh, rows, cols, lddh, xe, xe, "dh");
      g.in_place_in = &g.m[g.n - 1];
    }
    if (du != nullptr) {
      g.add(du, rows, cols, lddu, ye, ye, "du");
      g.add(h, rows, cols, ldh, xe, xe, "h");
      g.opt_vec(gamma, cols, pe, "gamma");
    }
    if (need_y) g.add(y, rows, cols, ldy, ye, ye, "y");
    if (cfg->post || du != nullptr) g.add(stats, 1, 4 * rows, 4 * rows, 4, 4, "stats");
    g.opt_vec(post_gamma, cols, pe, "post_gamma");
    if (dgate != nullptr || drow_gate != nullptr) g.opt_vec(post_beta, cols, pe, "post_beta");
    g.opt_vec(gate, cols, pe, "gate");
    g.opt_vec(row_gate, rows, 4, "row_gate");
  }
  g.outputs();
  if (rows > 0) {
    g.add(dx, rows, cols, lddx, xe, xe, "dx");
    g.add(dy, rows, cols, lddy, ye, ye, "dy");
    g.opt_vec(drow_gate, rows, 4, "drow_gate");
  }
  g.opt_vec(dpost_gamma, cols, ge, "dpost_gamma");
  g.opt_vec(dpost_beta, cols, ge, "dpost_beta");
  g.opt_vec(dgate, cols, ge, "dgate");
  g.opt_vec(dgamma, cols, ge, "dgamma");
  g.opt_vec(dbeta, cols, ge, "dbeta");
  if (need > 0) g.add(workspace, 1, need, need, 1, 16, "workspace");
  LOCO_TRY(g.check());
  if (rows == 0 && !params) return done();
  JoinBwdArgs a{};
  a.dh = dh, a.du = du, a.h = du != nullptr ? h : nullptr, a.y = need_y ? y : nullptr, a.stats = stats;
  a.post_gamma = rows > 0 ? post_gamma : nullptr, a.gate = rows > 0 ? gate : nullptr, a.row_gate = row_gate;
  a.post_beta = rows > 0 && (dgate != nullptr || drow_gate != nullptr) ? post_beta : nullptr;
  a.gamma = du != nullptr ? gamma : nullptr;
  a.dx = dx, a.dy = dy, a.dpost_gamma = dpost_gamma, a.dpost_beta = dpost_beta, a.dgate = dgate;
  a.drow_gate = drow_gate, a.dgamma = dgamma, a.dbeta = dbeta;
  a.partials = params ? static_cast<float*>(workspace) : nullptr;
  a.lddh = lddh, a.lddu = lddu, a.ldh = ldh, a.ldy = ldy, a.lddx = lddx, a.lddy = lddy, a.rows = rows, a.cols = cols;
  a.a = cfg->residual_scale, a.s = cfg->block_scale;
  a.rms = cfg->kind == LOCO_NORM_RMS, a.post = cfg->post, a.x_bf16 = cfg->x_dtype == LOCO_BF16;
  a.y_bf16 = cfg->y_dtype == LOCO_BF16, a.param_bf16 = cfg->param_dtype == LOCO_BF16;
  a.grad_bf16 = cfg->grad_dtype == LOCO_BF16;
  return launch_result(launch_join_backward(a, reinterpret_cast<cudaStream_t>(stream)), "loco_join_backward");
}

loco_status loco_logprob_forward(const void* logits, int32_t dtype, int64_t ld, int64_t rows, int64_t vocab, float scale,
                                 const int64_t* targets, float* logp, float* lse, float* entropy, int32_t top,
                                 int64_t* top_ids, float* top_logp, loco_stream_t stream) {
  LOCO_TRY(check_logits(dtype, rows, vocab, scale));
  if (top < 0 || top > LOCO_MAX_TOP)
    return fail(LOCO_ERR_INVALID_ARG, "top = %d outside [0, LOCO_MAX_TOP = %d]", top, LOCO_MAX_TOP);
  if (rows == 0) return done();
  const size_t e = elem_size(dtype);
  Args g;
  g.add(logits, rows, vocab, ld, e, e, "logits");
  if (logp != nullptr) g.vec(targets, rows, 8, "targets");
  g.outputs();
  g.opt_vec(logp, rows, 4, "logp");
  g.opt_vec(lse, rows, 4, "lse");
  g.opt_vec(entropy, rows, 4, "entropy");
  if (top > 0) {
    g.opt_vec(top_ids, rows * top, 8, "top_ids");
    g.opt_vec(top_logp, rows * top, 4, "top_logp");
  }
  LOCO_TRY(g.check());
  const bool list = top > 0 && (top_ids != nullptr || top_logp != nullptr);
  if (logp == nullptr && lse == nullptr && entropy == nullptr && !list) return done();
  const LogprobFwdArgs a{logits, ld, rows, vocab, scale, targets, logp, lse, entropy, top_ids, top_logp, list ? top : 0,
                         dtype == LOCO_BF16};
  return launch_result(launch_logprob_forward(a, reinterpret_cast<cudaStream_t>(stream)), "loco_logprob_forward");
}

loco_status loco_logprob_backward(const void* logits, int32_t dtype, int64_t ld, int64_t rows, int64_t vocab, float scale,
                                  const int64_t* targets, const float* lse, const float* entropy, const float* dlogp,
                                  const float* dentropy, void* dlogits, int64_t ldd, loco_stream_t stream) {
  LOCO_TRY(check_logits(dtype, rows, vocab, scale));
  if (rows == 0) return done();
  const size_t e = elem_size(dtype);
  Args g;
  g.add(logits, rows, vocab, ld, e, e, "logits");
  g.in_place_in = &g.m[0];
  g.vec(lse, rows, 4, "lse");
  if (dlogp != nullptr) {
    g.vec(dlogp, rows, 4, "dlogp");
    g.vec(targets, rows, 8, "targets");
  }
  if (dentropy != nullptr) {
    g.vec(dentropy, rows, 4, "dentropy");
    g.vec(entropy, rows, 4, "entropy");
  }
  g.outputs();
  g.add(dlogits, rows, vocab, ldd, e, e, "dlogits");
  LOCO_TRY(g.check());
  const LogprobBwdArgs a{logits, ld, rows, vocab, scale, targets, lse, entropy, dlogp, dentropy, dlogits, ldd,
                         dtype == LOCO_BF16};
  return launch_result(launch_logprob_backward(a, reinterpret_cast<cudaStream_t>(stream)), "loco_logprob_backward");
}

loco_status loco_adam_tensors(const loco_adam_tensors_config* cfg, const loco_adam_tensor* tensors, int32_t count,
                              const loco_adam_hparams* hp, int64_t t, const float* grad_scale, loco_stream_t stream) {
  if (cfg == nullptr) return fail(LOCO_ERR_INVALID_ARG, "cfg is NULL");
  if (hp == nullptr) return fail(LOCO_ERR_INVALID_ARG, "hp is NULL");
  if (cfg->state_bits != 32 && cfg->state_bits != 8)
    return fail(LOCO_ERR_UNSUPPORTED, "state_bits = %d (8 or 32)", cfg->state_bits);
  LOCO_TRY(check_dtype(cfg->param_dtype, "param_dtype"));
  LOCO_TRY(check_dtype(cfg->grad_dtype, "grad_dtype"));
  if (t < 1) return fail(LOCO_ERR_INVALID_ARG, "t = %lld (1-based)", (long long)t);
  if (!isfinite(hp->lr) || !isfinite(hp->eps) || !isfinite(hp->weight_decay) || hp->eps < 0.0f)
    return fail(LOCO_ERR_INVALID_ARG, "lr, eps, weight_decay must be finite and eps >= 0");
  if (!(hp->beta1 >= 0.0f && hp->beta1 < 1.0f) || !(hp->beta2 >= 0.0f && hp->beta2 < 1.0f))
    return fail(LOCO_ERR_INVALID_ARG, "beta1 = %g, beta2 = %g must lie in [0, 1)", hp->beta1, hp->beta2);
  if (count < 0) return fail(LOCO_ERR_INVALID_ARG, "count = %d < 0", count);
  if (count == 0) return done();
  if (tensors == nullptr) return fail(LOCO_ERR_INVALID_ARG, "tensors is NULL");
  for (int i = 0; i < count; ++i) {
    const loco_adam_tensor& x = tensors[i];
    if (x.n < 0 || x.n > LOCO_MAX_N)
      return fail(LOCO_ERR_INVALID_ARG, "tensors[%d].n = %lld outside [0, LOCO_MAX_N = 2^48]", i, (long long)x.n);
    if (!isfinite(x.lr_scale) || !isfinite(x.decay_scale))
      return fail(LOCO_ERR_INVALID_ARG, "tensors[%d]: lr_scale = %g and decay_scale = %g must be finite", i, x.lr_scale,
                  x.decay_scale);
    if (x.n > 0 && x.param_bf16 != nullptr && cfg->param_dtype == LOCO_BF16)
      return fail(LOCO_ERR_INVALID_ARG, "tensors[%d].param_bf16 must be NULL: the parameters are bf16", i);
  }
  Ranges all;
  LOCO_TRY(check_tensors(*cfg, tensors, count, grad_scale, &all));
  AdamTensorsArgs a;
  a.beta1 = hp->beta1, a.beta2 = hp->beta2;
  a.one_minus_beta1 = 1.0f - hp->beta1, a.one_minus_beta2 = 1.0f - hp->beta2;
  a.c2 = 1.0f;
  if (hp->bias_correction) {
    const double bc2 = 1.0 - pow(double(hp->beta2), double(t));
    a.c2 = hp->eps_inside_sqrt ? float(1.0 / bc2) : float(1.0 / sqrt(bc2));
  }
  a.eps = hp->eps, a.eps_inside_sqrt = hp->eps_inside_sqrt != 0;
  a.neg_zero = -0.0f;
  a.grad_scale = grad_scale;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (count <= kAdamFew) return launch_some<kAdamFew>(*cfg, tensors, 0, count, *hp, t, a, s);
  for (int at = 0; at < count; at += kAdamMany)
    LOCO_TRY(launch_some<kAdamMany>(*cfg, tensors, at, std::min(kAdamMany, count - at), *hp, t, a, s));
  return LOCO_OK;
}

loco_status loco_adam_state_decode(int32_t kind, const void* codes, const float* steps, int64_t n, void* out,
                                   int32_t out_dtype, loco_stream_t stream) {
  if (kind != LOCO_STATE_M && kind != LOCO_STATE_V)
    return fail(LOCO_ERR_UNSUPPORTED, "kind = %d (LOCO_STATE_M or LOCO_STATE_V)", kind);
  LOCO_TRY(check_dtype(out_dtype, "out_dtype"));
  if (n < 0 || n > LOCO_MAX_N)
    return fail(LOCO_ERR_INVALID_ARG, "n = %lld outside [0, LOCO_MAX_N = 2^48]", (long long)n);
  if (n == 0) return done();
  const int64_t nb = (n + LOCO_STATE_BLOCK - 1) / LOCO_STATE_BLOCK;
  const size_t oe = elem_size(out_dtype);
  const BufCheck b[3] = {{codes, size_t(nb) * LOCO_STATE_BLOCK, 16, "codes"}, {steps, size_t(nb) * 4, 4, "steps"},
                         {out, size_t(n) * oe, oe, "out"}};
  LOCO_TRY(check_buffers(b, 3));
  for (int i = 0; i < 2; ++i)
    if (overlap(b[i].p, b[i].bytes, out, b[2].bytes)) return fail(LOCO_ERR_INVALID_ARG, "out overlaps %s", b[i].name);
  return launch_result(launch_state_decode(kind == LOCO_STATE_V, codes, steps, n, out, out_dtype == LOCO_BF16,
                                           reinterpret_cast<cudaStream_t>(stream)),
                       "loco_adam_state_decode");
}

}  // extern "C"
