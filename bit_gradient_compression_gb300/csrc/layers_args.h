// Argument checks of the entry points that take matrices (layers_abi.cu, steps_abi.cu): everything is
// checked on the host before anything is launched, so a refused call writes nothing.
#pragma once

#include <math.h>

#include "abi_checks.h"
#include "loco.h"

namespace loco {

namespace {

constexpr int64_t kMaxDim = LOCO_MAX_DIM;

inline size_t elem_size(int32_t dtype) { return dtype == LOCO_BF16 ? 2 : 4; }

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
inline bool mats_overlap(const Mat& x, const Mat& y) {
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

constexpr int kMaxMats = 24;

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

inline loco_status check_dtype(int32_t d, const char* name) {
  if (d != LOCO_F32 && d != LOCO_BF16)
    return fail(LOCO_ERR_UNSUPPORTED, "%s = %d (LOCO_F32 or LOCO_BF16)", name, d);
  return LOCO_OK;
}

inline loco_status check_dim(int64_t v, int64_t least, const char* name) {
  if (v < least || v > kMaxDim)
    return fail(LOCO_ERR_INVALID_ARG, "%s = %lld outside [%lld, LOCO_MAX_DIM]", name, (long long)v, (long long)least);
  return LOCO_OK;
}

inline loco_status check_act(int32_t act) {
  if (act < LOCO_ACT_NONE || act > LOCO_ACT_SILU) return fail(LOCO_ERR_UNSUPPORTED, "act = %d", act);
  return LOCO_OK;
}

inline loco_status both_or_neither(const void* codes, const void* scales) {
  if ((codes == nullptr) != (scales == nullptr))
    return fail(LOCO_ERR_INVALID_ARG, "codes and scales go together: one of them is NULL");
  return LOCO_OK;
}

inline loco_status done() {
  return launch_result(cudaSuccess, "");
}

#define LOCO_TRY(call)                         \
  do {                                         \
    const loco_status st_ = (call);            \
    if (st_ != LOCO_OK) return st_;            \
  } while (0)

}  // namespace

}  // namespace loco
