// Layer norm and RMS norm: forward with an optional 8-bit checkpoint of the
// normalised rows, backward from the input or from that checkpoint, with the
// reduction of the parameters' gradients.
//
// Both directions are bound by memory.  A row belongs to a group of G threads
// (a warp up to 1024 columns, else a CTA) that keeps it in registers, so it is
// read once: the mean, then the sum of squared deviations (two passes over
// registers, no cancellation), then the output.  Thread t of a group holds
// vectors t, t + G, ... of 8 columns (WIDE), or single columns t, t + G, ...
// where a row cannot be loaded 16 bytes at a time; either way 32 consecutive
// columns are 4 lanes or 32 lanes of one warp, which gives a checkpoint block
// its largest magnitude with two shuffles or one warp reduction.
//
// The backward pass walks rows with a fixed grid; each thread keeps the sums of
// dgamma and dbeta of its own columns in registers over all its CTA's rows, one
// partial row per CTA goes to the workspace, and a second kernel adds the
// partial rows in order: no atomics, the same result every run.
#include <atomic>

#include "layers_common.cuh"

namespace loco {

namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Sums of N values over the group's G threads, the same in all of them.  `red` holds 32 floats per
// value; consecutive calls alternate between two such areas, so one barrier per call is enough.
template <int G, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float* red) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if constexpr (G > 32) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) red[i * 32 + warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = warp_sum(lane < G / 32 ? red[i * 32 + lane] : 0.0f);
  }
}

template <int G>
constexpr int kCtaThreads = G == 32 ? 256 : G;

// Column of element k of a thread's vector e.
template <int G, bool WIDE>
__device__ __forceinline__ int col_of(int t, int e, int k) {
  return WIDE ? (t + G * e) * 8 + k : t + G * (e * 8 + k);
}

// Eight elements of a row held by one thread, 0 past the last column.  RW: the kernel may write the row.
template <int G, bool WIDE, bool BF16, bool RW = false>
__device__ __forceinline__ void load_vec(const void* row, int cols, int t, int e, float v[8]) {
  const int c0 = col_of<G, WIDE>(t, e, 0);
  if (WIDE && c0 + 8 <= cols) {
    load8<RW>(row, c0, BF16, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = col_of<G, WIDE>(t, e, k);
      v[k] = c < cols ? (RW ? load_elem_rw(row, c, BF16) : load_elem(row, c, BF16)) : 0.0f;
    }
  }
}
template <int G, bool WIDE>
__device__ __forceinline__ void store_vec(void* row, int cols, int t, int e, int bf16, const float v[8]) {
  const int c0 = col_of<G, WIDE>(t, e, 0);
  if (WIDE && c0 + 8 <= cols) {
    store8(row, c0, bf16, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = col_of<G, WIDE>(t, e, k);
      if (c < cols) store_elem(row, c, bf16, v[k]);
    }
  }
}
// A parameter vector's elements; `wide`: it is 16-byte aligned.
template <int G, bool WIDE>
__device__ __forceinline__ void load_param(const void* p, int cols, int t, int e, int bf16, bool wide, float none,
                                           float v[8]) {
  const int c0 = col_of<G, WIDE>(t, e, 0);
  if (p == nullptr) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = none;
  } else if (WIDE && wide && c0 + 8 <= cols) {
    load8(p, c0, bf16, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = col_of<G, WIDE>(t, e, k);
      v[k] = c < cols ? load_elem(p, c, bf16) : none;
    }
  }
}

__device__ __forceinline__ const void* at(const void* p, int64_t i, int bf16) {
  return static_cast<const char*>(p) + i * (bf16 ? 2 : 4);
}
__device__ __forceinline__ void* at(void* p, int64_t i, int bf16) { return static_cast<char*>(p) + i * (bf16 ? 2 : 4); }

// Codes and scales of the vector's 8 values (0 past cols); every lane of the warp takes part.
template <int G, bool WIDE>
__device__ __forceinline__ void store_codes(const NormFwdArgs& a, int64_t row, int t, int e, int nb, const float v[8]) {
  if constexpr (WIDE) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, mag_bits(v[k]));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    const int g = t + G * e;
    if (g < nb * 4) {
      const uint32_t sc = ckpt_scale(m);
      const float inv = ckpt_inv_step(sc);
      reinterpret_cast<uint2*>(a.codes + row * nb * kCkptBlock)[g] =
          make_uint2(ckpt_pack4(v, inv), ckpt_pack4(v + 4, inv));
      if ((g & 3) == 0) a.scales[row * nb + g / 4] = uint8_t(sc);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = col_of<G, WIDE>(t, e, k);
      const uint32_t sc = ckpt_scale(__reduce_max_sync(0xFFFFFFFFu, mag_bits(v[k])));
      if (c / kCkptBlock < nb) {
        a.codes[row * nb * kCkptBlock + c] = int8_t(ckpt_code(v[k], ckpt_inv_step(sc)));
        if ((c & 31) == 0) a.scales[row * nb + c / kCkptBlock] = uint8_t(sc);
      }
    }
  }
}

template <int G, int NV, bool XBF16, bool WIDE>
__global__ void __launch_bounds__(kCtaThreads<G>) k_norm_fwd(NormFwdArgs a, bool pwide) {
  __shared__ float red[2][32];
  const int t = G == 32 ? threadIdx.x & 31 : threadIdx.x;
  const int64_t row = G == 32 ? int64_t(blockIdx.x) * (kCtaThreads<G> / 32) + threadIdx.x / 32 : blockIdx.x;
  if (row >= a.rows) return;  // the whole group: a warp, or (never) a CTA
  const int cols = int(a.cols), nb = (cols + kCkptBlock - 1) / kCkptBlock;
  const void* xr = at(a.x, row * a.ldx, XBF16);
  float x[NV][8];
#pragma unroll
  for (int e = 0; e < NV; ++e) load_vec<G, WIDE, XBF16>(xr, cols, t, e, x[e]);
  float mean = 0.0f;
  if (!a.rms) {
    float s[1] = {0.0f};
#pragma unroll
    for (int e = 0; e < NV; ++e)
#pragma unroll
      for (int k = 0; k < 8; ++k) s[0] += x[e][k];
    group_sum<G>(s, red[0]);
    mean = s[0] / float(cols);
  }
  float q[1] = {0.0f};
#pragma unroll
  for (int e = 0; e < NV; ++e)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[e][k] = col_of<G, WIDE>(t, e, k) < cols ? x[e][k] - mean : 0.0f;
      q[0] = fmaf(x[e][k], x[e][k], q[0]);
    }
  group_sum<G>(q, red[1]);
  const float rstd = 1.0f / sqrtf(q[0] / float(cols) + a.eps);
  if (t == 0) {
    if (a.mean != nullptr && !a.rms) a.mean[row] = mean;
    if (a.rstd != nullptr) a.rstd[row] = rstd;
  }
  void* yr = at(a.y, row * a.ldy, a.y_bf16);
#pragma unroll
  for (int e = 0; e < NV; ++e) {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[e][k] *= rstd;
    if (a.codes != nullptr) store_codes<G, WIDE>(a, row, t, e, nb, x[e]);
    if (col_of<G, WIDE>(t, e, 0) < cols) {
      float g[8], b[8];
      load_param<G, WIDE>(a.gamma, cols, t, e, a.param_bf16, pwide, 1.0f, g);
      load_param<G, WIDE>(a.beta, cols, t, e, a.param_bf16, pwide, 0.0f, b);
#pragma unroll
      for (int k = 0; k < 8; ++k) x[e][k] = fmaf(x[e][k], g[k], b[k]);
      store_vec<G, WIDE>(yr, cols, t, e, a.y_bf16, x[e]);
    }
  }
}

// Rows too long for the registers of a CTA: three passes over the row, which the L2 cache serves
// after the first.
constexpr int kLoop = 512;

template <bool XBF16>
__global__ void __launch_bounds__(kLoop) k_norm_fwd_long(NormFwdArgs a) {
  __shared__ float red[2][32];
  const int64_t row = blockIdx.x;
  const int cols = int(a.cols), nb = (cols + kCkptBlock - 1) / kCkptBlock;
  const void* xr = at(a.x, row * a.ldx, XBF16);
  float mean = 0.0f;
  if (!a.rms) {
    float s[1] = {0.0f};
    for (int64_t c = threadIdx.x; c < cols; c += kLoop) s[0] += load_elem(xr, c, XBF16);
    group_sum<kLoop>(s, red[0]);
    mean = s[0] / float(cols);
  }
  float q[1] = {0.0f};
  for (int64_t c = threadIdx.x; c < cols; c += kLoop) {
    const float d = load_elem(xr, c, XBF16) - mean;
    q[0] = fmaf(d, d, q[0]);
  }
  group_sum<kLoop>(q, red[1]);
  const float rstd = 1.0f / sqrtf(q[0] / float(cols) + a.eps);
  if (threadIdx.x == 0) {
    if (a.mean != nullptr && !a.rms) a.mean[row] = mean;
    if (a.rstd != nullptr) a.rstd[row] = rstd;
  }
  void* yr = at(a.y, row * a.ldy, a.y_bf16);
  const int64_t pitch = int64_t(nb) * kCkptBlock;  // a multiple of 32: whole warps enter and leave together
  for (int64_t c = threadIdx.x; c < pitch; c += kLoop) {
    const float v = c < cols ? (load_elem(xr, c, XBF16) - mean) * rstd : 0.0f;
    if (a.codes != nullptr) {
      const uint32_t sc = ckpt_scale(__reduce_max_sync(0xFFFFFFFFu, mag_bits(v)));
      a.codes[row * pitch + c] = int8_t(ckpt_code(v, ckpt_inv_step(sc)));
      if ((c & 31) == 0) a.scales[row * nb + c / kCkptBlock] = uint8_t(sc);
    }
    if (c < cols)
      store_elem(yr, c, a.y_bf16, fmaf(v, a.gamma ? load_elem(a.gamma, c, a.param_bf16) : 1.0f,
                                       a.beta ? load_elem(a.beta, c, a.param_bf16) : 0.0f));
  }
}

// ---------------------------------------------------------------------------------------- backward

// The normalised values of a thread's vector e, from x and the row's statistics or from the checkpoint.
template <int G, bool WIDE, bool XBF16, bool CKPT>
__device__ __forceinline__ void load_xhat(const NormBwdArgs& a, int64_t row, int cols, int nb, int t, int e,
                                          float mean, float rstd, float v[8]) {
  if constexpr (CKPT) {
    if constexpr (WIDE) {
      const int g = t + G * e;
      if (g < nb * 4) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(a.codes + row * nb * kCkptBlock) + g);
        const float st = ckpt_step(__ldg(a.scales + row * nb + g / 4));
        ckpt_unpack4(w.x, st, v);
        ckpt_unpack4(w.y, st, v + 4);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (g * 8 + k >= cols) v[k] = 0.0f;  // a bad block's padding reads back as NaN
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = 0.0f;
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int c = col_of<G, WIDE>(t, e, k);
        v[k] = c < cols ? float(__ldg(a.codes + row * nb * kCkptBlock + c)) *
                              ckpt_step(__ldg(a.scales + row * nb + c / kCkptBlock))
                        : 0.0f;
      }
    }
  } else {
    load_vec<G, WIDE, XBF16>(at(a.x, row * a.ldx, XBF16), cols, t, e, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = col_of<G, WIDE>(t, e, k) < cols ? (v[k] - mean) * rstd : 0.0f;
  }
}

template <int G, int NV, bool XBF16, bool WIDE, bool CKPT>
__global__ void __launch_bounds__(kCtaThreads<G>) k_norm_bwd(NormBwdArgs a, bool pwide) {
  __shared__ float red[2][64];
  extern __shared__ float cols_sm[];  // [2][cols], only where a CTA holds several groups
  constexpr int kGroups = kCtaThreads<G> / G;
  const int t = threadIdx.x % G, grp = threadIdx.x / G;
  const int cols = int(a.cols), nb = (cols + kCkptBlock - 1) / kCkptBlock;
  float dg[NV][8], db[NV][8];
#pragma unroll
  for (int e = 0; e < NV; ++e)
#pragma unroll
    for (int k = 0; k < 8; ++k) dg[e][k] = db[e][k] = 0.0f;
  int turn = 0;
  for (int64_t row = int64_t(blockIdx.x) * kGroups + grp; row < a.rows; row += int64_t(gridDim.x) * kGroups) {
    const float rstd = __ldg(a.rstd + row);
    const float mean = CKPT || a.rms ? 0.0f : __ldg(a.mean + row);
    const void* dyr = at(a.dy, row * a.lddy, a.y_bf16);
    float g[NV][8], xh[NV][8];
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < NV; ++e) {
      if (a.y_bf16)
        load_vec<G, WIDE, true>(dyr, cols, t, e, g[e]);
      else
        load_vec<G, WIDE, false>(dyr, cols, t, e, g[e]);
      load_xhat<G, WIDE, XBF16, CKPT>(a, row, cols, nb, t, e, mean, rstd, xh[e]);
      float gm[8];
      load_param<G, WIDE>(a.gamma, cols, t, e, a.param_bf16, pwide, 1.0f, gm);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        dg[e][k] = fmaf(g[e][k], xh[e][k], dg[e][k]);
        db[e][k] += g[e][k];
        g[e][k] *= gm[k];
        s[0] += g[e][k];
        s[1] = fmaf(g[e][k], xh[e][k], s[1]);
      }
    }
    group_sum<G>(s, red[turn]);
    turn ^= 1;
    const float c1 = a.rms ? 0.0f : s[0] / float(cols), c2 = s[1] / float(cols);
    void* dxr = at(a.dx, row * a.lddx, XBF16);
#pragma unroll
    for (int e = 0; e < NV; ++e) {
      if (col_of<G, WIDE>(t, e, 0) >= cols) continue;
      float r[8];
      if (a.residual != nullptr) {
        load_vec<G, WIDE, XBF16, true>(at(a.residual, row * a.ldr, XBF16), cols, t, e, r);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) r[k] = 0.0f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) r[k] = fmaf(rstd, fmaf(-xh[e][k], c2, g[e][k] - c1), r[k]);
      store_vec<G, WIDE>(dxr, cols, t, e, XBF16, r);
    }
  }
  if (a.partials == nullptr) return;
  float* out = a.partials + int64_t(blockIdx.x) * 2 * cols;
  if constexpr (kGroups == 1) {
#pragma unroll
    for (int e = 0; e < NV; ++e)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int c = col_of<G, WIDE>(t, e, k);
        if (c < cols) out[c] = dg[e][k], out[cols + c] = db[e][k];
      }
  } else {
    // the CTA's groups add their sums one after another
    for (int w = 0; w < kGroups; ++w) {
      if (grp == w) {
#pragma unroll
        for (int e = 0; e < NV; ++e)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int c = col_of<G, WIDE>(t, e, k);
            if (c < cols) {
              cols_sm[c] = (w ? cols_sm[c] : 0.0f) + dg[e][k];
              cols_sm[cols + c] = (w ? cols_sm[cols + c] : 0.0f) + db[e][k];
            }
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < 2 * cols; c += kCtaThreads<G>) out[c] = cols_sm[c];
  }
}

// One normalised value, for rows too long for registers.
template <bool XBF16>
__device__ __forceinline__ float xhat_at(const NormBwdArgs& a, int64_t row, int64_t c, int64_t nb, float mean, float rstd) {
  if (a.x != nullptr) return (load_elem(a.x, row * a.ldx + c, XBF16) - mean) * rstd;
  return float(__ldg(a.codes + row * nb * kCkptBlock + c)) * ckpt_step(__ldg(a.scales + row * nb + c / kCkptBlock));
}

template <bool XBF16>
__global__ void __launch_bounds__(kLoop) k_norm_bwd_long(NormBwdArgs a) {
  __shared__ float red[64];
  const int64_t row = blockIdx.x, cols = a.cols, nb = (cols + kCkptBlock - 1) / kCkptBlock;
  const float rstd = a.rstd[row], mean = a.x == nullptr || a.rms ? 0.0f : a.mean[row];
  float s[2] = {0.0f, 0.0f};
  for (int64_t c = threadIdx.x; c < cols; c += kLoop) {
    const float g = load_elem(a.dy, row * a.lddy + c, a.y_bf16) *
                    (a.gamma ? load_elem(a.gamma, c, a.param_bf16) : 1.0f);
    s[0] += g;
    s[1] = fmaf(g, xhat_at<XBF16>(a, row, c, nb, mean, rstd), s[1]);
  }
  group_sum<kLoop>(s, red);
  const float c1 = a.rms ? 0.0f : s[0] / float(cols), c2 = s[1] / float(cols);
  for (int64_t c = threadIdx.x; c < cols; c += kLoop) {
    const float g = load_elem(a.dy, row * a.lddy + c, a.y_bf16) *
                    (a.gamma ? load_elem(a.gamma, c, a.param_bf16) : 1.0f);
    const float r = a.residual != nullptr ? load_elem_rw(a.residual, row * a.ldr + c, XBF16) : 0.0f;
    store_elem(a.dx, row * a.lddx + c, XBF16,
               fmaf(rstd, fmaf(-xhat_at<XBF16>(a, row, c, nb, mean, rstd), c2, g - c1), r));
  }
}

// Column sums of a slice of rows, for the long rows: 32 columns per CTA, 8 rows at a time.
template <bool XBF16>
__global__ void __launch_bounds__(256) k_norm_bwd_cols(NormBwdArgs a, int64_t rows_per) {
  __shared__ float sm[2][8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int64_t c = int64_t(blockIdx.x) * 32 + lane, nb = (a.cols + kCkptBlock - 1) / kCkptBlock;
  const int64_t lo = int64_t(blockIdx.y) * rows_per, hi = min(lo + rows_per, a.rows);
  float dg = 0.0f, db = 0.0f;
  if (c < a.cols)
    for (int64_t row = lo + warp; row < hi; row += 8) {
      const float d = load_elem(a.dy, row * a.lddy + c, a.y_bf16);
      const float mean = a.x == nullptr || a.rms ? 0.0f : __ldg(a.mean + row);
      dg = fmaf(d, xhat_at<XBF16>(a, row, c, nb, mean, __ldg(a.rstd + row)), dg);
      db += d;
    }
  sm[0][warp][lane] = dg, sm[1][warp][lane] = db;
  __syncthreads();
  if (warp < 2 && c < a.cols) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += sm[warp][w][lane];
    a.partials[(int64_t(blockIdx.y) * 2 + warp) * a.cols + c] = v;
  }
}

// dgamma and dbeta from the partial rows, added in a fixed order: 32 columns per CTA, each of 32
// warps the rows p = warp, warp + 32, ..., the warps' sums in order.
__global__ void __launch_bounds__(1024) k_norm_bwd_join(const float* partials, int parts, int64_t cols, void* dgamma,
                                                        void* dbeta, int bf16) {
  __shared__ float sm[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int64_t c = int64_t(blockIdx.x) * 32 + lane;
  void* out = blockIdx.y == 0 ? dgamma : dbeta;
  if (out == nullptr) return;  // the whole CTA
  float v = 0.0f;
  if (c < cols)
    for (int p = warp; p < parts; p += 32) v += partials[(int64_t(p) * 2 + blockIdx.y) * cols + c];
  sm[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < cols) {
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < 32; ++w) v += sm[w][lane];
    store_elem(out, c, bf16, v);
  }
}

// ---------------------------------------------------------------------------------------- launches

bool wide_rows(const void* p, int64_t ld, int64_t rows, int bf16) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || ld * (bf16 ? 2 : 4) % 16 == 0);
}
bool wide_vec(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <int G, int NV>
cudaError_t fwd(const NormFwdArgs& a, bool wide, bool pwide, cudaStream_t s) {
  constexpr int T = kCtaThreads<G>;
  const unsigned grid = unsigned((a.rows + T / G - 1) / (T / G));
  if (a.x_bf16)
    (wide ? k_norm_fwd<G, NV, true, true> : k_norm_fwd<G, NV, true, false>)<<<grid, T, 0, s>>>(a, pwide);
  else
    (wide ? k_norm_fwd<G, NV, false, true> : k_norm_fwd<G, NV, false, false>)<<<grid, T, 0, s>>>(a, pwide);
  return cudaGetLastError();
}

template <int G, int NV, bool XBF16, bool WIDE, bool CKPT>
cudaError_t bwd_launch(const NormBwdArgs& a, bool pwide, int* parts, cudaStream_t s) {
  constexpr int T = kCtaThreads<G>, groups = T / G;
  const size_t sm = groups > 1 ? size_t(a.cols) * 8 : 0;
  static std::atomic<int> known[64];
  int dev = 0, cap = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || (cap = known[dev].load(std::memory_order_relaxed)) == 0) {
    int sms = 0, per = 0;
    if ((e = sm_count(&sms)) != cudaSuccess) return e;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, k_norm_bwd<G, NV, XBF16, WIDE, CKPT>, T,
                                                      groups > 1 ? size_t(G) * NV * 64 : 0);
    if (e != cudaSuccess) return e;
    cap = sms * (per < 1 ? 1 : per);
    if (cap > kNormPartials) cap = kNormPartials;
    if (dev < 64) known[dev].store(cap, std::memory_order_relaxed);
  }
  const int64_t want = (a.rows + groups - 1) / groups;
  *parts = int(want < cap ? want : cap);
  k_norm_bwd<G, NV, XBF16, WIDE, CKPT><<<*parts, T, sm, s>>>(a, pwide);
  return cudaGetLastError();
}

template <int G, int NV>
cudaError_t bwd(const NormBwdArgs& a, bool wide, bool pwide, int* parts, cudaStream_t s) {
  const bool ck = a.x == nullptr;
  if (a.x_bf16) {
    if (wide) return ck ? bwd_launch<G, NV, true, true, true>(a, pwide, parts, s) : bwd_launch<G, NV, true, true, false>(a, pwide, parts, s);
    return ck ? bwd_launch<G, NV, true, false, true>(a, pwide, parts, s) : bwd_launch<G, NV, true, false, false>(a, pwide, parts, s);
  }
  if (wide) return ck ? bwd_launch<G, NV, false, true, true>(a, pwide, parts, s) : bwd_launch<G, NV, false, true, false>(a, pwide, parts, s);
  return ck ? bwd_launch<G, NV, false, false, true>(a, pwide, parts, s) : bwd_launch<G, NV, false, false, false>(a, pwide, parts, s);
}

}  // namespace

cudaError_t launch_norm_forward(const NormFwdArgs& a, cudaStream_t s) {
  const bool wide = wide_rows(a.x, a.ldx, a.rows, a.x_bf16) && wide_rows(a.y, a.ldy, a.rows, a.y_bf16);
  const bool pwide = wide_vec(a.gamma) && wide_vec(a.beta);
  const int64_t pitch = (a.cols + kCkptBlock - 1) / kCkptBlock * kCkptBlock;
  if (pitch <= 256) return fwd<32, 1>(a, wide, pwide, s);
  if (pitch <= 512) return fwd<32, 2>(a, wide, pwide, s);
  if (pitch <= 1024) return fwd<32, 4>(a, wide, pwide, s);
  if (pitch <= 2048) return fwd<128, 2>(a, wide, pwide, s);
  if (pitch <= 4096) return fwd<256, 2>(a, wide, pwide, s);
  if (pitch <= 8192) return fwd<512, 2>(a, wide, pwide, s);
  if (pitch <= 16384) return fwd<512, 4>(a, wide, pwide, s);
  (a.x_bf16 ? k_norm_fwd_long<true> : k_norm_fwd_long<false>)<<<unsigned(a.rows), kLoop, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_norm_backward(const NormBwdArgs& a, cudaStream_t s) {
  int parts = 0;
  cudaError_t e = cudaSuccess;
  if (a.rows > 0) {
    const bool wide = wide_rows(a.dy, a.lddy, a.rows, a.y_bf16) && wide_rows(a.dx, a.lddx, a.rows, a.x_bf16) &&
                      (a.x == nullptr || wide_rows(a.x, a.ldx, a.rows, a.x_bf16)) &&
                      (a.residual == nullptr || wide_rows(a.residual, a.ldr, a.rows, a.x_bf16));
    const bool pwide = wide_vec(a.gamma);
    const int64_t pitch = (a.cols + kCkptBlock - 1) / kCkptBlock * kCkptBlock;
    if (pitch <= 256) e = bwd<32, 1>(a, wide, pwide, &parts, s);
    else if (pitch <= 512) e = bwd<32, 2>(a, wide, pwide, &parts, s);
    else if (pitch <= 1024) e = bwd<32, 4>(a, wide, pwide, &parts, s);
    else if (pitch <= 2048) e = bwd<128, 2>(a, wide, pwide, &parts, s);
    else if (pitch <= 4096) e = bwd<256, 2>(a, wide, pwide, &parts, s);
    else if (pitch <= 8192) e = bwd<512, 2>(a, wide, pwide, &parts, s);
    else {
      if (a.partials != nullptr) {
        // before dx, which may overwrite a residual but none of these inputs
        const int64_t strips = (a.cols + 31) / 32;
        const int64_t want = (a.rows + 63) / 64;
        parts = int(want < 64 ? want : 64);
        const int64_t per = (a.rows + parts - 1) / parts;
        const dim3 grid{unsigned(strips), unsigned(parts)};
        (a.x_bf16 ? k_norm_bwd_cols<true> : k_norm_bwd_cols<false>)<<<grid, 256, 0, s>>>(a, per);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
      }
      (a.x_bf16 ? k_norm_bwd_long<true> : k_norm_bwd_long<false>)<<<unsigned(a.rows), kLoop, 0, s>>>(a);
      e = cudaGetLastError();
    }
    if (e != cudaSuccess) return e;
  }
  if (a.dgamma == nullptr && a.dbeta == nullptr) return cudaSuccess;
  const dim3 grid{unsigned((a.cols + 31) / 32), 2};
  k_norm_bwd_join<<<grid, 1024, 0, s>>>(a.partials, parts, a.cols, a.dgamma, a.dbeta, a.grad_bf16);
  return cudaGetLastError();
}

}  // namespace loco
