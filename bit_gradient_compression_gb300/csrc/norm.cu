// Layer norm and RMS norm: forward with an optional 8-bit checkpoint of the
// normalised rows, backward from the input or from that checkpoint, with the
// reduction of the parameters' gradients.
//
// Both directions are bound by memory.  A row belongs to a group of G threads
// (a warp up to 256 columns, else up to a CTA) that keeps it in registers, so it
// is read once: the mean, then the sum of squared deviations (two passes over
// registers, no cancellation), then the output.  Thread t of a group holds
// vectors t, t + G, ... of 8 columns (WIDE), or single columns t, t + G, ...
// where a row cannot be loaded 16 bytes at a time; either way 32 consecutive
// columns are 4 lanes or 32 lanes of one warp, which gives a checkpoint block
// its largest magnitude with two shuffles or one warp reduction.
//
// The grid is as large as fits and walks the rows.  A row's sums need all of it,
// so the next rows have to be on their way meanwhile: WIDE threads copy their
// own 16-byte pieces of the next kStages - 1 rows into shared memory (cp.async;
// nobody else reads them, so no barrier is needed), the others load the next
// row into registers.
//
// In the backward pass each thread keeps the sums of dgamma and dbeta of its own
// columns in registers over all its rows, one partial row per CTA goes to the
// workspace, and a second kernel adds the partial rows in order: no atomics, the
// same result every run.
#include <atomic>

#include "device_common.cuh"
#include "layers_common.cuh"

namespace loco {

namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

template <int G>
constexpr int kCtaThreads = G < 256 ? 256 : G;

// Sums of N values over the group's G threads, the same in all of them; every thread of the CTA
// takes part.  `red` holds 32 floats per value, and consecutive calls of a loop alternate between
// two such areas, so that one barrier per call is enough.
template <int G, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float* red) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if constexpr (G > 32) {
    constexpr int kWarps = G / 32;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, first = warp / kWarps * kWarps;
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) red[i * 32 + warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = lane < kWarps ? red[i * 32 + first + lane] : 0.0f;
#pragma unroll
      for (int o = kWarps / 2; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
      v[i] = __shfl_sync(0xFFFFFFFFu, v[i], 0);
    }
  }
}

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
      reinterpret_cast<uint2*>(a.codes + row * nb * kCkptBlock)[g] = ckpt_pack8(v, m);
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

// ---- the next rows' pieces in shared memory (WIDE)

// A thread's 16-byte pieces: piece i of stage s at ring + ((s * pieces + i) * threads + thread) * 16.
template <int T>
__device__ __forceinline__ uint4* piece(uint8_t* ring, int pieces, int stage, int i) {
  return reinterpret_cast<uint4*>(ring) + (stage * pieces + i) * T + threadIdx.x;
}
// Starts the copy of a thread's whole vectors of one row: NV pieces (bf16) or 2 NV (fp32) from piece `first`.
template <int G, int NV>
__device__ __forceinline__ void copy_row(uint8_t* ring, int pieces, int stage, int first, const void* row, int cols, int t,
                                         int bf16) {
  constexpr int T = kCtaThreads<G>;
#pragma unroll
  for (int e = 0; e < NV; ++e) {
    const int c0 = (t + G * e) * 8;
    if (c0 + 8 > cols) continue;
    const char* q = static_cast<const char*>(row) + int64_t(c0) * (bf16 ? 2 : 4);
    if (bf16) {
      cp_async16(piece<T>(ring, pieces, stage, first + e), q);
    } else {
      cp_async16(piece<T>(ring, pieces, stage, first + 2 * e), q);
      cp_async16(piece<T>(ring, pieces, stage, first + 2 * e + 1), q + 16);
    }
  }
}
__device__ __forceinline__ void widen(uint4 a, float v[8]) {
  const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) v[2 * k] = __uint_as_float(u[k] << 16), v[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
}
// Vector e of the row that was copied; `row` itself serves a vector the row ends in.
template <int G, int NV, bool RW = false>
__device__ __forceinline__ void copied_vec(uint8_t* ring, int pieces, int stage, int first, const void* row, int cols,
                                           int t, int e, int bf16, float v[8]) {
  constexpr int T = kCtaThreads<G>;
  if ((t + G * e) * 8 + 8 <= cols) {
    if (bf16) {
      widen(*piece<T>(ring, pieces, stage, first + e), v);
    } else {
      const uint4 a = *piece<T>(ring, pieces, stage, first + 2 * e), b = *piece<T>(ring, pieces, stage, first + 2 * e + 1);
      const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(u[k]);
    }
  } else if (bf16) {
    load_vec<G, true, true, RW>(row, cols, t, e, v);
  } else {
    load_vec<G, true, false, RW>(row, cols, t, e, v);
  }
}

template <int G, int NV, bool XBF16>
constexpr int kFwdPieces = NV * (XBF16 ? 1 : 2);
// Stages: a row of 16384 fp32 columns takes 64 KB of shared memory.
template <int NV, bool XBF16>
constexpr int kFwdRing = XBF16 || NV < 4 ? 4 : 3;

template <int G, int NV, bool XBF16, bool WIDE>
__global__ void __launch_bounds__(kCtaThreads<G>, kCtaThreads<G> == 512 ? 1 : 2) k_norm_fwd(NormFwdArgs a, bool pwide) {
  __shared__ float red[2][32];
  extern __shared__ __align__(16) uint8_t ring[];
  constexpr int kGroups = kCtaThreads<G> / G, kP = kFwdPieces<G, NV, XBF16>, kFwdStages = kFwdRing<NV, XBF16>;
  constexpr bool kKeep = NV <= 2;  // gamma and beta stay in registers
  const int t = threadIdx.x % G, grp = threadIdx.x / G;
  const int cols = int(a.cols), nb = (cols + kCkptBlock - 1) / kCkptBlock;
  const int64_t step = int64_t(gridDim.x) * kGroups, first = int64_t(blockIdx.x) * kGroups + grp;
  float gm[NV][8], bt[NV][8], nx[NV][8];
  if constexpr (kKeep) {
#pragma unroll
    for (int e = 0; e < NV; ++e) {
      load_param<G, WIDE>(a.gamma, cols, t, e, a.param_bf16, pwide, 1.0f, gm[e]);
      load_param<G, WIDE>(a.beta, cols, t, e, a.param_bf16, pwide, 0.0f, bt[e]);
    }
  }
  const auto x_row = [&](int64_t row) { return at(a.x, row * a.ldx, XBF16); };
  if constexpr (WIDE) {
#pragma unroll
    for (int i = 0; i < kFwdStages - 1; ++i) {
      const int64_t row = first + i * step;
      if (row < a.rows) copy_row<G, NV>(ring, kP, i, 0, x_row(row), cols, t, XBF16);
      cp_async_commit();
    }
  } else if (first < a.rows) {
#pragma unroll
    for (int e = 0; e < NV; ++e) load_vec<G, WIDE, XBF16>(x_row(first), cols, t, e, nx[e]);
  }
  int stage = 0, turn = 0;
  // the CTA's groups go through the loop together
  for (int64_t row = first; row - grp < a.rows; row += step) {
    const bool live = row < a.rows;
    float x[NV][8];
    if constexpr (WIDE) {
      const int64_t ahead = row + (kFwdStages - 1) * step;
      if (ahead < a.rows)
        copy_row<G, NV>(ring, kP, (stage + kFwdStages - 1) % kFwdStages, 0, x_row(ahead), cols, t, XBF16);
      cp_async_commit();
      cp_async_wait<kFwdStages - 1>();
#pragma unroll
      for (int e = 0; e < NV; ++e) {
        if (live) {
          copied_vec<G, NV>(ring, kP, stage, 0, x_row(row), cols, t, e, XBF16, x[e]);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) x[e][k] = 0.0f;
        }
      }
      stage = (stage + 1) % kFwdStages;
    } else {
#pragma unroll
      for (int e = 0; e < NV; ++e)
#pragma unroll
        for (int k = 0; k < 8; ++k) x[e][k] = live ? nx[e][k] : 0.0f;
      if (row + step < a.rows) {
#pragma unroll
        for (int e = 0; e < NV; ++e) load_vec<G, WIDE, XBF16>(x_row(row + step), cols, t, e, nx[e]);
      }
    }
    float mean = 0.0f;
    if (!a.rms) {
      float s[1] = {0.0f};
#pragma unroll
      for (int e = 0; e < NV; ++e)
#pragma unroll
        for (int k = 0; k < 8; ++k) s[0] += x[e][k];
      group_sum<G>(s, red[turn]);
      turn ^= 1;
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
    group_sum<G>(q, red[turn]);
    turn ^= 1;
    const float rstd = 1.0f / sqrtf(q[0] / float(cols) + a.eps);
    if (t == 0 && live) {
      if (a.mean != nullptr && !a.rms) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    if (!live) continue;  // whole warps
    void* yr = at(a.y, row * a.ldy, a.y_bf16);
#pragma unroll
    for (int e = 0; e < NV; ++e) {
#pragma unroll
      for (int k = 0; k < 8; ++k) x[e][k] *= rstd;
      if (a.codes != nullptr) store_codes<G, WIDE>(a, row, t, e, nb, x[e]);
      if (col_of<G, WIDE>(t, e, 0) < cols) {
        if constexpr (kKeep) {
#pragma unroll
          for (int k = 0; k < 8; ++k) x[e][k] = fmaf(x[e][k], gm[e][k], bt[e][k]);
        } else {
          float g[8], b[8];
          load_param<G, WIDE>(a.gamma, cols, t, e, a.param_bf16, pwide, 1.0f, g);
          load_param<G, WIDE>(a.beta, cols, t, e, a.param_bf16, pwide, 0.0f, b);
#pragma unroll
          for (int k = 0; k < 8; ++k) x[e][k] = fmaf(x[e][k], g[k], b[k]);
        }
        store_vec<G, WIDE>(yr, cols, t, e, a.y_bf16, x[e]);
      }
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

// A row's contribution that one thread holds: dy, and x or the codes of the normalised row.
template <int G, int NV, bool XBF16, bool WIDE, bool CKPT>
struct BwdRow {
  float dy[NV][8], x[NV][8], r[NV][8];  // narrow: the values (x normalised only later)
  uint2 codes[NV];                      // WIDE from a checkpoint
  uint32_t scale[NV];
  float mean, rstd;
};

// 16-byte pieces of one stage: dy, then x, then the residual (fp32 takes two per vector).
template <int NV>
__host__ __device__ __forceinline__ int bwd_pieces(int y_bf16, int x_bf16, bool has_x, bool has_residual) {
  return NV * ((y_bf16 ? 1 : 2) + (x_bf16 ? 1 : 2) * ((has_x ? 1 : 0) + (has_residual ? 1 : 0)));
}
// As many rows ahead as shared memory holds for the widest types (a row of 8192 fp32 columns with
// fp32 dy and residual takes 96 KB).
template <int G, bool XBF16>
constexpr int kBwdStages = (G == 512 ? 2 : 3) + (XBF16 ? 1 : 0);

template <int G, int NV, bool XBF16, bool WIDE, bool CKPT>
__global__ void __launch_bounds__(kCtaThreads<G>, kCtaThreads<G> == 512 ? 1 : 2) k_norm_bwd(NormBwdArgs a, bool pwide) {
  __shared__ float red[2][64];
  extern __shared__ __align__(16) uint8_t ring[];  // the stages; after the rows, [2][cols] floats
  constexpr int T = kCtaThreads<G>, kGroups = T / G, kStages = kBwdStages<G, XBF16>;
  const int t = threadIdx.x % G, grp = threadIdx.x / G;
  const int cols = int(a.cols), nb = (cols + kCkptBlock - 1) / kCkptBlock;
  const int64_t step = int64_t(gridDim.x) * kGroups, first = int64_t(blockIdx.x) * kGroups + grp;
  const int pieces = bwd_pieces<NV>(a.y_bf16, XBF16, !CKPT, a.residual != nullptr);
  const int at_x = NV * (a.y_bf16 ? 1 : 2), at_r = at_x + (CKPT ? 0 : NV * (XBF16 ? 1 : 2));
  constexpr bool kKeep = WIDE || NV == 1;  // gamma stays in registers
  float dg[NV][8], db[NV][8], gm[NV][8];
#pragma unroll
  for (int e = 0; e < NV; ++e) {
    if constexpr (kKeep) load_param<G, WIDE>(a.gamma, cols, t, e, a.param_bf16, pwide, 1.0f, gm[e]);
#pragma unroll
    for (int k = 0; k < 8; ++k) dg[e][k] = db[e][k] = 0.0f;
  }
  // Starts the wide copies of a row.
  const auto copy = [&](int64_t row, int stage) {
    copy_row<G, NV>(ring, pieces, stage, 0, at(a.dy, row * a.lddy, a.y_bf16), cols, t, a.y_bf16);
    if constexpr (!CKPT) copy_row<G, NV>(ring, pieces, stage, at_x, at(a.x, row * a.ldx, XBF16), cols, t, XBF16);
    if (a.residual != nullptr)
      copy_row<G, NV>(ring, pieces, stage, at_r, at(a.residual, row * a.ldr, XBF16), cols, t, XBF16);
  };
  // Loads of a row that go to registers: its statistics, its codes, or all of it.
  BwdRow<G, NV, XBF16, WIDE, CKPT> nx;
  const auto load = [&](int64_t row) {
    nx.rstd = __ldg(a.rstd + row);
    nx.mean = CKPT || a.rms ? 0.0f : __ldg(a.mean + row);
    if constexpr (CKPT && WIDE) {
#pragma unroll
      for (int e = 0; e < NV; ++e) {
        const int g = t + G * e;
        nx.codes[e] = make_uint2(0, 0);
        nx.scale[e] = 1;
        if (g * 8 < cols) {
          nx.codes[e] = __ldg(reinterpret_cast<const uint2*>(a.codes + row * nb * kCkptBlock) + g);
          nx.scale[e] = __ldg(a.scales + row * nb + g / 4);
        }
      }
    }
    if constexpr (!WIDE) {
#pragma unroll
      for (int e = 0; e < NV; ++e) {
        if (a.y_bf16)
          load_vec<G, WIDE, true>(at(a.dy, row * a.lddy, true), cols, t, e, nx.dy[e]);
        else
          load_vec<G, WIDE, false>(at(a.dy, row * a.lddy, false), cols, t, e, nx.dy[e]);
        if constexpr (CKPT) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int c = col_of<G, WIDE>(t, e, k);
            nx.x[e][k] = c < cols ? float(__ldg(a.codes + row * nb * kCkptBlock + c)) *
                                        ckpt_step(__ldg(a.scales + row * nb + c / kCkptBlock))
                                  : 0.0f;
          }
        } else {
          load_vec<G, WIDE, XBF16>(at(a.x, row * a.ldx, XBF16), cols, t, e, nx.x[e]);
        }
      }
    }
  };
  if constexpr (WIDE) {
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      if (first + i * step < a.rows) copy(first + i * step, i);
      cp_async_commit();
    }
  }
  if (first < a.rows) load(first);
  int stage = 0, turn = 0;
  for (int64_t row = first; row - grp < a.rows; row += step) {
    const bool live = row < a.rows;
    float g[NV][8], xh[NV][8];
    float s[2] = {0.0f, 0.0f};
    const float rstd = live ? nx.rstd : 0.0f, mean = nx.mean;
    if constexpr (WIDE) {
      const int64_t ahead = row + (kStages - 1) * step;
      if (ahead < a.rows) copy(ahead, stage == 0 ? kStages - 1 : stage - 1);
      cp_async_commit();
      cp_async_wait<kStages - 1>();
    }
#pragma unroll
    for (int e = 0; e < NV; ++e) {
      if (live) {
        if constexpr (WIDE) {
          copied_vec<G, NV>(ring, pieces, stage, 0, at(a.dy, row * a.lddy, a.y_bf16), cols, t, e, a.y_bf16, g[e]);
          if constexpr (CKPT) {
            const float st = ckpt_step(nx.scale[e]);
            ckpt_unpack4(nx.codes[e].x, st, xh[e]);
            ckpt_unpack4(nx.codes[e].y, st, xh[e] + 4);
          } else {
            copied_vec<G, NV>(ring, pieces, stage, at_x, at(a.x, row * a.ldx, XBF16), cols, t, e, XBF16, xh[e]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) g[e][k] = nx.dy[e][k], xh[e][k] = nx.x[e][k];
        }
        if constexpr (!kKeep) load_param<G, WIDE>(a.gamma, cols, t, e, a.param_bf16, pwide, 1.0f, gm[e]);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if constexpr (!CKPT) xh[e][k] = (xh[e][k] - mean) * rstd;
          // past the last column (a bad block's padding reads back as NaN)
          if (col_of<G, WIDE>(t, e, k) >= cols) xh[e][k] = 0.0f;
          dg[e][k] = fmaf(g[e][k], xh[e][k], dg[e][k]);
          db[e][k] += g[e][k];
          g[e][k] *= gm[e][k];
          s[0] += g[e][k];
          s[1] = fmaf(g[e][k], xh[e][k], s[1]);
        }
      }
    }
    if (row + step < a.rows) load(row + step);
    group_sum<G>(s, red[turn]);
    turn ^= 1;
    const float c1 = a.rms ? 0.0f : s[0] / float(cols), c2 = s[1] / float(cols);
    if (live) {
      void* dxr = at(a.dx, row * a.lddx, XBF16);
#pragma unroll
      for (int e = 0; e < NV; ++e) {
        if (col_of<G, WIDE>(t, e, 0) >= cols) continue;
        float r[8];
        if (a.residual != nullptr) {
          const void* rr = at(a.residual, row * a.ldr, XBF16);
          if constexpr (WIDE)
            copied_vec<G, NV, true>(ring, pieces, stage, at_r, rr, cols, t, e, XBF16, r);
          else
            load_vec<G, WIDE, XBF16, true>(rr, cols, t, e, r);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) r[k] = 0.0f;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) r[k] = fmaf(rstd, fmaf(-xh[e][k], c2, g[e][k] - c1), r[k]);
        store_vec<G, WIDE>(dxr, cols, t, e, XBF16, r);
      }
    }
    if (++stage == kStages) stage = 0;
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
    // the CTA's groups add their sums one after another, where the stages were
    float* sum = reinterpret_cast<float*>(ring);
    cp_async_wait<0>();
    for (int w = 0; w < kGroups; ++w) {
      __syncthreads();
      if (grp == w) {
#pragma unroll
        for (int e = 0; e < NV; ++e)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int c = col_of<G, WIDE>(t, e, k);
            if (c < cols) {
              sum[c] = (w ? sum[c] : 0.0f) + dg[e][k];
              sum[cols + c] = (w ? sum[cols + c] : 0.0f) + db[e][k];
            }
          }
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * cols; c += T) out[c] = sum[c];
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

template <int G, int NV, bool XBF16, bool WIDE>
cudaError_t fwd_launch(const NormFwdArgs& a, bool pwide, cudaStream_t s) {
  constexpr int T = kCtaThreads<G>;
  constexpr size_t sm = WIDE ? size_t(kFwdRing<NV, XBF16>) * kFwdPieces<G, NV, XBF16> * T * 16 : 0;
  static LayerGrid cache;
  int cap = 0;
  const cudaError_t e = layer_grid(cache, reinterpret_cast<const void*>(&k_norm_fwd<G, NV, XBF16, WIDE>), T, sm, sm, &cap);
  if (e != cudaSuccess) return e;
  const int64_t want = (a.rows + T / G - 1) / (T / G);
  k_norm_fwd<G, NV, XBF16, WIDE><<<unsigned(want < cap ? want : cap), T, sm, s>>>(a, pwide);
  return cudaGetLastError();
}

template <int G, int NV>
cudaError_t fwd(const NormFwdArgs& a, bool wide, bool pwide, cudaStream_t s) {
  if (a.x_bf16) return wide ? fwd_launch<G, NV, true, true>(a, pwide, s) : fwd_launch<G, NV, true, false>(a, pwide, s);
  return wide ? fwd_launch<G, NV, false, true>(a, pwide, s) : fwd_launch<G, NV, false, false>(a, pwide, s);
}

template <int G, int NV, bool XBF16, bool WIDE, bool CKPT>
cudaError_t bwd_launch(const NormBwdArgs& a, bool pwide, int* parts, cudaStream_t s) {
  constexpr int T = kCtaThreads<G>, groups = T / G;
  const auto bytes = [](int y_bf16, bool residual) {
    // the stages, or where several groups join their sums of at most G * NV * 8 columns
    return WIDE ? size_t(kBwdStages<G, XBF16>) * bwd_pieces<NV>(y_bf16, XBF16, !CKPT, residual) * T * 16
                : size_t(groups > 1 ? G * NV * 64 : 0);
  };
  static_assert(!WIDE || groups == 1 || kBwdStages<G, XBF16> * T * 16 >= G * 64, "the sums fit where the stages were");
  const size_t sm = bytes(a.y_bf16, a.residual != nullptr);
  static LayerGrid cache[4];  // occupancy depends on the stage's size, of which there are four
  int cap = 0;
  const cudaError_t e = layer_grid(cache[(a.y_bf16 ? 1 : 0) + (a.residual != nullptr ? 2 : 0)],
                                   reinterpret_cast<const void*>(&k_norm_bwd<G, NV, XBF16, WIDE, CKPT>), T, sm,
                                   bytes(0, true), &cap);
  if (e != cudaSuccess) return e;
  if (cap > kNormPartials) cap = kNormPartials;
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
  if (pitch <= 512) return fwd<64, 1>(a, wide, pwide, s);
  if (pitch <= 1024) return fwd<128, 1>(a, wide, pwide, s);
  if (pitch <= 2048) return fwd<256, 1>(a, wide, pwide, s);
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
    else if (pitch <= 512) e = bwd<64, 1>(a, wide, pwide, &parts, s);
    else if (pitch <= 1024) e = bwd<128, 1>(a, wide, pwide, &parts, s);
    else if (pitch <= 2048) e = bwd<256, 1>(a, wide, pwide, &parts, s);
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
