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
// row into registers where they have them to spare.
//
// In the backward pass each thread keeps the sums of dgamma and dbeta of its own
// columns in registers over all its rows, one partial row per CTA goes to the
// workspace, and a second kernel adds the partial rows in order: no atomics, the
// same result every run.
//
// 16384 x 4096 bf16: forward 55 us (4.9 TB/s; 73 us with the checkpoint), bound by
// the two barriers a row with one row's work per CTA between them; backward 102 us
// (3.9 TB/s), with a residual 112 us, from a checkpoint 102 us, bound by waiting
// for each row's two sums (it issues in half of its cycles, at a quarter of the
// warps: the two CTAs a SM that its registers allow).
// Rows that take no 16-byte loads, 16384 x 2047: forward 53 us, backward 87 us.
#include <atomic>

#include "device_common.cuh"
#include "layers_common.cuh"
#include "tensor_core.cuh"

namespace loco {

namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

template <int G>
constexpr int kCtaThreads = G < 128 ? 128 : G;

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

__device__ __forceinline__ const char* at(const void* p, int64_t i, int bf16) {
  return static_cast<const char*>(p) + i * (bf16 ? 2 : 4);
}
__device__ __forceinline__ char* at(void* p, int64_t i, int bf16) { return static_cast<char*>(p) + i * (bf16 ? 2 : 4); }

// ---------------------------------------------------------------------------------------- WIDE: 16-byte pieces

// Piece i of a stage lies at stage + (i * threads + thread) * 16, so that a warp's accesses meet no
// bank twice.  A thread's addresses are kept as running pointers: with 8 columns a piece, computing
// them anew for each row took more instructions than the values themselves.
__device__ __forceinline__ Pair bits_pair(uint32_t lo, uint32_t hi) { return pair(__uint_as_float(lo), __uint_as_float(hi)); }

// Starts the copies of a thread's NV vectors of one row, G vectors apart; `row` points at its first.
template <int G, int NV, bool BF16>
__device__ __forceinline__ void copy_row(uint32_t dst, const char* row, const bool (&full)[NV]) {
  constexpr int T = kCtaThreads<G>, kBytes = BF16 ? 16 : 32;
#pragma unroll
  for (int e = 0; e < NV; ++e) {
    if (!full[e]) continue;
    copy_to_shared16(dst + e * (T * kBytes), row + e * (G * kBytes));
    if (!BF16) copy_to_shared16(dst + e * (T * kBytes) + T * 16, row + e * (G * kBytes) + 16);
  }
}
// The vector a row ends in, 0 past the end; `left` columns of it exist.  (The kernel may write a row
// that is also its residual.)
template <bool BF16>
__device__ __forceinline__ void load_last(const char* at, int left, Pair v[4]) {
  float f[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = k < left ? load_elem_rw(at, k, BF16) : 0.0f;
  pairs8(f, v);
}
// Vector e of the row copied to src; row() is its place in memory.
template <int G, int NV, bool BF16, typename Row>
__device__ __forceinline__ void copied(uint32_t src, int e, Row row, bool full, int left, Pair v[4]) {
  constexpr int T = kCtaThreads<G>, kBytes = BF16 ? 16 : 32;
  if (!full) {
    load_last<BF16>(row() + e * (G * kBytes), left, v);
  } else if (BF16) {
    widen8(shared16(src + e * (T * kBytes)), v);
  } else {
    const uint4 a = shared16(src + e * (T * kBytes)), b = shared16(src + e * (T * kBytes) + T * 16);
    v[0] = bits_pair(a.x, a.y), v[1] = bits_pair(a.z, a.w), v[2] = bits_pair(b.x, b.y), v[3] = bits_pair(b.z, b.w);
  }
}
template <bool BF16>
__device__ __forceinline__ void store_vec(char* at, bool full, int left, const Pair v[4]) {
  float f[8];
  floats8(v, f);
  if (full) {
    store8(at, 0, BF16, f);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < left) store_elem(at, k, BF16, f[k]);
  }
}
// Eight values of a parameter vector from column c0 on; `wide`: it starts on a 16-byte boundary.
__device__ __forceinline__ void load_param(const void* p, int cols, int c0, int bf16, bool wide, float none, Pair v[4]) {
  if (p != nullptr && wide && c0 + 8 <= cols) {
    if (bf16) {
      widen8(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + c0)), v);
    } else {
      float f[8];
      load8(p, c0, 0, f);
      pairs8(f, v);
    }
  } else {
    float f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = p != nullptr && c0 + k < cols ? load_elem(p, c0 + k, bf16) : none;
    pairs8(f, v);
  }
}
// 0 in the columns past the row's end, of which `left` are before it.
__device__ __forceinline__ void clear_past(Pair v[4], int left) {
  float f[8];
  floats8(v, f);
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k >= left) f[k] = 0.0f;
  pairs8(f, v);
}

// Stages: the row at work and the next ones.
constexpr int kFwdStages = 3;

// YBF16: type of y.  CTAs per SM: as many as 64 or 80 registers a thread allow.
template <int G, int NV, bool XBF16, bool YBF16>
__global__ void __launch_bounds__(kCtaThreads<G>, (NV == 1 ? 1024 : G <= 64 ? 640 : 768) / kCtaThreads<G>)
    k_norm_fwd(NormFwdArgs a, bool pwide) {
  __shared__ float red[2][32];
  extern __shared__ __align__(16) uint8_t ring[];
  constexpr int T = kCtaThreads<G>, kGroups = T / G, kX = XBF16 ? 16 : 32, kY = YBF16 ? 16 : 32;
  constexpr uint32_t kStage = NV * T * kX;
  constexpr bool kKeep = NV <= 2;  // gamma and beta stay in registers
  const int t = threadIdx.x % G, grp = threadIdx.x / G;
  const int cols = int(a.cols), nb = (cols + kCkptBlock - 1) / kCkptBlock;
  const int64_t step = int64_t(gridDim.x) * kGroups, first = int64_t(blockIdx.x) * kGroups + grp;
  bool full[NV], some[NV];
  Pair gm[NV][4], bt[NV][4];
#pragma unroll
  for (int e = 0; e < NV; ++e) {
    const int c0 = (t + G * e) * 8;
    full[e] = c0 + 8 <= cols, some[e] = c0 < cols;
    if constexpr (kKeep) {
      load_param(a.gamma, cols, c0, a.param_bf16, pwide, 1.0f, gm[e]);
      load_param(a.beta, cols, c0, a.param_bf16, pwide, 0.0f, bt[e]);
    }
  }
  const float inv_cols = 1.0f / float(cols);
  const int64_t x_step = step * a.ldx * (XBF16 ? 2 : 4), y_step = step * a.ldy * (YBF16 ? 2 : 4);
  const char* xp = at(a.x, first * a.ldx, XBF16) + t * kX;  // the row at work
  const char* xa = xp;                                      // the next to be copied
  char* yp = at(a.y, first * a.ldy, YBF16) + t * kY;
  const uint32_t base = smem_addr(ring) + threadIdx.x * 16, end = base + kFwdStages * kStage;
  uint32_t cur = base, nxt = base;
  int64_t ahead = first;
  const auto copy_next = [&]() {
    if (ahead < a.rows) copy_row<G, NV, XBF16>(nxt, xa, full);
    cp_async_commit();
    ahead += step, xa += x_step;
    if ((nxt += kStage) == end) nxt = base;
  };
#pragma unroll
  for (int i = 0; i < kFwdStages - 1; ++i) copy_next();
  int turn = 0;
  // the CTA's groups go through the loop together
  for (int64_t row = first; row - grp < a.rows; row += step, xp += x_step, yp += y_step) {
    const bool live = row < a.rows;
    copy_next();
    cp_async_wait<kFwdStages - 1>();
    Pair x[NV][4];
#pragma unroll
    for (int e = 0; e < NV; ++e) {
      if (some[e] && live) {
        copied<G, NV, XBF16>(cur, e, [&] { return xp; }, full[e], cols - (t + G * e) * 8, x[e]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) x[e][k] = pair(0.0f, 0.0f);
      }
    }
    if ((cur += kStage) == end) cur = base;
    float mean = 0.0f;
    if (!a.rms) {
      Pair s2 = x[0][0] + x[0][1], s3 = x[0][2] + x[0][3];
#pragma unroll
      for (int e = 1; e < NV; ++e) s2 = s2 + (x[e][0] + x[e][1]), s3 = s3 + (x[e][2] + x[e][3]);
      const float2 h = halves(s2 + s3);
      float s[1] = {h.x + h.y};
      group_sum<G>(s, red[turn]);
      turn ^= 1;
      mean = s[0] * inv_cols;
      const Pair less = pair(-mean, -mean);
#pragma unroll
      for (int e = 0; e < NV; ++e) {
        if (!some[e]) continue;
#pragma unroll
        for (int k = 0; k < 4; ++k) x[e][k] = x[e][k] + less;
        if (!full[e]) clear_past(x[e], cols - (t + G * e) * 8);
      }
    }
    Pair q2 = x[0][0] * x[0][0], q3 = x[0][1] * x[0][1];
    q2 = fma(x[0][2], x[0][2], q2), q3 = fma(x[0][3], x[0][3], q3);
#pragma unroll
    for (int e = 1; e < NV; ++e) {
      q2 = fma(x[e][0], x[e][0], q2), q3 = fma(x[e][1], x[e][1], q3);
      q2 = fma(x[e][2], x[e][2], q2), q3 = fma(x[e][3], x[e][3], q3);
    }
    const float2 h = halves(q2 + q3);
    float q[1] = {h.x + h.y};
    group_sum<G>(q, red[turn]);
    turn ^= 1;
    const float rstd = rsqrtf(fmaf(q[0], inv_cols, a.eps));
    if (t == 0 && live) {
      if (a.mean != nullptr && !a.rms) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    if (!live) continue;  // whole warps
    const Pair r2 = pair(rstd, rstd);
#pragma unroll
    for (int e = 0; e < NV; ++e) {
#pragma unroll
      for (int k = 0; k < 4; ++k) x[e][k] = x[e][k] * r2;
    }
    if (a.codes != nullptr) {
      int8_t* codes = a.codes + row * nb * kCkptBlock + t * 8;
      uint8_t* scales = a.scales + row * nb + t / 4;
#pragma unroll
      for (int e = 0; e < NV; ++e) {
        // a block is four lanes, whether or not the row reaches all of them
        float f[8];
        floats8(x[e], f);
        const uint32_t m = block_magnitude(f);
        if ((t + G * e) / 4 < nb) {
          *reinterpret_cast<uint2*>(codes + e * (G * 8)) = ckpt_pack8(f, m);
          if ((t & 3) == 0) scales[e * (G / 4)] = uint8_t(ckpt_scale(m));
        }
      }
    }
#pragma unroll
    for (int e = 0; e < NV; ++e) {
      if (!some[e]) continue;
      if constexpr (kKeep) {
#pragma unroll
        for (int k = 0; k < 4; ++k) x[e][k] = fma(x[e][k], gm[e][k], bt[e][k]);
      } else {
        Pair g[4], b[4];
        load_param(a.gamma, cols, (t + G * e) * 8, a.param_bf16, pwide, 1.0f, g);
        load_param(a.beta, cols, (t + G * e) * 8, a.param_bf16, pwide, 0.0f, b);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[e][k] = fma(x[e][k], g[k], b[k]);
      }
      store_vec<YBF16>(yp + e * (G * kY), full[e], cols - (t + G * e) * 8, x[e]);
    }
  }
}

// ---------------------------------------------------------------------------------------- narrow: single columns

// Column j of a thread: t + G * j.  Neighbouring lanes hold neighbouring columns, so that loads and
// stores of single elements still touch whole sectors, and a checkpoint block is one warp.
template <bool BF16>
struct Elem {
  typedef float type;
};
template <>
struct Elem<true> {
  typedef uint16_t type;
};
__device__ __forceinline__ float elem_value(float v) { return v; }
__device__ __forceinline__ float elem_value(uint16_t v) { return bf16_bits_to_f32(v); }

// A row's columns as they lie in memory, so that a row ahead takes few registers and no conversions.
// RW: the kernel may write this row later.
template <int G, int NE, bool BF16, bool RW>
__device__ __forceinline__ void fetch_cols(const char* row, int cols, int t, typename Elem<BF16>::type (&v)[NE]) {
  const typename Elem<BF16>::type* q = reinterpret_cast<const typename Elem<BF16>::type*>(row) + t;
#pragma unroll
  for (int j = 0; j < NE; ++j) v[j] = t < cols - G * j ? (RW ? q[G * j] : __ldg(q + G * j)) : typename Elem<BF16>::type(0);
}
template <int G, int NE, bool BF16>
__device__ __forceinline__ void load_cols(const char* row, int cols, int t, float (&v)[NE]) {
  typename Elem<BF16>::type raw[NE];
  fetch_cols<G, NE, BF16, false>(row, cols, t, raw);
#pragma unroll
  for (int j = 0; j < NE; ++j) v[j] = elem_value(raw[j]);
}
template <int G, int NE>
__device__ __forceinline__ void load_cols(const void* p, int cols, int t, int bf16, float none, float (&v)[NE]) {
  if (p == nullptr) {
#pragma unroll
    for (int j = 0; j < NE; ++j) v[j] = none;
  } else if (bf16) {
    load_cols<G, NE, true>(static_cast<const char*>(p), cols, t, v);
  } else {
    load_cols<G, NE, false>(static_cast<const char*>(p), cols, t, v);
  }
}
template <int G, int NE>
__device__ __forceinline__ void store_cols(char* row, int cols, int t, int bf16, const float (&v)[NE]) {
  if (bf16) {
    __nv_bfloat16* q = reinterpret_cast<__nv_bfloat16*>(row) + t;
#pragma unroll
    for (int j = 0; j < NE; ++j)
      if (t < cols - G * j) q[G * j] = __float2bfloat16_rn(v[j]);
  } else {
    float* q = reinterpret_cast<float*>(row) + t;
#pragma unroll
    for (int j = 0; j < NE; ++j)
      if (t < cols - G * j) q[G * j] = v[j];
  }
}

template <int G, int NE, bool XBF16>
__global__ void __launch_bounds__(kCtaThreads<G>, (G == 512 ? 1024 : 768) / kCtaThreads<G>) k_norm_fwd_narrow(NormFwdArgs a) {
  __shared__ float red[2][32];
  constexpr int kGroups = kCtaThreads<G> / G;
  const int t = threadIdx.x % G, grp = threadIdx.x / G;
  const int cols = int(a.cols), nb = (cols + kCkptBlock - 1) / kCkptBlock;
  const int64_t step = int64_t(gridDim.x) * kGroups;
  int turn = 0;
  typename Elem<XBF16>::type next[NE];
  const auto fetch = [&](int64_t row) {
    fetch_cols<G, NE, XBF16, false>(at(a.x, row * a.ldx, XBF16), row < a.rows ? cols : 0, t, next);
  };
  const int64_t first = int64_t(blockIdx.x) * kGroups + grp;
  constexpr bool kAhead = NE <= 8;  // more columns a thread leave no registers for a row ahead
  if (kAhead) fetch(first);
  for (int64_t row = first; row - grp < a.rows; row += step) {
    const bool live = row < a.rows;
    float x[NE];
    if (!kAhead) fetch(row);
#pragma unroll
    for (int j = 0; j < NE; ++j) x[j] = elem_value(next[j]);
    if (kAhead) fetch(row + step);
    float mean = 0.0f;
    if (!a.rms) {
      float s[1] = {0.0f}, s1 = 0.0f;
#pragma unroll
      for (int j = 0; j < NE; j += 2) s[0] += x[j], s1 += x[j + 1];
      s[0] += s1;
      group_sum<G>(s, red[turn]);
      turn ^= 1;
      mean = s[0] / float(cols);
    }
    float q[1] = {0.0f}, q1 = 0.0f;
#pragma unroll
    for (int j = 0; j < NE; j += 2) {
      x[j] = t < cols - G * j ? x[j] - mean : 0.0f;
      x[j + 1] = t < cols - G * (j + 1) ? x[j + 1] - mean : 0.0f;
      q[0] = fmaf(x[j], x[j], q[0]);
      q1 = fmaf(x[j + 1], x[j + 1], q1);
    }
    q[0] += q1;
    group_sum<G>(q, red[turn]);
    turn ^= 1;
    const float rstd = rsqrtf(q[0] / float(cols) + a.eps);
    if (t == 0 && live) {
      if (a.mean != nullptr && !a.rms) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    if (!live) continue;  // whole warps
#pragma unroll
    for (int j = 0; j < NE; ++j) x[j] *= rstd;
    if (a.codes != nullptr) {
      int8_t* c = a.codes + row * nb * kCkptBlock + t;
      uint8_t* sc = a.scales + row * nb + t / kCkptBlock;
#pragma unroll
      for (int j = 0; j < NE; ++j) {
        if (t / kCkptBlock >= nb - G / kCkptBlock * j) continue;  // a warp's 32 columns are one block
        const uint32_t s = ckpt_scale(__reduce_max_sync(0xFFFFFFFFu, mag_bits(x[j])));
        c[G * j] = int8_t(ckpt_code(x[j], ckpt_inv_step(s)));
        if ((t & 31) == 0) sc[G / kCkptBlock * j] = uint8_t(s);
      }
    }
    if (a.gamma != nullptr) {
      float g[NE];
      load_cols<G, NE>(a.gamma, cols, t, a.param_bf16, 1.0f, g);
#pragma unroll
      for (int j = 0; j < NE; ++j) x[j] *= g[j];
    }
    if (a.beta != nullptr) {
      float b[NE];
      load_cols<G, NE>(a.beta, cols, t, a.param_bf16, 0.0f, b);
#pragma unroll
      for (int j = 0; j < NE; ++j) x[j] += b[j];
    }
    store_cols<G, NE>(at(a.y, row * a.ldy, a.y_bf16), cols, t, a.y_bf16, x);
  }
}

// Rows too long for the registers of a CTA: three passes over the row, which the L2 cache serves
// after the first.
constexpr int kLoop = 512;

template <bool XBF16>
__global__ void __launch_bounds__(kLoop) k_norm_fwd_long(NormFwdArgs a) {
  __shared__ float red[2][32];
  const int64_t row = blockIdx.x, cols = a.cols, nb = (cols + kCkptBlock - 1) / kCkptBlock;
  const char* xr = at(a.x, row * a.ldx, XBF16);
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
  const float rstd = rsqrtf(q[0] / float(cols) + a.eps);
  if (threadIdx.x == 0) {
    if (a.mean != nullptr && !a.rms) a.mean[row] = mean;
    if (a.rstd != nullptr) a.rstd[row] = rstd;
  }
  char* yr = at(a.y, row * a.ldy, a.y_bf16);
  const int64_t pitch = nb * kCkptBlock;  // a multiple of 32: whole warps enter and leave together
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

// Rows of more columns than the registers of a CTA hold the sums of go to a cluster of two CTAs, 8192
// columns to the first and the rest to the second (16-byte boundaries and whole blocks of a checkpoint).
// Each sees its columns as a matrix of its own; the sums of a row are exchanged.  4096 x 16384 bf16 takes
// 152 us so, against 718 us in three passes over memory (the sums, dx, the columns' sums).
constexpr int kHalf = 8192;
__device__ __forceinline__ void own_half(NormBwdArgs& a, bool xbf16, int rank) {
  const int64_t c = int64_t(rank) * kHalf;
  const auto shift = [&](const void* p, int bf16) { return p == nullptr ? p : at(p, c, bf16); };
  a.dy = shift(a.dy, a.y_bf16);
  a.x = shift(a.x, xbf16);
  a.gamma = shift(a.gamma, a.param_bf16);
  a.residual = shift(a.residual, xbf16);
  a.dx = const_cast<void*>(shift(a.dx, xbf16));
  if (a.codes != nullptr) a.codes += c, a.scales += c / kCkptBlock;
  if (a.partials != nullptr) a.partials += c;
}
// The sums of both CTAs, in their order; consecutive calls alternate between two places.
__device__ __forceinline__ void cluster_sum(float (&s)[2], float (*place)[2], int turn) {
  if (threadIdx.x == 0) place[turn][0] = s[0], place[turn][1] = s[1];
  cluster_sync();
  const uint32_t p = smem_u32(place[turn]);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    s[i] = cluster_load(cluster_addr(p + 4 * i, 0)) + cluster_load(cluster_addr(p + 4 * i, 1));
}

// Partial sums of a CTA's rows to the workspace.  `mine(c, i)` gives a thread's sum i (0 dgamma, 1
// dbeta) of its columns through `each`; where a CTA holds several groups they add up one after another
// in shared memory first.
template <int G, typename Each>
__device__ __forceinline__ void write_partials(const NormBwdArgs& a, int64_t part, float* sum, Each each) {
  constexpr int T = kCtaThreads<G>, kGroups = T / G;
  const int cols = int(a.cols), grp = threadIdx.x / G;
  float* out = a.partials + part * 2 * cols;
  if constexpr (kGroups == 1) {
    each([&](int c, float dg, float db) { out[c] = dg, out[cols + c] = db; });
  } else {
    for (int w = 0; w < kGroups; ++w) {
      __syncthreads();
      if (grp == w)
        each([&](int c, float dg, float db) {
          sum[c] = (w ? sum[c] : 0.0f) + dg;
          sum[cols + c] = (w ? sum[cols + c] : 0.0f) + db;
        });
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * cols; c += T) out[c] = sum[c];
  }
}

// As many rows ahead as shared memory holds for the widest types (a row of 8192 fp32 columns with
// fp32 dy and residual takes 96 KB).
template <int G, bool XBF16, bool YBF16>
constexpr int kBwdStages = G == 512 && !(XBF16 && YBF16) ? 2 : 3;

template <int G, int NV, bool XBF16, bool YBF16, bool CKPT, bool PAIR = false>
__global__ void __launch_bounds__(kCtaThreads<G>, G == 512 ? 1 : G < 128 ? 5 : (NV == 1 ? 768 : 512) / kCtaThreads<G>)
    k_norm_bwd(NormBwdArgs a, bool pwide) {
  __shared__ float red[2][64];
  __shared__ float halves_sum[2][2];
  extern __shared__ __align__(16) uint8_t ring[];  // the stages, and gamma; after the rows, [2][cols] sums
  constexpr int T = kCtaThreads<G>, kGroups = T / G, kStages = kBwdStages<G, XBF16, YBF16>;
  constexpr int kX = XBF16 ? 16 : 32, kY = YBF16 ? 16 : 32;
  constexpr uint32_t at_x = NV * T * kY, at_r = at_x + NV * T * (CKPT ? 16 : kX);
  const int t = threadIdx.x % G, grp = threadIdx.x / G;
  const int nb = int((a.cols + kCkptBlock - 1) / kCkptBlock), rank = PAIR ? int(cluster_rank()) : 0;
  const int cols = PAIR ? (rank ? int(a.cols) - kHalf : kHalf) : int(a.cols);  // this CTA's
  const int64_t block = PAIR ? blockIdx.x / 2 : blockIdx.x, blocks = PAIR ? gridDim.x / 2 : gridDim.x;
  const int64_t step = blocks * kGroups, first = block * kGroups + grp;
  if constexpr (PAIR) own_half(a, XBF16, rank);
  const bool with_r = a.residual != nullptr;
  const uint32_t stage_bytes = at_r + (with_r ? NV * T * kX : 0);
  const uint32_t base = smem_addr(ring) + threadIdx.x * 16, end = base + kStages * stage_bytes;
  const uint32_t gamma = end;  // each thread's own values behind the stages
  bool full[NV], some[NV];
  Pair dg[NV][4], db[NV][4];
#pragma unroll
  for (int e = 0; e < NV; ++e) {
    const int c0 = (t + G * e) * 8;
    full[e] = c0 + 8 <= cols, some[e] = c0 < cols;
    Pair v[4];
    load_param(a.gamma, cols, c0, a.param_bf16, pwide, 1.0f, v);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 lo = halves(v[2 * i]), hi = halves(v[2 * i + 1]);
      to_shared16(gamma + (2 * e + i) * T * 16, make_uint4(__float_as_uint(lo.x), __float_as_uint(lo.y),
                                                           __float_as_uint(hi.x), __float_as_uint(hi.y)));
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) dg[e][k] = db[e][k] = pair(0.0f, 0.0f);
  }
  const float inv_cols = 1.0f / float(int(a.cols));
  // the thread's place in a row of each matrix
  const auto dy_at = [&](int64_t row) { return at(a.dy, row * a.lddy, YBF16) + t * kY; };
  const auto x_at = [&](int64_t row) { return at(a.x, row * a.ldx, XBF16) + t * kX; };
  const auto r_at = [&](int64_t row) { return at(a.residual, row * a.ldr, XBF16) + t * kX; };
  uint32_t cur = base;
  const auto copy_next = [&](int64_t ahead, uint32_t nxt) {
    if (ahead < a.rows) {
      copy_row<G, NV, YBF16>(nxt, dy_at(ahead), full);
      if constexpr (CKPT) {
        const int8_t* codes = a.codes + ahead * nb * kCkptBlock + t * 8;
#pragma unroll
        for (int e = 0; e < NV; ++e)  // the padding of a ragged block is part of it
          if (some[e]) copy_to_shared8(nxt + at_x + e * (T * 16), codes + e * (G * 8));
      } else {
        copy_row<G, NV, XBF16>(nxt + at_x, x_at(ahead), full);
      }
      if (with_r) copy_row<G, NV, XBF16>(nxt + at_r, r_at(ahead), full);
    }
    cp_async_commit();
  };
  // What of the next row goes to registers: its statistics and scales.
  float next_rstd = 0.0f, next_mean = 0.0f;
  uint32_t next_scale[NV];
  const auto load = [&](int64_t row) {
    next_rstd = __ldg(a.rstd + row);
    if (!CKPT && !a.rms) next_mean = __ldg(a.mean + row);
    if constexpr (CKPT) {
#pragma unroll
      for (int e = 0; e < NV; ++e) next_scale[e] = some[e] ? __ldg(a.scales + row * nb + (t + G * e) / 4) : 1u;
    }
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) copy_next(first + i * step, base + i * stage_bytes);
  if (first < a.rows) load(first);
  int turn = 0;
  for (int64_t row = first; row - grp < a.rows; row += step) {
    const bool live = row < a.rows;
    copy_next(row + (kStages - 1) * step, (cur == base ? end : cur) - stage_bytes);
    cp_async_wait<kStages - 1>();
    const float rstd = next_rstd;
    const Pair r2 = pair(rstd, rstd), less = pair(-next_mean, -next_mean);
    uint32_t scale[NV];
    if constexpr (CKPT) {
#pragma unroll
      for (int e = 0; e < NV; ++e) scale[e] = next_scale[e];
    }
    // dy, the normalised values and gamma of vector e, read from shared memory before and after the sums
    const auto values = [&](int e, Pair (&d)[4], Pair (&xh)[4], Pair (&gm)[4]) {
      const int left = cols - (t + G * e) * 8;
      copied<G, NV, YBF16>(cur, e, [&] { return dy_at(row); }, full[e], left, d);
      if constexpr (CKPT) {
        const uint2 w = shared8(cur + at_x + e * (T * 16));
        ckpt_pairs4(w.x, scale[e], xh);
        ckpt_pairs4(w.y, scale[e], xh + 2);
      } else {
        copied<G, NV, XBF16>(cur + at_x, e, [&] { return x_at(row); }, full[e], left, xh);
#pragma unroll
        for (int k = 0; k < 4; ++k) xh[k] = (xh[k] + less) * r2;  // nearly exact; x r - m r rounds m r, for the whole row alike
      }
      if (!full[e]) clear_past(xh, left);  // (a bad block's padding reads back as NaN)
      const uint4 lo = shared16(gamma + 2 * e * T * 16), hi = shared16(gamma + (2 * e + 1) * T * 16);
      gm[0] = bits_pair(lo.x, lo.y), gm[1] = bits_pair(lo.z, lo.w);
      gm[2] = bits_pair(hi.x, hi.y), gm[3] = bits_pair(hi.z, hi.w);
    };
    float s[2] = {0.0f, 0.0f};
    if (live) {
      Pair s0 = pair(0.0f, 0.0f), s1 = s0;
#pragma unroll
      for (int e = 0; e < NV; ++e) {
        if (!some[e]) continue;
        Pair d[4], xh[4], gm[4];
        values(e, d, xh, gm);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          dg[e][k] = fma(d[k], xh[k], dg[e][k]);
          db[e][k] = db[e][k] + d[k];
          const Pair g = d[k] * gm[k];
          s0 = s0 + g;
          s1 = fma(g, xh[k], s1);
        }
      }
      const float2 h0 = halves(s0), h1 = halves(s1);
      s[0] = h0.x + h0.y, s[1] = h1.x + h1.y;
    }
    if (row + step < a.rows) load(row + step);
    group_sum<G>(s, red[turn]);
    if constexpr (PAIR) cluster_sum(s, halves_sum, turn);
    turn ^= 1;
    if (live) {
      char* op = at(a.dx, row * a.lddx, XBF16) + t * kX;
      // dx = r (g - c1 - xhat c2) + residual
      const float c1 = a.rms ? 0.0f : s[0] * inv_cols * -rstd, c2 = s[1] * inv_cols * -rstd;
      const Pair k1 = pair(c1, c1), k2 = pair(c2, c2);
#pragma unroll
      for (int e = 0; e < NV; ++e) {
        if (!some[e]) continue;
        Pair d[4], xh[4], gm[4], r[4];
        values(e, d, xh, gm);
#pragma unroll
        for (int k = 0; k < 4; ++k) d[k] = fma(xh[k], k2, fma(d[k] * gm[k], r2, k1));
        if (with_r) {
          copied<G, NV, XBF16>(cur + at_r, e, [&] { return r_at(row); }, full[e], cols - (t + G * e) * 8, r);
#pragma unroll
          for (int k = 0; k < 4; ++k) d[k] = d[k] + r[k];
        }
        store_vec<XBF16>(op + e * (G * kX), full[e], cols - (t + G * e) * 8, d);
      }
    }
    if ((cur += stage_bytes) == end) cur = base;
  }
  if constexpr (PAIR) cluster_sync();  // the other has read this one's last sums
  if (a.partials == nullptr) return;
  cp_async_wait<0>();
  write_partials<G>(a, block, reinterpret_cast<float*>(ring), [&](auto put) {
#pragma unroll
    for (int e = 0; e < NV; ++e)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 g = halves(dg[e][k]), b = halves(db[e][k]);
        const int c = (t + G * e) * 8 + 2 * k;
        if (c < cols) put(c, g.x, b.x);
        if (c + 1 < cols) put(c + 1, g.y, b.y);
      }
  });
}

template <int G, int NE, bool XBF16, bool YBF16, bool CKPT, bool PAIR = false>
__global__ void __launch_bounds__(kCtaThreads<G>, (G >= 1024 ? 1024 : 512) / kCtaThreads<G>) k_norm_bwd_narrow(NormBwdArgs a) {
  __shared__ float red[2][64];
  __shared__ float halves_sum[2][2];
  extern __shared__ float sums[];  // [2][cols] where a CTA holds several groups
  constexpr int kGroups = kCtaThreads<G> / G;
  const int t = threadIdx.x % G, grp = threadIdx.x / G;
  const int nb = int((a.cols + kCkptBlock - 1) / kCkptBlock), rank = PAIR ? int(cluster_rank()) : 0;
  const int cols = PAIR ? (rank ? int(a.cols) - kHalf : kHalf) : int(a.cols);  // this CTA's
  const int64_t block = PAIR ? blockIdx.x / 2 : blockIdx.x, blocks = PAIR ? gridDim.x / 2 : gridDim.x;
  const int64_t step = blocks * kGroups;
  if constexpr (PAIR) own_half(a, XBF16, rank);
  constexpr bool kAhead = G < 1024;  // 1024 threads leave no registers for a row ahead
  float dg[NE], db[NE];
#pragma unroll
  for (int j = 0; j < NE; ++j) dg[j] = db[j] = 0.0f;
  int turn = 0;
  typename Elem<YBF16>::type next_d[NE];
  typename Elem<XBF16>::type next_x[NE];
  uint32_t next_c[NE];  // a code and its scale
  const auto fetch = [&](int64_t row) {
    const int n = row < a.rows ? cols : 0;
    fetch_cols<G, NE, YBF16, false>(at(a.dy, row * a.lddy, YBF16), n, t, next_d);
    if constexpr (CKPT) {
      const int8_t* c = a.codes + row * nb * kCkptBlock + t;
      const uint8_t* sc = a.scales + row * nb + t / kCkptBlock;
#pragma unroll
      for (int j = 0; j < NE; ++j)
        next_c[j] = t < n - G * j ? uint32_t(uint8_t(__ldg(c + G * j))) | uint32_t(__ldg(sc + G / kCkptBlock * j)) << 8 : 0u;
    } else {
      fetch_cols<G, NE, XBF16, false>(at(a.x, row * a.ldx, XBF16), n, t, next_x);
    }
  };
  const int64_t first = block * kGroups + grp;
  if (kAhead) fetch(first);
  for (int64_t row = first; row - grp < a.rows; row += step) {
    const bool live = row < a.rows;
    float d[NE], xh[NE], s[2] = {0.0f, 0.0f}, rstd = 0.0f;
    if (!kAhead) fetch(row);
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      d[j] = elem_value(next_d[j]);
      xh[j] = CKPT ? float(int8_t(next_c[j])) * ckpt_step(next_c[j] >> 8) : elem_value(next_x[j]);
    }
    if (kAhead) fetch(row + step);
    typename Elem<XBF16>::type r[kAhead ? NE : 1];
    if constexpr (kAhead)
      if (a.residual != nullptr)
        fetch_cols<G, NE, XBF16, true>(at(a.residual, row * a.ldr, XBF16), live ? cols : 0, t, r);
    if (live) {
      rstd = __ldg(a.rstd + row);
      if constexpr (!CKPT) {
        const float mean = a.rms ? 0.0f : __ldg(a.mean + row);
#pragma unroll
        for (int j = 0; j < NE; ++j) xh[j] = t < cols - G * j ? (xh[j] - mean) * rstd : 0.0f;
      }
      float gm[NE];
      load_cols<G, NE>(a.gamma, cols, t, a.param_bf16, 1.0f, gm);
#pragma unroll
      for (int j = 0; j < NE; ++j) {
        dg[j] = fmaf(d[j], xh[j], dg[j]);
        db[j] += d[j];
        d[j] *= gm[j];
        s[0] += d[j];
        s[1] = fmaf(d[j], xh[j], s[1]);
      }
    }
    group_sum<G>(s, red[turn]);
    if constexpr (PAIR) cluster_sum(s, halves_sum, turn);
    turn ^= 1;
    if (!live) continue;  // whole warps
    const float c1 = a.rms ? 0.0f : s[0] / float(int(a.cols)), c2 = s[1] / float(int(a.cols));
    if (a.residual != nullptr) {
#pragma unroll
      for (int j = 0; j < NE; ++j) {
        float v = 0.0f;
        if constexpr (kAhead) {
          v = elem_value(r[j]);
        } else if (t < cols - G * j) {
          v = load_elem_rw(at(a.residual, row * a.ldr, XBF16), t + G * j, XBF16);
        }
        d[j] = fmaf(rstd, fmaf(-xh[j], c2, d[j] - c1), v);
      }
    } else {
#pragma unroll
      for (int j = 0; j < NE; ++j) d[j] = rstd * fmaf(-xh[j], c2, d[j] - c1);
    }
    store_cols<G, NE>(at(a.dx, row * a.lddx, XBF16), cols, t, XBF16, d);
  }
  if constexpr (PAIR) cluster_sync();  // the other has read this one's last sums
  if (a.partials == nullptr) return;
  write_partials<G>(a, block, sums, [&](auto put) {
#pragma unroll
    for (int j = 0; j < NE; ++j)
      if (t < cols - G * j) put(t + G * j, dg[j], db[j]);
  });
}

// Rows too long for registers: eight columns a thread at a time, the sums of a row in one kernel (which
// the L2 cache serves its second pass), those of the columns in another.

// Columns c to c + 7 of one row, 0 past its end: 16-byte loads, put together from two where they have to be.
template <bool BF16>
__device__ __forceinline__ void load_eight(const void* p, int64_t ld, int64_t rows, int64_t cols, int64_t row, int64_t c,
                                           float v[8]) {
  const char* lo = static_cast<const char*>(p);
  if (c + 8 <= cols) {
    load8_any<BF16>(at(p, row * ld + c, BF16), lo, at(p, (rows - 1) * ld + cols, BF16), v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = c + k < cols ? load_elem(p, row * ld + c + k, BF16) : 0.0f;
  }
}
// dy and the normalised values of eight columns.
template <bool XBF16>
__device__ __forceinline__ void long_values(const NormBwdArgs& a, int64_t row, int64_t c, int64_t nb, float mean, float rstd,
                                            float (&d)[8], float (&xh)[8]) {
  if (a.y_bf16)
    load_eight<true>(a.dy, a.lddy, a.rows, a.cols, row, c, d);
  else
    load_eight<false>(a.dy, a.lddy, a.rows, a.cols, row, c, d);
  if (a.x != nullptr) {
    load_eight<XBF16>(a.x, a.ldx, a.rows, a.cols, row, c, xh);
#pragma unroll
    for (int k = 0; k < 8; ++k) xh[k] = (xh[k] - mean) * rstd;
  } else {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(a.codes + row * nb * kCkptBlock + c));
    const float step = ckpt_step(__ldg(a.scales + row * nb + c / kCkptBlock));
    ckpt_unpack4(w.x, step, xh);
    ckpt_unpack4(w.y, step, xh + 4);
  }
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (c + k >= a.cols) xh[k] = 0.0f;  // (a bad block's padding reads back as NaN)
}
__device__ __forceinline__ void load_gamma(const NormBwdArgs& a, int64_t c, float (&g)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) g[k] = a.gamma != nullptr && c + k < a.cols ? load_elem(a.gamma, c + k, a.param_bf16) : 1.0f;
}

// wide: rows of dx and of the residual start on 16-byte boundaries.
template <bool XBF16>
__global__ void __launch_bounds__(kLoop, 1) k_norm_bwd_long(NormBwdArgs a, bool wide) {
  __shared__ float red[64];
  const int64_t row = blockIdx.x, cols = a.cols, nb = (cols + kCkptBlock - 1) / kCkptBlock;
  const float rstd = a.rstd[row], mean = a.x == nullptr || a.rms ? 0.0f : a.mean[row];
  float s[2] = {0.0f, 0.0f};
#pragma unroll 2
  for (int64_t c = threadIdx.x * 8; c < cols; c += kLoop * 8) {
    float d[8], xh[8], g[8];
    long_values<XBF16>(a, row, c, nb, mean, rstd, d, xh);
    load_gamma(a, c, g);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      d[k] *= g[k];
      s[0] += d[k];
      s[1] = fmaf(d[k], xh[k], s[1]);
    }
  }
  group_sum<kLoop>(s, red);
  const float c1 = a.rms ? 0.0f : s[0] / float(cols), c2 = s[1] / float(cols);
#pragma unroll 2
  for (int64_t c = threadIdx.x * 8; c < cols; c += kLoop * 8) {
    float d[8], xh[8], g[8];
    long_values<XBF16>(a, row, c, nb, mean, rstd, d, xh);
    load_gamma(a, c, g);
#pragma unroll
    for (int k = 0; k < 8; ++k) d[k] = rstd * fmaf(-xh[k], c2, d[k] * g[k] - c1);
    const bool full = wide && c + 8 <= cols;
    if (a.residual != nullptr) {
      if (full) {
        load8<true>(a.residual, row * a.ldr + c, XBF16, g);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) g[k] = c + k < cols ? load_elem_rw(a.residual, row * a.ldr + c + k, XBF16) : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) d[k] += g[k];
    }
    if (full) {
      store8(a.dx, row * a.lddx + c, XBF16, d);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c + k < cols) store_elem(a.dx, row * a.lddx + c + k, XBF16, d[k]);
    }
  }
}

// Column sums of a slice of rows: 256 columns per CTA, a warp every eighth row.
constexpr int kColWarps = 8, kColStrip = 256;
template <bool XBF16>
__global__ void __launch_bounds__(kColWarps * 32) k_norm_bwd_cols(NormBwdArgs a, int64_t rows_per) {
  __shared__ float sm[2][kColWarps][kColStrip];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int64_t c = int64_t(blockIdx.x) * kColStrip + lane * 8, nb = (a.cols + kCkptBlock - 1) / kCkptBlock;
  const int64_t lo = int64_t(blockIdx.y) * rows_per, hi = min(lo + rows_per, a.rows);
  float dg[8], db[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) dg[k] = db[k] = 0.0f;
  if (c < a.cols) {
#pragma unroll 2
    for (int64_t row = lo + warp; row < hi; row += kColWarps) {
      float d[8], xh[8];
      long_values<XBF16>(a, row, c, nb, a.x == nullptr || a.rms ? 0.0f : __ldg(a.mean + row), __ldg(a.rstd + row), d, xh);
#pragma unroll
      for (int k = 0; k < 8; ++k) dg[k] = fmaf(d[k], xh[k], dg[k]), db[k] += d[k];
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) sm[0][warp][k * 32 + lane] = dg[k], sm[1][warp][k * 32 + lane] = db[k];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t col = int64_t(blockIdx.x) * kColStrip + lane * 8 + warp;
    if (col >= a.cols) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kColWarps; ++w) v += sm[i][w][threadIdx.x];
    a.partials[(int64_t(blockIdx.y) * 2 + i) * a.cols + col] = v;
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

void pair_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, int pairs, int threads, size_t smem, cudaStream_t s) {
  cfg->gridDim = dim3(unsigned(pairs) * 2);
  cfg->blockDim = dim3(unsigned(threads));
  cfg->dynamicSmemBytes = smem;
  cfg->stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg->attrs = attr;
  cfg->numAttrs = 1;
}
// Clusters of two CTAs that the current device holds at once, at most kNormPartials.  (The kernel's limit
// of shared memory has been set by layer_grid.)
template <typename Kernel>
cudaError_t pair_slots(LayerGrid& cache, Kernel kernel, int threads, size_t smem, int* slots) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < LayerGrid::kDevices && (*slots = cache.cap[dev].load(std::memory_order_acquire)) > 0) return cudaSuccess;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  pair_config(&cfg, attr, kNormPartials, threads, smem, nullptr);
  if ((e = cudaOccupancyMaxActiveClusters(slots, kernel, &cfg)) != cudaSuccess) return e;
  if (*slots < 1) return cudaErrorInvalidConfiguration;
  if (*slots > kNormPartials) *slots = kNormPartials;
  if (dev < LayerGrid::kDevices) cache.cap[dev].store(*slots, std::memory_order_release);
  return cudaSuccess;
}

// Narrow kernels hold half as many columns a thread, in groups of twice the threads.
template <int G, int NV, bool XBF16, bool YBF16>
cudaError_t fwd_launch(const NormFwdArgs& a, bool wide, bool pwide, cudaStream_t s) {
  static LayerGrid cache[2];
  constexpr int H = NV == 1 ? G : 2 * G, NE = NV == 1 ? 8 : NV * 4;
  const int T = wide ? kCtaThreads<G> : kCtaThreads<H>, groups = T / (wide ? G : H);
  const auto wide_kernel = k_norm_fwd<G, NV, XBF16, YBF16>;
  const auto narrow_kernel = k_norm_fwd_narrow<H, NE, XBF16>;
  const size_t sm = wide ? size_t(kFwdStages) * NV * kCtaThreads<G> * (XBF16 ? 16 : 32) : 0;
  int cap = 0;
  const cudaError_t e = wide ? layer_grid(cache[0], reinterpret_cast<const void*>(wide_kernel), T, sm, sm, &cap)
                             : layer_grid(cache[1], reinterpret_cast<const void*>(narrow_kernel), T, sm, sm, &cap);
  if (e != cudaSuccess) return e;
  const int64_t want = (a.rows + groups - 1) / groups;
  const unsigned grid = unsigned(want < cap ? want : cap);
  if (wide)
    wide_kernel<<<grid, T, sm, s>>>(a, pwide);
  else
    narrow_kernel<<<grid, T, 0, s>>>(a);
  return cudaGetLastError();
}

template <int G, int NV>
cudaError_t fwd(const NormFwdArgs& a, bool wide, bool pwide, cudaStream_t s) {
  if (a.x_bf16)
    return a.y_bf16 ? fwd_launch<G, NV, true, true>(a, wide, pwide, s) : fwd_launch<G, NV, true, false>(a, wide, pwide, s);
  return a.y_bf16 ? fwd_launch<G, NV, false, true>(a, wide, pwide, s) : fwd_launch<G, NV, false, false>(a, wide, pwide, s);
}

template <typename Kernel, typename... Args>
cudaError_t launch_pairs(Kernel kernel, int pairs, int threads, size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  pair_config(&cfg, attr, pairs, threads, smem, s);
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int G, int NV, bool PAIR, bool XBF16, bool YBF16, bool CKPT>
cudaError_t bwd_launch(const NormBwdArgs& a, bool wide, bool pwide, int* parts, cudaStream_t s) {
  static LayerGrid cache[3];  // wide: occupancy depends on whether a stage holds a residual
  constexpr int H = NV == 1 ? G : 2 * G, NE = NV == 1 ? 8 : NV * 4;
  const auto wide_kernel = k_norm_bwd<G, NV, XBF16, YBF16, CKPT, PAIR>;
  const auto narrow_kernel = k_norm_bwd_narrow<H, NE, XBF16, YBF16, CKPT, PAIR>;
  const int T = wide ? kCtaThreads<G> : kCtaThreads<H>, groups = T / (wide ? G : H);
  const auto bytes = [](bool residual) {
    constexpr int kX = XBF16 ? 16 : 32, kY = YBF16 ? 16 : 32;
    return size_t(NV) * kCtaThreads<G> *
           (kBwdStages<G, XBF16, YBF16> * (kY + (CKPT ? 16 : kX) + (residual ? kX : 0)) + 32);
  };
  static_assert(kCtaThreads<G> == G || 2 * kCtaThreads<G> * 16 >= 2 * G * 8 * 4, "the sums fit where the stages were");
  const size_t sm = wide ? bytes(a.residual != nullptr) : size_t(groups > 1 ? H * NE * 8 : 0);
  int cap = 0;
  const cudaError_t e = wide ? layer_grid(cache[a.residual != nullptr], reinterpret_cast<const void*>(wide_kernel), T, sm,
                                          bytes(true), &cap)
                             : layer_grid(cache[2], reinterpret_cast<const void*>(narrow_kernel), T, sm, sm, &cap);
  if (e != cudaSuccess) return e;
  if constexpr (PAIR) {
    static LayerGrid pairs[3];
    const cudaError_t f = wide ? pair_slots(pairs[a.residual != nullptr], wide_kernel, T, sm, &cap)
                               : pair_slots(pairs[2], narrow_kernel, T, sm, &cap);
    if (f != cudaSuccess) return f;
    *parts = int(a.rows < cap ? a.rows : cap);
    return wide ? launch_pairs(wide_kernel, *parts, T, sm, s, a, pwide) : launch_pairs(narrow_kernel, *parts, T, sm, s, a);
  }
  if (cap > kNormPartials) cap = kNormPartials;
  const int64_t want = (a.rows + groups - 1) / groups;
  *parts = int(want < cap ? want : cap);
  if (wide)
    wide_kernel<<<*parts, T, sm, s>>>(a, pwide);
  else
    narrow_kernel<<<*parts, T, sm, s>>>(a);
  return cudaGetLastError();
}

template <int G, int NV, bool PAIR, bool XBF16>
cudaError_t bwd_y(const NormBwdArgs& a, bool wide, bool pwide, int* parts, cudaStream_t s) {
  const bool ck = a.x == nullptr;
  if (a.y_bf16)
    return ck ? bwd_launch<G, NV, PAIR, XBF16, true, true>(a, wide, pwide, parts, s)
              : bwd_launch<G, NV, PAIR, XBF16, true, false>(a, wide, pwide, parts, s);
  return ck ? bwd_launch<G, NV, PAIR, XBF16, false, true>(a, wide, pwide, parts, s)
            : bwd_launch<G, NV, PAIR, XBF16, false, false>(a, wide, pwide, parts, s);
}
template <int G, int NV, bool PAIR = false>
cudaError_t bwd(const NormBwdArgs& a, bool wide, bool pwide, int* parts, cudaStream_t s) {
  return a.x_bf16 ? bwd_y<G, NV, PAIR, true>(a, wide, pwide, parts, s) : bwd_y<G, NV, PAIR, false>(a, wide, pwide, parts, s);
}

}  // namespace

cudaError_t launch_norm_forward(const NormFwdArgs& a, cudaStream_t s) {
  const bool wide = wide_rows(a.x, a.ldx, a.rows, a.x_bf16) && wide_rows(a.y, a.ldy, a.rows, a.y_bf16);
  const bool pwide = wide_vec(a.gamma) && wide_vec(a.beta);
  const int64_t pitch = (a.cols + kCkptBlock - 1) / kCkptBlock * kCkptBlock;
  if (pitch <= 256) return fwd<32, 1>(a, wide, pwide, s);
  if (pitch <= 512) return fwd<32, 2>(a, wide, pwide, s);
  if (pitch <= 1024) return fwd<64, 2>(a, wide, pwide, s);
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
    else if (pitch <= 512) e = bwd<64, 1>(a, wide, pwide, &parts, s);
    else if (pitch <= 1024) e = bwd<128, 1>(a, wide, pwide, &parts, s);
    else if (pitch <= 2048) e = bwd<256, 1>(a, wide, pwide, &parts, s);
    else if (pitch <= 4096) e = bwd<256, 2>(a, wide, pwide, &parts, s);
    else if (pitch <= kHalf) e = bwd<512, 2>(a, wide, pwide, &parts, s);
    else if (pitch <= 2 * kHalf) e = bwd<512, 2, true>(a, wide, pwide, &parts, s);
    else {
      if (a.partials != nullptr) {
        // before dx, which may overwrite a residual but none of these inputs
        const int64_t strips = (a.cols + kColStrip - 1) / kColStrip;
        const int64_t want = (a.rows + 63) / 64;
        parts = int(want < 64 ? want : 64);
        const int64_t per = (a.rows + parts - 1) / parts;
        const dim3 grid{unsigned(strips), unsigned(parts)};
        (a.x_bf16 ? k_norm_bwd_cols<true> : k_norm_bwd_cols<false>)<<<grid, kColWarps * 32, 0, s>>>(a, per);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
      }
      const bool out_wide = wide_rows(a.dx, a.lddx, a.rows, a.x_bf16) &&
                            (a.residual == nullptr || wide_rows(a.residual, a.ldr, a.rows, a.x_bf16));
      (a.x_bf16 ? k_norm_bwd_long<true> : k_norm_bwd_long<false>)<<<unsigned(a.rows), kLoop, 0, s>>>(a, out_wide);
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
