// The products of a linear layer's forward and backward passes, with their
// epilogues, on the fifth-generation tensor cores.
//
// All three are D[n][m] = sum_k A[m][k] B[n][k] with m along the output's
// contiguous columns and n along its rows:
//   forward          y[t][n]  = x w^T       m = n (rows of w),     n = t, k = k
//   input gradient   dx[t][k] = dy w        m = k (columns of w),  n = t, k = n
//   weight gradient  dw[n][k] = dy^T x      m = k (columns of x),  n = n, k = t
// A CTA computes tiles of 128 m by bn n (16 to 256), 64 k at a time; a pair of
// CTAs computes 256 m with half of n's operand each, which halves what a product
// reads of it from shared memory.  Operands whose memory runs along k, or along m
// or n, are both taken as they lie (the tensor core's operand descriptors name
// the direction), so nothing is transposed.
//
// Warps: 0 issues TMA loads, 1 issues products, 12 from warp 4 on run the epilogue
// out of tensor memory (8 where it may do everything, 4 beside loaders; two
// accumulators, so it overlaps the next tile's products), and, in the LOADERS
// kernels, 8 more write operands that TMA cannot fetch into the same swizzled
// layout: rows that start on no 16-byte boundary, and checkpoints, which they
// turn into bf16 (exactly, as steps are powers of two).
//
// Few tiles and a long k: `split` CTAs of a cluster share a tile, each with a
// part of k; they leave their partial tiles in shared memory, and each adds up,
// in the order of the parts, the columns it then finishes.
//
// Large products are bound by the tensor cores (and, for seconds on end, by the
// board's power).  Measured, one launch at a time, in TFLOP/s against 1917 of the
// largest library product: forward 8192 x 14336 x 4096 504 us, 1906; with tanh
// GELU and a checkpoint of the pre-activation 595 us, 1615; input gradient 517 us,
// 1860; weight gradient 531 us, 1810; from a checkpoint 673 us, 1430, with a column
// scale 711 us (the loaders' conversion, which every n tile repeats: decoding the
// codes first and taking the product of that is 559 us).
// Few rows are bound by reading w, small products by filling the pipeline once.
//
// The tensor cores add in fp32 but cut each partial sum instead of rounding it.  Of the
// sum of its terms' magnitudes, in units of 2^-24, a sum over k = 4096 (11008) is off by
// 0.32 (0.58) on average and 2.2 (3.6) at most; sums rounded in fp32 by 0.16 (0.19) and
// 3.1 (3.2).  It is the accumulator that the hardware has.
#include <atomic>

#include "layers_common.cuh"
#include "tensor_core.cuh"

namespace loco {

namespace {

constexpr int kTileM = 128, kTileK = 64;
constexpr int kLoadWarps = 8, kLoadGroups = 4;  // loader warps work in pairs, each on every fourth k tile
constexpr int kChunk = 16;                     // output rows an epilogue warp turns over at a time
constexpr int kChunkPitch = 36;                // floats per row of 32 columns: 16-byte reads of 8 rows x 4 lanes meet no bank twice

__device__ unsigned long long g_timeouts;

// What an epilogue may be asked for.  A kernel carries the code of its kind alone: with all of it in
// every kernel, the epilogue's loop missed the instruction cache (a third of its stalls).
enum Epilogue {
  kPlain = 0,    // the sums, and a bias
  kForward = 1,  // bias, activation, checkpoint
  kWeight = 2,   // scale and shift
  kAny = 3       // all of it, with a residual and the slope at a checkpoint
};

template <int BN, bool LOADERS, bool PAIR, int EPI>
struct Shape {
  // Epilogue warps: two per quarter of the accumulator's lanes, or one where loader warps need the registers.
  static constexpr int kEpi = LOADERS ? 4 : EPI == kAny ? 8 : 12;
  static constexpr int kWarps = 4 + kEpi + (LOADERS ? kLoadWarps : 0);
  static constexpr int kStageOut = kEpi * kChunk * kChunkPitch * 4;
  static constexpr int kABytes = kTileM * kTileK * 2, kBRows = PAIR ? BN / 2 : BN, kBBytes = kBRows * kTileK * 2, kStage = kABytes + kBBytes;
  static constexpr int kStages = 200 * 1024 / kStage;
  static constexpr int kTmemCols = 2 * BN < 32 ? 32 : 2 * BN;
  static constexpr size_t kSmem = 1024 + size_t(kStages) * kStage + 256 + kStageOut;
};

struct Params {
  LinearArgs a;
  int a_tma, b_tma;
  int a_cut, b_cut;        // the operand's map is cut into 64-wide columns: one box per tile (see make_cut_map)
  int out_wide, res_wide;  // rows of out and residual start on 16-byte boundaries
  int64_t tiles_m, tiles_n;
  int bn;                    // output rows of a tile: the kernel's BN, or fewer (a multiple of 16, of 32 in a pair)
  int ktiles, split, slots;  // slots: tiles that are worked on at once
  uint64_t wait_ns;  // limit of every wait, longer than the longest tile
};

// Waits as a warp: every lane sees the barrier's phase, and all agree on the outcome.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t limit) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, limit)) != 0;
}

// Tiles in bands of 16 along m, so that the CTAs at work at one time share operand tiles in L2.
__device__ __forceinline__ void tile_at(const Params& p, int64_t tile, int64_t* tm, int64_t* tn) {
  constexpr int64_t kBand = 16;
  const int64_t band = tile / (kBand * p.tiles_n), in = tile - band * kBand * p.tiles_n;
  const int64_t wide = min(kBand, p.tiles_m - band * kBand);
  *tn = in / wide;
  *tm = band * kBand + (in - *tn * wide);
}

// ------------------------------------------------------------------ loaders

// Byte offset of 16-byte unit u (8 values along m) of k-row r of a tile that runs along m: 64-value
// chunks of 64 rows of 128 bytes.  (A tile that runs along k has 128 bytes of k in each row, swizzled alike.)
__device__ __forceinline__ uint32_t unit_offset(int r, int u) {
  return uint32_t(u >> 3) * (kTileK * 128) + uint32_t(r) * 128 + uint32_t(((u & 7) ^ (r & 7)) << 4);
}

__device__ __forceinline__ void st_shared16(uint32_t dst, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ void st_shared4(uint32_t dst, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_shared4(uint32_t src) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(src) : "memory");
  return v;
}
__device__ __forceinline__ void ld_shared8(uint32_t src, float* v) {
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "r"(src) : "memory");
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
               : "r"(src + 16)
               : "memory");
}

// A tile of ROWS (m or n) x 64 (k) bf16 values by the 64 threads of a loader group; 0 for k past the
// matrix.  A unit that starts on no 16-byte boundary is put together from the aligned sixteen bytes on
// either side.  A thread takes the units of every eighth row at the same place in the row (and, along m or
// n, of the next 128 bytes): eight rows are a multiple of 16 bytes, so all its units lie equally far from a
// boundary, and the places it reads and writes are eight rows apart.  Every load of a batch is made, without
// branches, so that all are in flight: those that would leave the matrix are moved inside it.  What they give
// for rows or columns past the matrix along m or n only reaches outputs that are never stored.  In the tiles
// at its edges along k, and where it begins and ends, the units are then mended: cleared past the last k, and
// read element by element where the aligned pieces around them are not all in the matrix.
constexpr int kGroupThreads = kLoadWarps / kLoadGroups * 32;
template <int ROWS, int kBatch>
__device__ __forceinline__ void fill_plain(uint32_t dst, const void* src, int64_t ld, int mn, int64_t row0,
                                           int64_t rows, int64_t k0, int64_t ks, int tid) {
  constexpr int kUnits = ROWS / 8;  // of a thread
  static_assert(kGroupThreads == 64 && kUnits % kBatch == 0 && 8 % kBatch == 0, "whole batches of one column of units");
  const int64_t r0 = mn ? k0 : row0, rlim = mn ? ks : rows, c0 = mn ? row0 : k0, clim = mn ? rows : ks;
  const char* lo = static_cast<const char*>(src);
  const char* hi = lo + ((rlim - 1) * ld + clim) * 2;
  const char* tile = lo + (r0 * ld + c0) * 2;
  const int all_rows = mn ? kTileK : ROWS, all_cols = mn ? ROWS : kTileK;
  const int rleft = int(min(rlim - r0, int64_t(all_rows))), cleft = int(min(clim - c0, int64_t(all_cols)));
  const int64_t pitch = ld * 2;
  const char* end = tile + (rleft - 1) * pitch + cleft * 2;  // of what the tile holds of the matrix
  const bool edge = k0 + kTileK > ks || (tile - lo < 16 && (reinterpret_cast<uintptr_t>(lo) & 15) != 0) || hi - end < 32;
  const bool inside = !edge && rleft == all_rows && cleft == all_cols;
  // the first and the last aligned places to read 32 bytes from
  const char* first = lo + (-reinterpret_cast<uintptr_t>(lo) & 15);
  const char* most = hi - 32 - (reinterpret_cast<uintptr_t>(hi) & 15);
  const bool any = most >= first;
  const int r = tid >> 3, u = tid & 7;
  const char* q = tile + r * pitch + u * 16;
  const uint32_t off = uint32_t(reinterpret_cast<uintptr_t>(q)) & 15u, to = dst + r * 128 + ((u ^ r) << 4);
  const int64_t step = 8 * pitch;
  if (any) {
#pragma unroll 1
    for (int i0 = 0; i0 < kUnits; i0 += kBatch) {
      uint4 x[kBatch], y[kBatch];
      const char* b = q - off + (mn ? (i0 & 7) * step + (i0 >> 3) * 128 : i0 * step);
      if (inside) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          x[i] = __ldg(reinterpret_cast<const uint4*>(b));
          y[i] = __ldg(reinterpret_cast<const uint4*>(b) + 1);
          b += step;
        }
      } else {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const char* c = b < first ? first : b > most ? most : b;
          x[i] = __ldg(reinterpret_cast<const uint4*>(c));
          y[i] = __ldg(reinterpret_cast<const uint4*>(c) + 1);
          b += step;
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) st_shared16(to + (i0 + i) * 1024, shifted16(x[i], y[i], off));
    }
  }
  if (!edge) return;
#pragma unroll 1
  for (int i = 0; i < kUnits; ++i) {
    const int ri = r + (mn ? i & 7 : i) * 8, ui = u + (mn ? i >> 3 : 0) * 8, n = ri < rleft ? cleft - ui * 8 : 0;
    const char* at = tile + ri * pitch + ui * 16;
    const bool safe = any && at - off >= first && at - off <= most;
    if (n >= 8 && safe) continue;
    if (n <= 0) {
      st_shared16(to + i * 1024, make_uint4(0, 0, 0, 0));
      continue;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t w = 0;
      if (n > 2 * k) {
        if (safe) {
          w = ld_shared4(to + i * 1024 + 4 * k);
        } else {
          w = __ldg(reinterpret_cast<const uint16_t*>(at) + 2 * k);
          if (n > 2 * k + 1) w |= uint32_t(__ldg(reinterpret_cast<const uint16_t*>(at) + 2 * k + 1)) << 16;
        }
        if (n == 2 * k + 1) w &= 0xFFFFu;
      }
      st_shared4(to + i * 1024 + 4 * k, w);
    }
  }
}

// A thread's share of a tile of 128 (m) x 64 (k) values of a checkpoint [k][m]: 16 codes along m of
// every eighth k row, with their scales.  Lanes 0-3 and 4-7 of eight hold 64 columns of two
// neighbouring rows, whose places in the swizzle differ in their lowest bit: 8 lanes, 8 bank groups.
constexpr int kPartRows = 8;
static_assert(kGroupThreads * kPartRows == kTileK * kTileM / 16, "64 threads hold a tile");
struct CkptPart {
  uint4 w[kPartRows];
  uint32_t scale[kPartRows];
};
__device__ __forceinline__ int part_row(int tid) { return ((tid >> 2) & 1) + ((tid >> 4) << 1); }  // the first
__device__ __forceinline__ int part_half(int tid) { return (tid & 3) + ((tid >> 3) & 1) * 4; }     // of 8 along m

// Where a thread's codes of one k tile lie.
struct CkptPlace {
  const int8_t* codes;
  const uint8_t* scales;
  int left;    // k rows of the checkpoint from the thread's first on, 0 past its columns
  bool whole;  // the whole tile lies in it
};
__device__ __forceinline__ CkptPlace ckpt_place(const LinearArgs& a, int64_t nb, int64_t m0, int64_t k0, int tid) {
  const int h = part_half(tid);
  const int64_t blk = m0 / kCkptBlock + h / 2, first = k0 + part_row(tid);
  return {a.a_codes + (first * nb + blk) * kCkptBlock + (h & 1) * 16, a.a_scales + first * nb + blk,
          blk < nb ? int(max(int64_t(0), min(a.K - first, int64_t(kTileK)))) : 0,
          m0 + kTileM <= nb * kCkptBlock && k0 + kTileK <= a.K};
}
__device__ __forceinline__ void fetch_ckpt(CkptPart& c, int i, const CkptPlace& at, int64_t nb) {
  const int64_t row = i * 8 * nb;
  if (at.whole) {
    c.w[i] = __ldg(reinterpret_cast<const uint4*>(at.codes + row * kCkptBlock));
    c.scale[i] = __ldg(at.scales + row);
  } else {
    c.w[i] = make_uint4(0, 0, 0, 0);
    c.scale[i] = 1;
    if (i * 8 < at.left) {
      c.w[i] = __ldg(reinterpret_cast<const uint4*>(at.codes + row * kCkptBlock));
      c.scale[i] = __ldg(at.scales + row);
    }
  }
}
// Turns a part into bf16 in the stage and fetches the next into the registers that come free, so that a
// load has a whole k tile's work to arrive.
__device__ __forceinline__ void fill_ckpt(uint32_t dst, CkptPart& c, const CkptPlace& next, int64_t nb, int tid) {
  const uint32_t d0 = dst + unit_offset(part_row(tid), 2 * part_half(tid));
  const uint32_t d1 = dst + unit_offset(part_row(tid), 2 * part_half(tid) + 1);
#pragma unroll
  for (int i = 0; i < kPartRows; ++i) {
    const uint32_t st = ckpt_step_bf16x2(c.scale[i]);
    const uint2 v0 = decode4_bf16(c.w[i].x, st), v1 = decode4_bf16(c.w[i].y, st);
    const uint2 v2 = decode4_bf16(c.w[i].z, st), v3 = decode4_bf16(c.w[i].w, st);
    fetch_ckpt(c, i, next, nb);
    st_shared16(d0 + i * 1024, make_uint4(v0.x, v0.y, v1.x, v1.y));
    st_shared16(d1 + i * 1024, make_uint4(v2.x, v2.y, v3.x, v3.y));
  }
}

// ------------------------------------------------------------------ epilogue

// The epilogue works on eight consecutive columns of a row per lane, four lanes to a checkpoint
// block, so that every access to memory is a 16- or 8-byte one where alignment allows.

// What belongs to a lane's eight columns.
struct Columns {
  int64_t m;      // the first
  int live;       // how many of them the output has
  float mul[8];   // col_scale
  float add[8];   // col_shift, or the bias
};

template <int EPI>
__device__ __forceinline__ Columns columns_of(const LinearArgs& a, int64_t m) {
  Columns c;
  c.m = m;
  c.live = int(max(int64_t(0), min(int64_t(8), a.M - m)));
  const void* add = EPI >= kWeight && a.col_shift != nullptr ? a.col_shift : a.bias;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    c.mul[k] = EPI >= kWeight && a.col_scale != nullptr && k < c.live ? load_elem(a.col_scale, m + k, a.param_bf16) : 1.0f;
    c.add[k] = add != nullptr && k < c.live ? load_elem(add, m + k, a.param_bf16) : 0.0f;
  }
  return c;
}

// What the epilogue of one row's eight columns reads, fetched ahead of its use.
struct Ahead {
  uint4 r0, r1;   // the residual: eight bf16 in r0, or eight fp32
  uint2 z;        // eight codes of the checkpointed pre-activation
  uint32_t zs;    // and their scale
};

template <int EPI>
__device__ __forceinline__ Ahead fetch_ahead(const Params& p, const Columns& c, int64_t n, bool row) {
  const LinearArgs& a = p.a;
  Ahead h;
  h.r0 = h.r1 = make_uint4(0, 0, 0, 0);
  h.z = make_uint2(0, 0);
  h.zs = 1;
  if (EPI != kAny || !row || c.live <= 0) return h;
  if (a.residual != nullptr) {
    const char* q = static_cast<const char*>(a.residual) + (n * a.ldr + c.m) * (a.out_bf16 ? 2 : 4);
    if (p.res_wide && c.live == 8) {
      h.r0 = *reinterpret_cast<const uint4*>(q);
      if (!a.out_bf16) h.r1 = *reinterpret_cast<const uint4*>(q + 16);
    } else if (a.out_bf16) {
      uint32_t e[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) e[k] = k < c.live ? uint32_t(reinterpret_cast<const uint16_t*>(q)[k]) : 0u;
      h.r0 = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
    } else {
      uint32_t e[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) e[k] = k < c.live ? reinterpret_cast<const uint32_t*>(q)[k] : 0u;
      h.r0 = make_uint4(e[0], e[1], e[2], e[3]);
      h.r1 = make_uint4(e[4], e[5], e[6], e[7]);
    }
  }
  if (a.z_codes != nullptr) {
    const int64_t nb = (a.M + kCkptBlock - 1) / kCkptBlock;
    h.z = __ldg(reinterpret_cast<const uint2*>(a.z_codes + n * nb * kCkptBlock + c.m));
    h.zs = __ldg(a.z_scales + n * nb + c.m / kCkptBlock);
  }
  return h;
}

// Row n of the lane's columns, v the sums over k.  Every lane of the warp takes part; `row`: the row exists.
// With `keep` the result goes back to that place in shared memory instead of the output.
template <int EPI>
__device__ __forceinline__ void finish(const Params& p, const Columns& c, float (&v)[8], int64_t n, bool row,
                                       const Ahead& h, uint32_t keep = 0) {
  const LinearArgs& a = p.a;
  if (EPI >= kWeight && (a.col_scale != nullptr || a.col_shift != nullptr)) {
    const float rs = a.col_shift != nullptr && row ? __ldg(a.row_sum + n) : 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = fmaf(c.add[k], rs, v[k] * c.mul[k]);
  } else if (a.bias != nullptr) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] += c.add[k];
  }
  if ((EPI == kForward || EPI == kAny) && a.save_codes != nullptr) {
    uint32_t mag = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (k >= c.live) v[k] = 0.0f;
      mag = max(mag, mag_bits(v[k]));
    }
    mag = max(mag, __shfl_xor_sync(0xFFFFFFFFu, mag, 1));
    mag = max(mag, __shfl_xor_sync(0xFFFFFFFFu, mag, 2));
    const int64_t nb = (a.M + kCkptBlock - 1) / kCkptBlock, blk = c.m / kCkptBlock;
    if (row && blk < nb) {
      *reinterpret_cast<uint2*>(a.save_codes + n * nb * kCkptBlock + c.m) = ckpt_pack8(v, mag);
      if ((c.m & 31) == 0) a.save_scales[n * nb + blk] = uint8_t(ckpt_scale(mag));
    }
  }
  if (!row || c.live <= 0) return;
  if (EPI == kAny && a.z_codes != nullptr) {
    float z[8];
    const float st = ckpt_step(h.zs);
    ckpt_unpack4(h.z.x, st, z);
    ckpt_unpack4(h.z.y, st, z + 4);
    mul_slope(v, z, a.act);
  } else if (EPI == kForward || EPI == kAny) {
    apply_act(v, a.act);
  }
  if (EPI == kAny && a.residual != nullptr) {
    const uint32_t w[8] = {h.r0.x, h.r0.y, h.r0.z, h.r0.w, h.r1.x, h.r1.y, h.r1.z, h.r1.w};
    if (a.out_bf16) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] += __uint_as_float(w[k] << 16);
        v[2 * k + 1] += __uint_as_float(w[k] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] += __uint_as_float(w[k]);
    }
  }
  const int64_t at = n * a.ldo + c.m;
  if (keep != 0) {
    st_shared16(keep, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
    st_shared16(keep + 16, make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])));
  } else if (p.out_wide && c.live == 8) {
    store8(a.out, at, a.out_bf16, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < c.live) store_elem(a.out, at + k, a.out_bf16, v[k]);
  }
}

// The same where the tile lies wholly inside an output of wide rows: rows n and n + 8 of the lane's
// columns at a time, with no bounds, and each choice made once for sixteen values.
template <int EPI>
__device__ __forceinline__ void fetch_whole(const LinearArgs& a, const Columns& c, int64_t n, int64_t nb, Ahead (&h)[2]) {
  if (EPI != kAny) return;
  if (a.residual != nullptr) {
    const int oe = a.out_bf16 ? 2 : 4;
    const char* q = static_cast<const char*>(a.residual) + (n * a.ldr + c.m) * oe;
    const int64_t eight = 8 * a.ldr * oe;
    h[0].r0 = *reinterpret_cast<const uint4*>(q);
    h[1].r0 = *reinterpret_cast<const uint4*>(q + eight);
    if (!a.out_bf16) {
      h[0].r1 = *reinterpret_cast<const uint4*>(q + 16);
      h[1].r1 = *reinterpret_cast<const uint4*>(q + eight + 16);
    }
  }
  if (a.z_codes != nullptr) {
    const int64_t at = n * nb * kCkptBlock + c.m;
    h[0].z = __ldg(reinterpret_cast<const uint2*>(a.z_codes + at));
    h[1].z = __ldg(reinterpret_cast<const uint2*>(a.z_codes + at + 8 * nb * kCkptBlock));
    h[0].zs = __ldg(a.z_scales + at / kCkptBlock);
    h[1].zs = __ldg(a.z_scales + at / kCkptBlock + 8 * nb);
  }
}
template <int EPI>
__device__ __forceinline__ void finish_whole(const LinearArgs& a, const Columns& c, float (&v)[16], int64_t n, int64_t nb,
                                             const Ahead (&h)[2]) {
  if (EPI >= kWeight && (a.col_scale != nullptr || a.col_shift != nullptr)) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float rs = a.col_shift != nullptr ? __ldg(a.row_sum + n + 8 * i) : 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[8 * i + k] = fmaf(c.add[k], rs, v[8 * i + k] * c.mul[k]);
    }
  } else if (a.bias != nullptr) {
#pragma unroll
    for (int k = 0; k < 16; ++k) v[k] += c.add[k & 7];
  }
  if ((EPI == kForward || EPI == kAny) && a.save_codes != nullptr) {
    const int64_t at = n * nb * kCkptBlock + c.m;
    const uint32_t m0 = block_magnitude(v), m1 = block_magnitude(v + 8);
    *reinterpret_cast<uint2*>(a.save_codes + at) = ckpt_pack8(v, m0);
    *reinterpret_cast<uint2*>(a.save_codes + at + 8 * nb * kCkptBlock) = ckpt_pack8(v + 8, m1);
    if ((c.m & 31) == 0) {
      a.save_scales[at / kCkptBlock] = uint8_t(ckpt_scale(m0));
      a.save_scales[at / kCkptBlock + 8 * nb] = uint8_t(ckpt_scale(m1));
    }
  }
  if (EPI == kAny && a.z_codes != nullptr) {
    float z[16];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      Pair q[4];
      ckpt_pairs4(h[i].z.x, h[i].zs, q);
      ckpt_pairs4(h[i].z.y, h[i].zs, q + 2);
      floats8(q, z + 8 * i);
    }
    mul_slope(v, z, a.act);
  } else if (EPI == kForward || EPI == kAny) {
    apply_act(v, a.act);
  }
  const int oe = a.out_bf16 ? 2 : 4;
  char* out = static_cast<char*>(a.out) + (n * a.ldo + c.m) * oe;
  const int64_t eight = 8 * a.ldo * oe;
  if (a.out_bf16) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float* u = v + 8 * i;
      if (EPI == kAny && a.residual != nullptr) {
        const uint32_t w[4] = {h[i].r0.x, h[i].r0.y, h[i].r0.z, h[i].r0.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          u[2 * k] += __uint_as_float(w[k] << 16), u[2 * k + 1] += __uint_as_float(w[k] & 0xFFFF0000u);
      }
      *reinterpret_cast<uint4*>(out + i * eight) = make_uint4(pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3]),
                                                              pack_bf16x2(u[4], u[5]), pack_bf16x2(u[6], u[7]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float* u = v + 8 * i;
      if (EPI == kAny && a.residual != nullptr) {
        const uint32_t w[8] = {h[i].r0.x, h[i].r0.y, h[i].r0.z, h[i].r0.w, h[i].r1.x, h[i].r1.y, h[i].r1.z, h[i].r1.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] += __uint_as_float(w[k]);
      }
      *reinterpret_cast<float4*>(out + i * eight) = make_float4(u[0], u[1], u[2], u[3]);
      *reinterpret_cast<float4*>(out + i * eight + 16) = make_float4(u[4], u[5], u[6], u[7]);
    }
  }
}

// ------------------------------------------------------------------ the kernel

template <int BN, bool LOADERS, bool PAIR, int EPI>
__global__ void __launch_bounds__(Shape<BN, LOADERS, PAIR, EPI>::kWarps * 32, 1)
    k_linear(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
             const __grid_constant__ Params p) {
  using S = Shape<BN, LOADERS, PAIR, EPI>;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  const uint32_t bars = base + S::kStages * S::kStage;
  const auto full = [&](int s) { return bars + 8u * s; };
  const auto empty = [&](int s) { return bars + 8u * (S::kStages + s); };
  const auto acc_full = [&](int b) { return bars + 8u * (2 * S::kStages + b); };
  const auto acc_empty = [&](int b) { return bars + 8u * (2 * S::kStages + 2 + b); };
  const uint32_t drain = bars + 8u * (2 * S::kStages + 4);
  const uint32_t tmem_at = bars + 8u * (2 * S::kStages + 5);
  static_assert(8 * (2 * S::kStages + 6) <= 256, "barriers fit behind the stages");

  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int rank = PAIR || p.split > 1 ? int(cluster_rank()) : 0;
  const int ctas = PAIR ? 2 : p.split;  // of a cluster: they share a tile
  const int64_t workers = gridDim.x / ctas, worker = blockIdx.x / ctas;
  const int64_t tiles = p.tiles_m * p.tiles_n;
  const int kt0 = PAIR ? 0 : int(int64_t(p.ktiles) * rank / p.split);
  const int kt1 = PAIR ? p.ktiles : int(int64_t(p.ktiles) * (rank + 1) / p.split);
  const int brows = PAIR ? p.bn / 2 : p.bn;  // rows of B that the CTA loads
  // First output column of the CTA's part of a tile.
  const auto col0 = [&](int64_t tm) { return PAIR ? tm * (2 * kTileM) + rank * kTileM : tm * kTileM; };
  // The CTA that issues a pair's products is its first; its barriers count for both.
  static_assert(!(PAIR && LOADERS), "a pair's operands come by TMA: loaders would have to publish across CTAs");
  const auto lead = [&](uint32_t bar) { return PAIR ? cluster_addr(bar, 0) : bar; };
  // A warp has read its part of an accumulator (ordered by tcgen05 fences: no memory is handed over).
  const auto drained = [&](uint32_t bar) {
    if (PAIR)
      mbar_arrive_remote(lead(bar));
    else
      mbar_arrive(bar);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(full(s), 1 + (LOADERS ? kLoadWarps / kLoadGroups : 0));
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), S::kEpi * (PAIR ? 2 : 1));
    }
    mbar_init(drain, 1);
    mbar_init_fence();
    if (p.a_tma) tma_prefetch_map(&ta);
    if (p.b_tma) tma_prefetch_map(&tb);
  }
  if (warp == 2) tmem_alloc<PAIR>(tmem_at, S::kTmemCols);
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // the barriers of both are ready
  tc_fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(tmem) : "r"(tmem_at));
  bool gave_up = false;

  if (warp == 0 && lane == 0) {
    // ---- TMA loads (in the LOADERS kernels possibly of one operand, or none)
    int stage = 0, phase = 0;
    int64_t issued = 0;
    for (int64_t tile = worker; tile < tiles && !gave_up; tile += workers) {
      int64_t tm, tn;
      tile_at(p, tile, &tm, &tn);
      const int m0 = int(col0(tm)), n0 = int(tn * p.bn) + (PAIR ? rank * brows : 0);
      // B's boxes are whole ones: 64 wide along n, however little of the last is used
      const int bboxes = (brows + 63) / 64;
      const uint32_t bbytes = p.a.b_mn ? uint32_t(bboxes) * (kTileK * 128) : uint32_t(brows) * 128;
      for (int kt = kt0; kt < kt1; ++kt) {
        if (!mbar_wait(empty(stage), phase ^ 1, p.wait_ns)) {
          gave_up = true;
          break;
        }
        const uint32_t sa = base + stage * S::kStage, sb = sa + S::kABytes, bar = lead(full(stage));
        const int k0 = kt * kTileK;
        // the bytes of both CTAs of a pair
        if (!PAIR || rank == 0)
          mbar_arrive_expect(full(stage), ((p.a_tma ? S::kABytes : 0) + (p.b_tma ? bbytes : 0)) * (PAIR ? 2 : 1));
        if (p.a_tma) {
          if (!p.a.a_mn) {
            tma_load_2d<PAIR>(sa, &ta, k0, m0, bar);
          } else if (p.a_cut) {
            tma_load_3d<PAIR>(sa, &ta, 0, k0, m0 / 64, bar);
          } else {
#pragma unroll
            for (int c = 0; c < kTileM / 64; ++c) tma_load_2d<PAIR>(sa + c * (kTileK * 128), &ta, m0 + c * 64, k0, bar);
          }
        }
        if (p.b_tma) {
          if (!p.a.b_mn) {
            tma_load_2d<PAIR>(sb, &tb, k0, n0, bar);
          } else if (p.b_cut) {
            tma_load_3d<PAIR>(sb, &tb, 0, k0, n0 / 64, bar);
          } else {
            for (int c = 0; c < bboxes; ++c) tma_load_2d<PAIR>(sb + c * (kTileK * 128), &tb, n0 + c * 64, k0, bar);
          }
        }
        ++issued;
        if (++stage == S::kStages) stage = 0, phase ^= 1;
      }
    }
    // The CTA stays until the products have read its last stages: their signals come here, and say that the copies landed.
    for (int i = 0, s = stage, ph = phase; i < S::kStages && !gave_up; ++i) {
      gave_up = !mbar_wait(empty(s), ph ^ 1, p.wait_ns);
      if (++s == S::kStages) s = 0, ph ^= 1;
    }
    if (gave_up) {
      // Let the copies in flight land at least.  (The second CTA of a pair has them counted
      // at the first's barriers; it waits a time in which any copy has landed.)
      if (PAIR && rank != 0) {
        for (int i = 0; i < 100; ++i) __nanosleep(100000);
      } else {
        for (int i = 0; i < S::kStages && i < issued; ++i) {
          if (--stage < 0) stage = S::kStages - 1, phase ^= 1;
          if (!mbar_wait(full(stage), phase, p.wait_ns)) break;
        }
      }
    }
  } else if (warp == 1 && lane == 0 && (!PAIR || rank == 0)) {
    // ---- products
    const uint32_t desc = mma_desc(PAIR ? 2 * kTileM : kTileM, p.bn, p.a.a_mn, p.a.b_mn);
    const uint32_t chunk = kTileK * 128;
    const uint64_t astep = p.a.a_mn ? 2048 / 16 : 32 / 16, bstep = p.a.b_mn ? 2048 / 16 : 32 / 16;
    bool ran = false;
    int stage = 0, phase = 0, buf = 0, bphase = 0;
    for (int64_t tile = worker; tile < tiles && !gave_up; tile += workers) {
      if (kt0 == kt1) break;
      if (!mbar_wait(acc_empty(buf), bphase ^ 1, p.wait_ns)) {
        gave_up = true;
        break;
      }
      tc_fence_after();
      const uint32_t d = tmem + buf * BN;
      for (int kt = kt0; kt < kt1; ++kt) {
        if (!mbar_wait(full(stage), phase, p.wait_ns)) {
          gave_up = true;
          break;
        }
        // Orders the loaders' writes, seen through the barrier, before the tensor core's reads.  (A fence
        // by the loaders themselves would wait for their loads of the next k tiles.)
        if (LOADERS) fence_async_shared();
        tc_fence_after();
        const uint32_t sa = base + stage * S::kStage;
        const uint64_t da = smem_desc(sa, chunk), db = smem_desc(sa + S::kABytes, chunk);
#pragma unroll
        for (int k = 0; k < kTileK / 16; ++k) mma_bf16<PAIR>(d, da + k * astep, db + k * bstep, desc, kt > kt0 || k > 0);
        mma_commit<PAIR>(empty(stage));
        if (++stage == S::kStages) stage = 0, phase ^= 1;
      }
      if (gave_up) break;
      mma_commit<PAIR>(acc_full(buf));
      ran = true;
      buf ^= 1;
      if (buf == 0) bphase ^= 1;
    }
    // Nor does tensor memory go while products write it, even if the epilogue gave its wait up.
    if (!gave_up && ran) gave_up = !mbar_wait(acc_full(buf ^ 1), buf == 0 ? bphase ^ 1 : bphase, p.wait_ns);
    if (gave_up) {
      mma_commit<PAIR>(drain);
      mbar_wait(drain, 0, p.wait_ns);
    }
  } else if (warp >= 4 && warp < 4 + S::kEpi) {
    // ---- epilogue: lane i of a warp reads row q*32 + i of the accumulator, an output column; 16
    // output rows at a time are turned over in shared memory so that a lane has 8 columns of a row.
    const int q = warp & 3, half = (warp - 4) / 4;
    constexpr int kStride = S::kEpi / 4 * kChunk;  // output rows between a warp's chunks
    const uint32_t mine = bars + 256 + uint32_t(warp - 4) * (kChunk * kChunkPitch * 4);
    const int sub = lane / 4, seg = lane & 3;
    int buf = 0, bphase = 0;
    for (int64_t tile = worker; tile < tiles; tile += workers) {
      int64_t tm, tn;
      tile_at(p, tile, &tm, &tn);
      const int64_t n0 = tn * p.bn;
      const int rows = int(min(int64_t(p.bn), p.a.N - n0));
      Columns col;
      Ahead ahead[kChunk / 8];
      static_assert(kChunk == 16, "finish_whole takes two rows of eight");
      // wholly inside an output of wide rows?
      const bool whole = p.split == 1 && rows == p.bn && col0(tm) + kTileM <= p.a.M && p.out_wide &&
                         (p.a.residual == nullptr || p.res_wide);
      const int64_t nb = (p.a.M + kCkptBlock - 1) / kCkptBlock;
      const int64_t m0 = col0(tm) + q * 32;  // the warp's columns
      if (p.split == 1) {
        col = columns_of<EPI>(p.a, col0(tm) + q * 32 + seg * 8);
        if (whole) {
          if (half * kChunk < rows) fetch_whole<EPI>(p.a, col, n0 + half * kChunk + sub, nb, ahead);
        } else {
#pragma unroll
          for (int i = 0; i < kChunk / 8; ++i) {
            const int j = half * kChunk + i * 8 + sub;
            ahead[i] = fetch_ahead<EPI>(p, col, n0 + j, j < rows);
          }
        }
      }
      if (kt0 < kt1) {
        if (!warp_wait(acc_full(buf), bphase, p.wait_ns)) {
          gave_up = true;
          break;
        }
        tc_fence_after();
        if (half * kChunk >= rows && lane == 0) drained(acc_empty(buf));
      }
#pragma unroll 1
      for (int j0 = half * kChunk; j0 < rows; j0 += kStride) {
        uint32_t w[16];
        if (kt0 < kt1) {
          tmem_load16(tmem + buf * BN + j0 + (uint32_t(q * 32) << 16), w);
          tmem_wait_loads();
          if (j0 + kStride >= rows) {
            // the warp's part of the accumulator has been read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) drained(acc_empty(buf));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = 0;
        }
        if (p.split > 1) {
          // the whole tile stays in shared memory as [n][m], for the cluster
#pragma unroll
          for (int i = 0; i < 16; ++i)
            st_shared4(base + uint32_t(((j0 + i) * kTileM + q * 32 + lane) * 4), w[i]);
          continue;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) st_shared4(mine + uint32_t(i * kChunkPitch + lane) * 4, w[i]);
        __syncwarp();
        float v[kChunk / 8 * 8];
#pragma unroll
        for (int i = 0; i < kChunk / 8; ++i) ld_shared8(mine + uint32_t((i * 8 + sub) * kChunkPitch + seg * 8) * 4, v + 8 * i);
        __syncwarp();
        if (whole) {
          const Ahead now[2] = {ahead[0], ahead[1]};
          if (j0 + kStride < rows) fetch_whole<EPI>(p.a, col, n0 + j0 + kStride + sub, nb, ahead);
          finish_whole<EPI>(p.a, col, v, n0 + j0 + sub, nb, now);
          continue;
        }
#pragma unroll
        for (int i = 0; i < kChunk / 8; ++i) {
          const Ahead now = ahead[i];
          const int j = j0 + i * 8 + sub, nx = j + kStride;
          ahead[i] = fetch_ahead<EPI>(p, col, n0 + nx, nx < rows);
          float (&u)[8] = reinterpret_cast<float (&)[8]>(v[8 * i]);
          finish<EPI>(p, col, u, n0 + j, j < rows, now,
                      p.out_wide ? 0u : mine + uint32_t((i * 8 + sub) * kChunkPitch + seg * 8) * 4);
        }
        if (!p.out_wide) {
          // Rows that take no 16-byte stores: a column per lane, so that a store meets one row's lines and
          // not those of eight rows (4095 x 4097 x 4099 of aligned operands, bf16 output: 192 us so, 136 us here).
          __syncwarp();
          const int some = m0 + lane < p.a.M ? min(rows - j0, kChunk) : 0;
          int64_t at = (n0 + j0) * p.a.ldo + m0 + lane;
#pragma unroll 4
          for (int i = 0; i < some; ++i, at += p.a.ldo)
            store_elem(p.a.out, at, p.a.out_bf16, __uint_as_float(ld_shared4(mine + uint32_t(i * kChunkPitch + lane) * 4)));
          __syncwarp();
        }
      }
      buf ^= 1;
      if (buf == 0) bphase ^= 1;
    }
  } else if (warp >= 4 + S::kEpi) {
    if constexpr (LOADERS) {
    // ---- plain loads and checkpoints.  A k tile takes a group longer than its products take, mostly
    // in waiting; four groups on four k tiles keep up with them.
    const int index = warp - 4 - S::kEpi, group = index / (kLoadWarps / kLoadGroups);
    const int tid = threadIdx.x % kGroupThreads;
    const int64_t nb = (p.a.M + kCkptBlock - 1) / kCkptBlock;
    const int nk = kt1 - kt0;
    // position of a step of this CTA's k tiles, all tiles counted through
    struct Place {
      int64_t tile, tm, tn;
      int kt;
    };
    const auto advance = [&](Place& at, int by) {
      at.kt += by;
      bool moved = by == 0;
      while (at.kt >= kt1 && at.tile < tiles) at.kt -= nk, at.tile += workers, moved = true;
      if (moved && at.tile < tiles) tile_at(p, at.tile, &at.tm, &at.tn);
    };
    Place now{worker, 0, 0, kt0};
    if (nk > 0) {
      advance(now, 0);
      advance(now, group);
    } else {
      now.tile = tiles;
    }
    const auto place = [&](const Place& at) {
      if (at.tile >= tiles) return CkptPlace{p.a.a_codes, p.a.a_scales, 0, false};
      return ckpt_place(p.a, nb, col0(at.tm), int64_t(at.kt) * kTileK, tid);
    };
    int stage = group, phase = 0;
    static_assert(S::kStages >= kLoadGroups, "a group's first stage is one of the ring's");
    // Fills the stages of the group's k tiles; fill(stage) goes on to the next of them.
    const auto walk = [&](auto fill) {
      while (now.tile < tiles) {
        if (!warp_wait(empty(stage), phase ^ 1, p.wait_ns)) {
          gave_up = true;
          break;
        }
        fill(base + stage * S::kStage);
        __syncwarp();
        if (lane == 0) mbar_arrive(full(stage));
        stage += kLoadGroups;
        if (stage >= S::kStages) stage -= S::kStages, phase ^= 1;
      }
    };
    if (p.a.a_codes != nullptr) {
      CkptPart part;
      const CkptPlace at = place(now);
#pragma unroll
      for (int i = 0; i < kPartRows; ++i) fetch_ckpt(part, i, at, nb);
      walk([&](uint32_t sa) {
        if (!p.b_tma)
          fill_plain<S::kBRows, 4>(sa + S::kABytes, p.a.b, p.a.ldb, p.a.b_mn, now.tn * p.bn, p.a.N,
                                   int64_t(now.kt) * kTileK, p.a.K, tid);
        advance(now, kLoadGroups);
        fill_ckpt(sa, part, place(now), nb, tid);
      });
    } else {
      walk([&](uint32_t sa) {
        const int64_t k0 = int64_t(now.kt) * kTileK;
        if (!p.b_tma)
          fill_plain<S::kBRows, 8>(sa + S::kABytes, p.a.b, p.a.ldb, p.a.b_mn, now.tn * p.bn, p.a.N, k0, p.a.K, tid);
        if (!p.a_tma) fill_plain<kTileM, 8>(sa, p.a.a, p.a.lda, p.a.a_mn, col0(now.tm), p.a.M, k0, p.a.K, tid);
        advance(now, kLoadGroups);
      });
    }
    }
  }
  if (gave_up && lane == 0) atomicAdd(&g_timeouts, 1ull);
  __syncwarp();

  if (!PAIR && p.split > 1) {
    // One tile per cluster.  Its parts lie in the CTAs' shared memory as [n][m]; each CTA adds up
    // and finishes its share of the rows.
    int64_t tm, tn;
    tile_at(p, worker, &tm, &tn);
    const int64_t n0 = tn * p.bn;
    const int rows = int(min(int64_t(p.bn), p.a.N - n0));
    // A part whose sums did not come is NaN, not what its memory holds: so is the output then.
    if (__syncthreads_or(gave_up))
      for (int i = threadIdx.x; i < rows * kTileM; i += S::kWarps * 32) st_shared4(base + uint32_t(i) * 4, 0x7FC00000u);
    cluster_sync();
    const int q = warp & 3, side = warp / 4, sides = S::kWarps / 4;
    const int sub = lane / 4, seg = lane & 3;
    const Columns col = columns_of<EPI>(p.a, tm * kTileM + q * 32 + seg * 8);
    const int share = (rows + p.split - 1) / p.split, lo = share * rank, hi = min(rows, lo + share);
    for (int j0 = lo + side * 8; j0 < hi; j0 += sides * 8) {
      const int j = min(j0 + sub, hi - 1);
      const bool row = j0 + sub < hi;
      const Ahead h = fetch_ahead<EPI>(p, col, n0 + j, row);
      const uint32_t at = base + uint32_t((j * kTileM + q * 32 + seg * 8) * 4);
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = 0.0f;
      for (int r = 0; r < p.split; ++r) {
        float w[8];
        cluster_load8(cluster_addr(at, uint32_t(r)), w);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += w[k];
      }
      finish<EPI>(p, col, v, n0 + j, row, h);
    }
    cluster_sync();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if constexpr (PAIR) cluster_sync();  // neither leaves while the other may read or signal it
  if (warp == 2) tmem_free<PAIR>(tmem, S::kTmemCols);
}

// ------------------------------------------------------------------ few rows

// A forward pass of at most TT <= 4 rows of x: bound by reading w once (1 x 11008 x 4096: 14.6 us, 6.2 TB/s,
// of which the launch is 2 us).  32 rows of w per CTA, four per
// warp: a lane takes 8 of every 256 k of them, kAhead such loads of each row in flight, and the warp
// adds up its lanes.  The tensor cores would have 128 x 16 tiles mostly of zeros to fill, and too few of them
// to keep every SM reading.
constexpr int kRowWarps = 8, kRowsPerWarp = 4;

template <int TT, int kAhead, int EPI = kAny>
__global__ void __launch_bounds__(kRowWarps * 32, kAhead == 2 && TT == 1 ? 3 : 2) k_linear_rows(const __grid_constant__ Params p) {
  __shared__ float sums[TT][kRowWarps * kRowsPerWarp + 4];
  const LinearArgs& a = p.a;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int64_t m0 = int64_t(blockIdx.x) * (kRowWarps * kRowsPerWarp);
  const uint16_t* w = static_cast<const uint16_t*>(a.a);
  const uint16_t* x = static_cast<const uint16_t*>(a.b);
  const uint16_t* rows[kRowsPerWarp];
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i) rows[i] = w + min(m0 + warp * kRowsPerWarp + i, a.M - 1) * a.lda;
  Pair acc[kRowsPerWarp][TT];
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[i][t] = pair(0.0f, 0.0f);
  const auto step = [&](const uint4 (&wv)[kRowsPerWarp], int64_t k) {
    Pair wp[kRowsPerWarp][4];
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i) widen8(wv[i], wp[i]);
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      Pair xp[4];
      widen8(t < a.N ? __ldg(reinterpret_cast<const uint4*>(x + t * a.ldb + k)) : make_uint4(0, 0, 0, 0), xp);
#pragma unroll
      for (int i = 0; i < kRowsPerWarp; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][t] = fma(wp[i][j], xp[j], acc[i][t]);
    }
  };
  int64_t k = lane * 8;
  for (; k + (kAhead - 1) * 256 + 8 <= a.K; k += kAhead * 256) {
    uint4 wv[kAhead][kRowsPerWarp];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int i = 0; i < kRowsPerWarp; ++i) wv[j][i] = __ldcs(reinterpret_cast<const uint4*>(rows[i] + k + j * 256));
#pragma unroll
    for (int j = 0; j < kAhead; ++j) step(wv[j], k + j * 256);
  }
  for (; k + 8 <= a.K; k += 256) {
    uint4 wv[kRowsPerWarp];
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i) wv[i] = __ldcs(reinterpret_cast<const uint4*>(rows[i] + k));
    step(wv, k);
  }
  const int64_t last = (a.K & ~int64_t(7)) + lane;  // the values after the last whole eight
  if (last < a.K) {
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i)
#pragma unroll
      for (int t = 0; t < TT; ++t)
        if (t < a.N)
          acc[i][t] = acc[i][t] + pair(bf16_bits_to_f32(__ldg(rows[i] + last)) * bf16_bits_to_f32(__ldg(x + t * a.ldb + last)), 0.0f);
  }
#pragma unroll
  for (int i = 0; i < kRowsPerWarp; ++i)
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const float2 h = halves(acc[i][t]);
      float v = h.x + h.y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
      if (lane == 0) sums[t][warp * kRowsPerWarp + i] = v;
    }
  __syncthreads();
  if (warp == 0) {
    const int t = lane / 4, seg = lane & 3;
    const bool row = t < a.N;
    const Columns col = columns_of<EPI>(a, m0 + seg * 8);
    const Ahead h = fetch_ahead<EPI>(p, col, t, row);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = row ? sums[t < TT ? t : 0][seg * 8 + j] : 0.0f;
    finish<EPI>(p, col, v, t, row, h);
  }
}

// Four loads of a row in flight where there are few CTAs per SM, else two and more CTAs (1 row of x:
// 4096 x 11008 21.2 against 18.7 us, 11008 x 4096 14.6 against 18.6 us).
cudaError_t launch_rows(const Params& p, int sms, cudaStream_t s) {
  const unsigned grid = unsigned((p.a.M + 31) / 32);
  const bool deep = int64_t(grid) <= 2 * int64_t(sms);
  const auto kernel = p.a.N == 1   ? (deep ? k_linear_rows<1, 4> : k_linear_rows<1, 2>)
                      : p.a.N == 2 ? (deep ? k_linear_rows<2, 4> : k_linear_rows<2, 2>)
                                   : k_linear_rows<4, 2>;
  kernel<<<grid, kRowWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ launch

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static EncodeFn fn = []() -> EncodeFn {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// Whether TMA can fetch the matrix: base and rows on 16-byte boundaries.
bool tma_can(const void* p, int64_t rows, int64_t ld) {
  return p != nullptr && reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || ld % 8 == 0);
}

// Map of a bf16 matrix of `rows` rows of `cols` contiguous values, in boxes of 64 x box_rows.  (A
// pitch that is no multiple of 8 belongs to a single row, whose pitch is never used.)
cudaError_t make_map(CUtensorMap* map, const void* p, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
  const EncodeFn fn = encode_fn();
  if (fn == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)}, strides[1] = {cuuint64_t((ld + 7) / 8 * 8) * 2};
  const cuuint32_t box[2] = {kTileK, cuuint32_t(box_rows)}, one[2] = {1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box, one,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Map of a bf16 matrix of `rows` rows of `cols` contiguous values, cols a multiple of 64, as columns of
// 64: boxes of 64 x 64 rows x `columns`, which arrive column after column.  A tile whose rows run along
// m or n is one such box instead of two to four: the thread that issues them is busy enough (8192 x 14336
// x 4096 weight gradient 683 -> 598 us).
cudaError_t make_cut_map(CUtensorMap* map, const void* p, int64_t rows, int64_t cols, int64_t ld, int columns) {
  const EncodeFn fn = encode_fn();
  if (fn == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {64, cuuint64_t(rows), cuuint64_t(cols / 64)};
  const cuuint64_t strides[2] = {cuuint64_t((ld + 7) / 8 * 8) * 2, 128};
  const cuuint32_t box[3] = {64, kTileK, cuuint32_t(columns)}, one[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, one,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int BN, bool LOADERS, bool PAIR, int EPI>
cudaError_t launch_kind(const Params& in, cudaStream_t s) {
  using S = Shape<BN, LOADERS, PAIR, EPI>;
  Params p = in;
  const int brows = PAIR ? p.bn / 2 : p.bn;
  p.a_cut = p.a.a_mn && p.a.M % 64 == 0;
  p.b_cut = p.a.b_mn && p.a.N % 64 == 0 && brows % 64 == 0;
  static std::atomic<bool> ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(k_linear<BN, LOADERS, PAIR, EPI>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(S::kSmem));
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev].store(true, std::memory_order_release);
  }
  CUtensorMap ta{}, tb{};
  const LinearArgs& a = p.a;
  if (p.a_tma && p.ktiles > 0) {
    e = p.a_cut ? make_cut_map(&ta, a.a, a.K, a.M, a.lda, kTileM / 64)
        : a.a_mn ? make_map(&ta, a.a, a.K, a.M, a.lda, kTileK)
                 : make_map(&ta, a.a, a.M, a.K, a.lda, kTileM);
    if (e != cudaSuccess) return e;
  }
  if (p.b_tma && p.ktiles > 0) {
    e = p.b_cut ? make_cut_map(&tb, a.b, a.K, a.N, a.ldb, brows / 64)
        : a.b_mn ? make_map(&tb, a.b, a.K, a.N, a.ldb, kTileK)
                 : make_map(&tb, a.b, a.N, a.K, a.ldb, brows);
    if (e != cudaSuccess) return e;
  }
  const int64_t tiles = p.tiles_m * p.tiles_n;
  const int ctas = PAIR ? 2 : p.split;
  const int64_t workers = p.split > 1 || tiles < p.slots ? tiles : p.slots, grid = workers * ctas;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(S::kWarps * 32);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(ctas);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_linear<BN, LOADERS, PAIR, EPI>, ta, tb, p);
}

// Kernels of 128 columns and more come in kinds; those with loaders in all but the forward one.
template <int BN, bool LOADERS, bool PAIR>
cudaError_t launch(const Params& p, cudaStream_t s) {
  const LinearArgs& a = p.a;
  const bool affine = a.col_scale != nullptr || a.col_shift != nullptr, more = a.residual != nullptr || a.z_codes != nullptr;
  const bool forward = a.act != LOCO_ACT_NONE || a.save_codes != nullptr;
  if constexpr (BN >= 128) {
    if (!more && !forward && !affine) return launch_kind<BN, LOADERS, PAIR, kPlain>(p, s);
    if constexpr (LOADERS)
      if (!more && !forward) return launch_kind<BN, LOADERS, PAIR, kWeight>(p, s);
    if constexpr (!LOADERS)
      if (!more && !affine) return launch_kind<BN, LOADERS, PAIR, kForward>(p, s);
  }
  return launch_kind<BN, LOADERS, PAIR, kAny>(p, s);
}

// Clusters of 1, 2, 4 and 8 CTAs of these kernels (one CTA per SM) that the current device holds at
// once: fewer than its SMs would make up, as a cluster lies within one group of SMs.
cudaError_t cluster_slots(int (&slots)[4]) {
  static std::atomic<int> known[64][4];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  using S = Shape<64, false, false, kAny>;
  for (int i = 0; i < 4; ++i) {
    if (dev < 64 && (slots[i] = known[dev][i].load(std::memory_order_relaxed)) > 0) continue;
    e = cudaFuncSetAttribute(k_linear<64, false, false, kAny>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(S::kSmem));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(8 * 64);
    cfg.blockDim = dim3(S::kWarps * 32);
    cfg.dynamicSmemBytes = S::kSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1u << i;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaOccupancyMaxActiveClusters(&slots[i], k_linear<64, false, false, kAny>, &cfg)) != cudaSuccess) return e;
    if (slots[i] < 1) slots[i] = 1;
    if (dev < 64) known[dev][i].store(slots[i], std::memory_order_relaxed);
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t s) {
  cudaError_t e;
  Params p{};
  p.a = a;
  p.a_tma = a.a_codes == nullptr && tma_can(a.a, a.a_mn ? a.K : a.M, a.lda);
  p.b_tma = tma_can(a.b, a.b_mn ? a.K : a.N, a.ldb);
  p.ktiles = int((a.K + kTileK - 1) / kTileK);
  if (p.ktiles == 0) p.a_tma = p.b_tma = 1;  // nothing is read
  p.wait_ns = 2000000000ull + uint64_t(p.ktiles) * 20000ull;
  const size_t oe = a.out_bf16 ? 2 : 4;
  p.out_wide = reinterpret_cast<uintptr_t>(a.out) % 16 == 0 && (a.N <= 1 || a.ldo * oe % 16 == 0);
  p.res_wide = reinterpret_cast<uintptr_t>(a.residual) % 16 == 0 && (a.N <= 1 || a.ldr * oe % 16 == 0);
  const bool loaders = !p.a_tma || !p.b_tma;

  int slots[4];  // clusters of 1, 2, 4, 8 CTAs that the device runs at once
  if ((e = cluster_slots(slots)) != cudaSuccess) return e;
  // Few rows of x and rows of w enough for every SM (1 row, 11008 x 4096: 24.8 us with tensor cores).
  if (!a.a_mn && !a.b_mn && !loaders && a.N <= 4 && p.ktiles > 0 && a.M >= 32 * 76) {
    p.split = 1;
    return launch_rows(p, slots[0], s);
  }

  // The tile's width, the split of k or the pairing of CTAs that finish first by this estimate (in
  // units of a 256-wide tile's 64 k): waves x (each part's k tiles at the width's rate + a fixed cost
  // of filling the pipeline and of the epilogue).
  int best_bn = 0, best_split = 1;
  bool best_pair = false;
  double best = 0.0;
  const auto consider = [&](int bn, int split, bool pair) {
    const int64_t tm = (a.M + (pair ? 2 : 1) * kTileM - 1) / ((pair ? 2 : 1) * kTileM), tn = (a.N + bn - 1) / bn;
    const int64_t tiles = tm * tn, most = slots[pair || split == 2 ? 1 : split == 4 ? 2 : split == 8 ? 3 : 0];
    if (split > 1 && (p.ktiles < 2 * split || tiles > most)) return;
    // B's boxes along n are 64 wide: with parts of boxes, lines are fetched twice (8192 x 14336 x 4096
    // weight gradient at 224: 705 us, at 256: 577 us)
    if (a.b_mn && bn % (pair ? 128 : 64) != 0) return;
    const double waves = double((tiles + most - 1) / most);
    const double per_k = (bn < 64 ? 0.35 : 0.2 + bn / 320.0) * (pair ? 0.85 : 1.0);
    const double t = waves * (double((p.ktiles + split - 1) / split) * per_k + 4.0 + bn / 64.0 + (split > 1 || pair ? 3.0 : 0.0));
    if (best_bn == 0 || t < best) best = t, best_bn = bn, best_split = split, best_pair = pair;
  };
  // Widths between the kernels' own fill a last wave better (4096 x 4096 x 4096 at 224: 4 whole waves).
  static const int widths[] = {16, 32, 64, 128, 160, 192, 224, 256};
  for (const int bn : widths) {
    if (bn < 64 && (a.b_mn || loaders)) continue;
    if (bn > 64 && bn / 2 >= a.N) continue;  // more than half of it would be empty
    for (int split = 1; split <= 8; split *= 2) consider(bn, split, false);
    if (bn > 128 && !loaders) consider(bn, 1, true);
  }
  p.split = best_split;
  p.bn = best_bn;
  p.slots = slots[best_pair ? 1 : 0];
  p.tiles_m = (a.M + (best_pair ? 2 : 1) * kTileM - 1) / ((best_pair ? 2 : 1) * kTileM);
  p.tiles_n = (a.N + best_bn - 1) / best_bn;
  if (best_pair) return launch<256, false, true>(p, s);
  if (loaders) {
    switch (best_bn) {
      case 64: return launch<64, true, false>(p, s);
      case 128: return launch<128, true, false>(p, s);
      default: return launch<256, true, false>(p, s);
    }
  }
  switch (best_bn) {
    case 16: return launch<16, false, false>(p, s);
    case 32: return launch<32, false, false>(p, s);
    case 64: return launch<64, false, false>(p, s);
    case 128: return launch<128, false, false>(p, s);
    default: return launch<256, false, false>(p, s);
  }
}

// ------------------------------------------------------------------ column sums (the bias's gradient)

namespace {

// 64 columns per CTA: 8 lanes of 8 columns (one 16-byte load), 4 rows per warp, 16 warps; the CTAs of
// a cluster share the rows, and the first adds their sums in order.  Bound by memory: 4 loads per
// lane are kept in flight.
constexpr int kSumWarps = 16, kSumRows = kSumWarps * 4;

__global__ void __launch_bounds__(kSumWarps * 32) k_col_sum(ColSumArgs a, int parts) {
  __shared__ float sm[kSumWarps][64];
  __shared__ float part[64];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int rank = parts > 1 ? int(cluster_rank()) : 0;
  const int64_t c = int64_t(blockIdx.x / parts) * 64 + (lane & 7) * 8;
  const int64_t lo = a.rows * rank / parts, hi = a.rows * (rank + 1) / parts;
  const uint16_t* x = static_cast<const uint16_t*>(a.x);
  float s[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) s[k] = 0.0f;
  if (c + 8 <= a.cols && reinterpret_cast<uintptr_t>(x) % 16 == 0 && a.ldx % 8 == 0) {
    int64_t r = lo + warp * 4 + lane / 8;
    for (; r + 3 * kSumRows < hi; r += 4 * kSumRows) {
      uint4 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(x + (r + i * kSumRows) * a.ldx + c));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          s[2 * k] += __uint_as_float(u[k] << 16);
          s[2 * k + 1] += __uint_as_float(u[k] & 0xFFFF0000u);
        }
      }
    }
    for (; r < hi; r += kSumRows) {
      float v[8];
      load8(x, r * a.ldx + c, 1, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) s[k] += v[k];
    }
  } else {
#pragma unroll 2
    for (int64_t r = lo + warp * 4 + lane / 8; r < hi; r += kSumRows) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (c + k < a.cols) s[k] += bf16_bits_to_f32(__ldg(x + r * a.ldx + c + k));
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    s[k] += __shfl_xor_sync(0xFFFFFFFFu, s[k], 8);
    s[k] += __shfl_xor_sync(0xFFFFFFFFu, s[k], 16);
    if (lane < 8) sm[warp][lane * 8 + k] = s[k];
  }
  __syncthreads();
  float v = 0.0f;
  if (threadIdx.x < 64) {
#pragma unroll
    for (int w = 0; w < kSumWarps; ++w) v += sm[w][threadIdx.x];
    part[threadIdx.x] = v;
  }
  const int64_t col = int64_t(blockIdx.x / parts) * 64 + threadIdx.x;
  if (parts > 1) {
    cluster_sync();
    if (rank == 0 && threadIdx.x < 64) {
      v = 0.0f;
      for (int r = 0; r < parts; ++r) v += cluster_load(cluster_addr(smem_u32(&part[threadIdx.x]), uint32_t(r)));
    }
    cluster_sync();
  }
  if (rank == 0 && threadIdx.x < 64 && col < a.cols) {
    if (a.sum_f32 != nullptr) a.sum_f32[col] = v;
    if (a.out != nullptr) store_elem(a.out, col, a.out_bf16, v);
  }
}

}  // namespace

cudaError_t launch_col_sum(const ColSumArgs& a, cudaStream_t s) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int64_t strips = (a.cols + 63) / 64;
  int parts = 1;
  while (parts < 8 && strips * parts < 4 * sms && a.rows >= int64_t(parts) * 2 * kSumRows) parts *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(strips * parts));
  cfg.blockDim = dim3(kSumWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(parts);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_col_sum, a, parts);
}

cudaError_t read_linear_timeouts(int64_t* count) {
  unsigned long long v = 0;
  const cudaError_t e = cudaMemcpyFromSymbol(&v, g_timeouts, sizeof v);
  if (e == cudaSuccess) *count = int64_t(v);
  return e;
}

}  // namespace loco
