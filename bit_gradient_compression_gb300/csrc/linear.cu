// The products of a linear layer's forward and backward passes, with their
// epilogues, on the fifth-generation tensor cores.
//
// All three are D[n][m] = sum_k A[m][k] B[n][k] with m along the output's
// contiguous columns and n along its rows:
//   forward          y[t][n]  = x w^T       m = n (rows of w),     n = t, k = k
//   input gradient   dx[t][k] = dy w        m = k (columns of w),  n = t, k = n
//   weight gradient  dw[n][k] = dy^T x      m = k (columns of x),  n = n, k = t
// A CTA computes tiles of 128 m by BN n, 64 k at a time.  Operands whose memory
// runs along k, or along m or n, are both taken as they lie (the tensor core's
// operand descriptors name the direction), so nothing is transposed.  An output
// row's 32 consecutive columns are the 32 lanes of a warp of the epilogue: its
// loads and stores are whole sectors, and a checkpoint block is one warp
// reduction.
//
// Warps: 0 issues TMA loads, 1 issues products, 4..7 run the epilogue out of
// tensor memory (two accumulators, so it overlaps the next tile's products),
// and, in the LOADERS kernels, 8..15 write operands that TMA cannot fetch into
// the same swizzled layout: rows that start on no 16-byte boundary, and
// checkpoints, which they turn into bf16 (exactly, as steps are powers of two).
//
// Few tiles and a long k: `split` CTAs of a cluster share a tile, each with a
// part of k; they leave their partial tiles in shared memory, and each adds up,
// in the order of the parts, the columns it then finishes.
#include <atomic>

#include "layers_common.cuh"
#include "tensor_core.cuh"

namespace loco {

namespace {

constexpr int kTileM = 128, kTileK = 64;
constexpr int kLoadWarps = 8;

__device__ unsigned long long g_timeouts;

template <int BN>
struct Shape {
  static constexpr int kABytes = kTileM * kTileK * 2, kBBytes = BN * kTileK * 2, kStage = kABytes + kBBytes;
  static constexpr int kStages = 200 * 1024 / kStage;
  static constexpr int kTmemCols = 2 * BN < 32 ? 32 : 2 * BN;
  static constexpr size_t kSmem = 1024 + size_t(kStages) * kStage + 256;
};

struct Params {
  LinearArgs a;
  int a_tma, b_tma;
  int64_t tiles_m, tiles_n;
  int ktiles, split;
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

// Byte offset of 16-byte unit u of row r of a tile whose rows run along k (128 bytes each), or of
// unit u (8 values along m or n) of k-row r: 64-value chunks of 64 rows.
__device__ __forceinline__ uint32_t unit_offset(int mn, int r, int u) {
  return (mn ? uint32_t(u >> 3) * (kTileK * 128) : 0u) + uint32_t(r) * 128 + uint32_t(((u & 7) ^ (r & 7)) << 4);
}

__device__ __forceinline__ void st_shared16(uint32_t dst, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// A tile of ROWS (m or n) x 64 (k) bf16 values by plain loads; 0 outside the matrix.
template <int ROWS>
__device__ __forceinline__ void fill_plain(uint32_t dst, const void* src, int64_t ld, int mn, int64_t row0,
                                           int64_t rows, int64_t k0, int64_t ks, int tid) {
  constexpr int kItems = ROWS * 8;  // 16-byte units
  const int per = mn ? ROWS / 8 : 8;
  const int64_t r0 = mn ? k0 : row0, rlim = mn ? ks : rows, c0 = mn ? row0 : k0, clim = mn ? rows : ks;
  const uint16_t* base = static_cast<const uint16_t*>(src);
#pragma unroll 2
  for (int i = tid; i < kItems; i += kLoadWarps * 32) {
    const int r = i / per, u = i - r * per;
    const int64_t row = r0 + r, col = c0 + u * 8;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row < rlim && col < clim) {
      const uint16_t* q = base + row * ld + col;
      if (col + 8 <= clim && (reinterpret_cast<uintptr_t>(q) & 15) == 0) {
        v = __ldg(reinterpret_cast<const uint4*>(q));
      } else {
        uint32_t h[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) h[k] = col + k < clim ? uint32_t(__ldg(q + k)) : 0u;
        v = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
      }
    }
    st_shared16(dst + unit_offset(mn, r, u), v);
  }
}

// A tile of 128 (m) x 64 (k) values of a checkpoint [k][m]; 0 outside it.
__device__ __forceinline__ void fill_ckpt(uint32_t dst, const int8_t* codes, const uint8_t* scales, int64_t nb,
                                          int64_t m0, int64_t k0, int64_t ks, int tid) {
#pragma unroll
  for (int i = tid; i < kTileM / 16 * kTileK; i += kLoadWarps * 32) {
    const int r = i / 8, h = i % 8;  // k row, 16 codes along m
    const int64_t blk = m0 / kCkptBlock + h / 2;
    uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
    if (k0 + r < ks && blk < nb) {
      const int64_t at = (k0 + r) * nb + blk;
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(codes + at * kCkptBlock) + (h & 1));
      const float st = ckpt_step(__ldg(scales + at));
      float v[16];
      ckpt_unpack4(w.x, st, v), ckpt_unpack4(w.y, st, v + 4), ckpt_unpack4(w.z, st, v + 8), ckpt_unpack4(w.w, st, v + 12);
      lo = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
      hi = make_uint4(pack_bf16x2(v[8], v[9]), pack_bf16x2(v[10], v[11]), pack_bf16x2(v[12], v[13]),
                      pack_bf16x2(v[14], v[15]));
    }
    st_shared16(dst + unit_offset(1, r, 2 * h), lo);
    st_shared16(dst + unit_offset(1, r, 2 * h + 1), hi);
  }
}

// ------------------------------------------------------------------ epilogue

// What belongs to the thread's output column m.
struct Column {
  int64_t m;
  bool live;
  float scale, shift, bias;
};

__device__ __forceinline__ Column column_of(const LinearArgs& a, int64_t m) {
  Column c{m, m < a.M, 1.0f, 0.0f, 0.0f};
  if (c.live) {
    if (a.col_scale != nullptr) c.scale = load_elem(a.col_scale, m, a.param_bf16);
    if (a.col_shift != nullptr) c.shift = load_elem(a.col_shift, m, a.param_bf16);
    if (a.bias != nullptr) c.bias = load_elem(a.bias, m, a.param_bf16);
  }
  return c;
}

// NJ output rows n0 .. n0 + count (a warp-uniform count) of the thread's column; every lane takes part.
template <int NJ>
__device__ __forceinline__ void finish(const LinearArgs& a, const Column& c, float (&v)[NJ], int64_t n0, int count) {
  const int64_t nb = (a.M + kCkptBlock - 1) / kCkptBlock, blk = c.m / kCkptBlock;
  float res[NJ], z[NJ];
  if (a.residual != nullptr) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      res[j] = c.live && j < count ? load_elem_rw(a.residual, (n0 + j) * a.ldr + c.m, a.out_bf16) : 0.0f;
  }
  if (a.z_codes != nullptr) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      z[j] = 0.0f;
      if (c.live && j < count) {
        const int64_t at = (n0 + j) * nb + blk;
        z[j] = float(__ldg(a.z_codes + at * kCkptBlock + (c.m & 31))) * ckpt_step(__ldg(a.z_scales + at));
      }
    }
  }
  if (a.col_scale != nullptr) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) v[j] *= c.scale;
  }
  if (a.col_shift != nullptr) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if (j < count) v[j] = fmaf(c.shift, __ldg(a.row_sum + n0 + j), v[j]);
  }
  if (a.bias != nullptr) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) v[j] += c.bias;
  }
  if (a.save_codes != nullptr && blk < nb) {  // uniform: a warp's 32 columns are one block
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      if (j >= count) continue;
      const uint32_t sc = ckpt_scale(__reduce_max_sync(0xFFFFFFFFu, c.live ? mag_bits(v[j]) : 0u));
      const int64_t at = (n0 + j) * nb + blk;
      a.save_codes[at * kCkptBlock + (c.m & 31)] = c.live ? int8_t(ckpt_code(v[j], ckpt_inv_step(sc))) : int8_t(0);
      if ((c.m & 31) == 0) a.save_scales[at] = uint8_t(sc);
    }
  }
  if (a.z_codes != nullptr) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) v[j] *= act_slope(z[j], a.act);
  } else if (a.act != LOCO_ACT_NONE) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) v[j] = act_value(v[j], a.act);
  }
  if (a.residual != nullptr) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) v[j] += res[j];
  }
  if (c.live) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if (j < count) store_elem(a.out, (n0 + j) * a.ldo + c.m, a.out_bf16, v[j]);
  }
}

// ------------------------------------------------------------------ the kernel

template <int BN, bool LOADERS>
__global__ void __launch_bounds__(LOADERS ? 256 + kLoadWarps * 32 : 256, 1)
    k_linear(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
             const __grid_constant__ Params p) {
  using S = Shape<BN>;
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
  const int rank = p.split > 1 ? int(cluster_rank()) : 0;
  const int64_t workers = gridDim.x / p.split, worker = blockIdx.x / p.split;
  const int64_t tiles = p.tiles_m * p.tiles_n;
  const int kt0 = int(int64_t(p.ktiles) * rank / p.split), kt1 = int(int64_t(p.ktiles) * (rank + 1) / p.split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(full(s), 1 + (LOADERS ? kLoadWarps : 0));
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), 4);
    }
    mbar_init(drain, 1);
    mbar_init_fence();
    if (p.a_tma) tma_prefetch_map(&ta);
    if (p.b_tma) tma_prefetch_map(&tb);
  }
  if (warp == 2) tmem_alloc(tmem_at, S::kTmemCols);
  tc_fence_before();
  __syncthreads();
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
      const int m0 = int(tm * kTileM), n0 = int(tn * BN);
      for (int kt = kt0; kt < kt1; ++kt) {
        if (!mbar_wait(empty(stage), phase ^ 1, p.wait_ns)) {
          gave_up = true;
          break;
        }
        const uint32_t sa = base + stage * S::kStage, sb = sa + S::kABytes;
        const int k0 = kt * kTileK;
        mbar_arrive_expect(full(stage), (p.a_tma ? S::kABytes : 0) + (p.b_tma ? S::kBBytes : 0));
        if (p.a_tma) {
          if (!p.a.a_mn) {
            tma_load_2d(sa, &ta, k0, m0, full(stage));
          } else {
#pragma unroll
            for (int c = 0; c < kTileM / 64; ++c)
              tma_load_2d(sa + c * (kTileK * 128), &ta, m0 + c * 64, k0, full(stage));
          }
        }
        if (p.b_tma) {
          if (!p.a.b_mn) {
            tma_load_2d(sb, &tb, k0, n0, full(stage));
          } else {
#pragma unroll
            for (int c = 0; c < (BN < 64 ? 1 : BN / 64); ++c)
              tma_load_2d(sb + c * (kTileK * 128), &tb, n0 + c * 64, k0, full(stage));
          }
        }
        ++issued;
        if (++stage == S::kStages) stage = 0, phase ^= 1;
      }
    }
    if (gave_up) {
      // let the copies in flight land before the CTA ends
      for (int i = 0; i < S::kStages && i < issued; ++i) {
        if (--stage < 0) stage = S::kStages - 1, phase ^= 1;
        if (!mbar_wait(full(stage), phase, p.wait_ns)) break;
      }
    }
  } else if (warp == 1 && lane == 0) {
    // ---- products
    const uint32_t desc = mma_desc(kTileM, BN, p.a.a_mn, p.a.b_mn);
    const uint32_t chunk = kTileK * 128;
    const uint64_t astep = p.a.a_mn ? 2048 / 16 : 32 / 16, bstep = p.a.b_mn ? 2048 / 16 : 32 / 16;
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
        tc_fence_after();
        const uint32_t sa = base + stage * S::kStage;
        const uint64_t da = smem_desc(sa, chunk), db = smem_desc(sa + S::kABytes, chunk);
#pragma unroll
        for (int k = 0; k < kTileK / 16; ++k) mma_bf16(d, da + k * astep, db + k * bstep, desc, kt > kt0 || k > 0);
        mma_commit(empty(stage));
        if (++stage == S::kStages) stage = 0, phase ^= 1;
      }
      if (gave_up) break;
      mma_commit(acc_full(buf));
      buf ^= 1;
      if (buf == 0) bphase ^= 1;
    }
    if (gave_up) {
      mma_commit(drain);
      mbar_wait(drain, 0, p.wait_ns);
    }
  } else if (warp >= 4 && warp < 8) {
    // ---- epilogue: lane i of warp 4 + q holds row q*32 + i of the accumulator
    const int q = warp - 4;
    int buf = 0, bphase = 0;
    for (int64_t tile = worker; tile < tiles; tile += workers) {
      int64_t tm, tn;
      tile_at(p, tile, &tm, &tn);
      const Column col = column_of(p.a, tm * kTileM + q * 32 + lane);
      const int64_t n0 = tn * BN;
      const int rows = int(min(int64_t(BN), p.a.N - n0));
      if (kt0 < kt1) {
        if (!warp_wait(acc_full(buf), bphase, p.wait_ns)) {
          gave_up = true;
          break;
        }
        tc_fence_after();
      }
#pragma unroll 1
      for (int j = 0; j < rows; j += 16) {
        uint32_t w[16];
        if (kt0 < kt1) {
          tmem_load16(tmem + buf * BN + j + (uint32_t(q * 32) << 16), w);
          tmem_wait_loads();
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = 0;
        }
        if (j + 16 >= rows && kt0 < kt1) {
          // the accumulator has been read: the next tile but one may overwrite it
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(acc_empty(buf));
        }
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(w[i]);
        if (p.split > 1) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(base + uint32_t(((j + i) * kTileM + q * 32 + lane) * 4)), "f"(v[i])
                         : "memory");
        } else {
          finish<16>(p.a, col, v, n0 + j, min(16, rows - j));
        }
      }
      buf ^= 1;
      if (buf == 0) bphase ^= 1;
    }
  } else if (LOADERS && warp >= 8) {
    // ---- plain loads and checkpoints
    const int tid = threadIdx.x - 256;
    const int64_t nb = (p.a.M + kCkptBlock - 1) / kCkptBlock;
    int stage = 0, phase = 0;
    for (int64_t tile = worker; tile < tiles && !gave_up; tile += workers) {
      int64_t tm, tn;
      tile_at(p, tile, &tm, &tn);
      for (int kt = kt0; kt < kt1; ++kt) {
        if (!warp_wait(empty(stage), phase ^ 1, p.wait_ns)) {
          gave_up = true;
          break;
        }
        const uint32_t sa = base + stage * S::kStage, sb = sa + S::kABytes;
        const int64_t k0 = int64_t(kt) * kTileK;
        if (!p.a_tma) {
          if (p.a.a_codes != nullptr)
            fill_ckpt(sa, p.a.a_codes, p.a.a_scales, nb, tm * kTileM, k0, p.a.K, tid);
          else
            fill_plain<kTileM>(sa, p.a.a, p.a.lda, p.a.a_mn, tm * kTileM, p.a.M, k0, p.a.K, tid);
        }
        if (!p.b_tma) fill_plain<BN>(sb, p.a.b, p.a.ldb, p.a.b_mn, tn * BN, p.a.N, k0, p.a.K, tid);
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(full(stage));
        if (++stage == S::kStages) stage = 0, phase ^= 1;
      }
    }
  }
  if (gave_up && lane == 0) atomicAdd(&g_timeouts, 1ull);
  __syncwarp();

  if (p.split > 1) {
    // One tile per cluster.  Its parts lie in the CTAs' shared memory as [n][m]; each CTA adds up
    // and finishes its share of the rows.
    cluster_sync();
    int64_t tm, tn;
    tile_at(p, worker, &tm, &tn);
    const int q = warp & 3, side = warp / 4, sides = LOADERS ? 4 : 2;
    const Column col = column_of(p.a, tm * kTileM + q * 32 + lane);
    const int64_t n0 = tn * BN;
    const int rows = int(min(int64_t(BN), p.a.N - n0));
    const int share = (rows + p.split - 1) / p.split, lo = share * rank, hi = min(rows, lo + share);
    for (int j = lo + side * 4; j < hi; j += sides * 4) {
      float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int r = 0; r < p.split; ++r) {
        const uint32_t at = cluster_addr(base + uint32_t((j * kTileM + q * 32 + lane) * 4), uint32_t(r));
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = cluster_load(at + (j + i < hi ? i : 0) * (kTileM * 4));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += w[i];
      }
      finish<4>(p.a, col, v, n0 + j, min(4, hi - j));
    }
    cluster_sync();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) tmem_free(tmem, S::kTmemCols);
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

template <int BN, bool LOADERS>
cudaError_t launch(const Params& p, int sms, cudaStream_t s) {
  using S = Shape<BN>;
  static std::atomic<bool> ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(k_linear<BN, LOADERS>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(S::kSmem));
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev].store(true, std::memory_order_release);
  }
  CUtensorMap ta{}, tb{};
  const LinearArgs& a = p.a;
  if (p.a_tma && p.ktiles > 0) {
    e = a.a_mn ? make_map(&ta, a.a, a.K, a.M, a.lda, kTileK) : make_map(&ta, a.a, a.M, a.K, a.lda, kTileM);
    if (e != cudaSuccess) return e;
  }
  if (p.b_tma && p.ktiles > 0) {
    e = a.b_mn ? make_map(&tb, a.b, a.K, a.N, a.ldb, kTileK) : make_map(&tb, a.b, a.N, a.K, a.ldb, BN);
    if (e != cudaSuccess) return e;
  }
  const int64_t tiles = p.tiles_m * p.tiles_n;
  const int64_t grid = p.split > 1 ? tiles * p.split : (tiles < sms ? tiles : sms);
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(LOADERS ? 256 + kLoadWarps * 32 : 256);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(p.split);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_linear<BN, LOADERS>, ta, tb, p);
}

}  // namespace

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t s) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  Params p{};
  p.a = a;
  p.a_tma = a.a_codes == nullptr && tma_can(a.a, a.a_mn ? a.K : a.M, a.lda);
  p.b_tma = tma_can(a.b, a.b_mn ? a.K : a.N, a.ldb);
  p.ktiles = int((a.K + kTileK - 1) / kTileK);
  if (p.ktiles == 0) p.a_tma = p.b_tma = 1;  // nothing is read
  p.wait_ns = 2000000000ull + uint64_t(p.ktiles) * 20000ull;
  const bool loaders = !p.a_tma || !p.b_tma;
  p.tiles_m = (a.M + kTileM - 1) / kTileM;

  // The tile's width and the split of k that finish first by this estimate (in units of a 256-wide
  // tile's 64 k): waves x (each part's k tiles at the width's rate + a fixed cost of filling the
  // pipeline and of the epilogue).
  static const int widths[] = {16, 32, 64, 128, 256};
  int best_bn = 0, best_split = 1;
  double best = 0.0;
  for (const int bn : widths) {
    if (bn < 64 && (a.b_mn || loaders)) continue;
    if (bn > 64 && bn / 2 >= a.N) continue;  // more than half of it would be empty
    const int64_t tn = (a.N + bn - 1) / bn, tiles = p.tiles_m * tn;
    for (int split = 1; split <= 8; split *= 2) {
      if (split > 1 && (p.ktiles < 2 * split || tiles * split > sms)) break;
      const double waves = double((tiles * split + sms - 1) / sms);
      const double per_k = bn >= 256 ? 1.0 : bn == 128 ? 0.6 : bn == 64 ? 0.4 : 0.35;
      const double t = waves * (double((p.ktiles + split - 1) / split) * per_k + 4.0 + bn / 64.0 + (split > 1 ? 3.0 : 0.0));
      if (best_bn == 0 || t < best) best = t, best_bn = bn, best_split = split;
    }
  }
  p.split = best_split;
  p.tiles_n = (a.N + best_bn - 1) / best_bn;
  if (loaders) {
    switch (best_bn) {
      case 64: return launch<64, true>(p, sms, s);
      case 128: return launch<128, true>(p, sms, s);
      default: return launch<256, true>(p, sms, s);
    }
  }
  switch (best_bn) {
    case 16: return launch<16, false>(p, sms, s);
    case 32: return launch<32, false>(p, sms, s);
    case 64: return launch<64, false>(p, sms, s);
    case 128: return launch<128, false>(p, sms, s);
    default: return launch<256, false>(p, sms, s);
  }
}

// ------------------------------------------------------------------ column sums (the bias's gradient)

namespace {

// 64 columns per CTA, its 16 warps each every 16th row of the CTA's share; the CTAs of a cluster
// share the rows, and the first adds their sums in order.
constexpr int kSumWarps = 16;

__global__ void __launch_bounds__(kSumWarps * 32) k_col_sum(ColSumArgs a, int parts) {
  __shared__ float sm[kSumWarps][64];
  __shared__ float part[64];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int rank = parts > 1 ? int(cluster_rank()) : 0;
  const int64_t c = int64_t(blockIdx.x / parts) * 64 + lane * 2;
  const int64_t lo = a.rows * rank / parts, hi = a.rows * (rank + 1) / parts;
  const uint16_t* x = static_cast<const uint16_t*>(a.x);
  float s0 = 0.0f, s1 = 0.0f;
  const bool pair = (reinterpret_cast<uintptr_t>(x) % 4 == 0) && a.ldx % 2 == 0 && c + 1 < a.cols;
  if (c < a.cols) {
#pragma unroll 4
    for (int64_t r = lo + warp; r < hi; r += kSumWarps) {
      const uint16_t* q = x + r * a.ldx + c;
      if (pair) {
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(q));
        s0 += __uint_as_float(w << 16);
        s1 += __uint_as_float(w & 0xFFFF0000u);
      } else {
        s0 += bf16_bits_to_f32(__ldg(q));
        if (c + 1 < a.cols) s1 += bf16_bits_to_f32(__ldg(q + 1));
      }
    }
  }
  sm[warp][lane * 2] = s0;
  sm[warp][lane * 2 + 1] = s1;
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
  while (parts < 8 && strips * parts < sms && a.rows >= int64_t(parts) * 2 * kSumWarps * 4) parts *= 2;
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
