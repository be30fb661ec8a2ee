// 8-bit activation checkpoints: a matrix to codes and scales, and back through
// an activation or a norm's scale and shift.
//
// Both are single passes bound by memory: bf16 values cost 2 + 1 + 1/32 bytes
// each way.  A block of 32 values spans 4 threads of 8 values (one or two
// 16-byte loads each), whose largest magnitude is two shuffles away; rows that
// no wide load can start on take one value per lane, a block per warp.
#include <atomic>

#include "layers_common.cuh"

namespace loco {

cudaError_t sm_count(int* sms) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (*sms = known[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
  e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && dev < 64) known[dev].store(*sms, std::memory_order_relaxed);
  return e;
}

cudaError_t layer_grid(LayerGrid& cache, const void* kernel, int threads, size_t smem_bytes, size_t smem_most, int* cap) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < LayerGrid::kDevices && (*cap = cache.cap[dev].load(std::memory_order_acquire)) > 0) return cudaSuccess;
  if (smem_most > 40 * 1024) {  // the default limit of 48 KB counts static shared memory too
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem_most));
    if (e != cudaSuccess) return e;
  }
  int sms = 0, per = 0;
  if ((e = sm_count(&sms)) != cudaSuccess) return e;
  if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, smem_bytes)) != cudaSuccess) return e;
  if (per <= 0) return cudaErrorInvalidConfiguration;
  *cap = sms * per;
  if (dev < LayerGrid::kDevices) cache.cap[dev].store(*cap, std::memory_order_release);
  return cudaSuccess;
}

namespace {

constexpr int kThreads = 256;

// A warp takes runs of kVec x 256 columns of a row, 8 columns a lane and vector: the position is worked
// out once per run, and kVec loads are in flight.  `runs` of them per row cover its padded blocks.
constexpr int kVec = 4, kRunCols = kVec * 256;

template <bool BF16>
__global__ void __launch_bounds__(kThreads) k_encode_wide(EncodeArgs a, Divisor per_row, int64_t nb, int64_t runs) {
  const int lane = threadIdx.x & 31;
  const int64_t step = int64_t(gridDim.x) * (kThreads / 32);
  for (int64_t i = int64_t(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32; i < runs; i += step) {
    const int64_t row = divide(i, per_row), c0 = (i - row * per_row.d) * kRunCols + lane * 8;
    const char* x = static_cast<const char*>(a.x) + (row * a.ldx + c0) * (BF16 ? 2 : 4);
    int8_t* codes = a.codes + row * nb * kCkptBlock + c0;
    uint8_t* scales = a.scales + row * nb + c0 / kCkptBlock;
    const int64_t left = a.cols - c0, pad = nb * kCkptBlock - c0;  // columns from the lane's first on
    float v[kVec][8];
    if (left >= kRunCols - 256 + 8) {
#pragma unroll
      for (int e = 0; e < kVec; ++e) load8(x, e * 256, BF16, v[e]);
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        if (left >= e * 256 + 8) {
          load8(x, e * 256, BF16, v[e]);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) v[e][k] = e * 256 + k < left ? load_elem(x, e * 256 + k, BF16) : 0.0f;
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      const uint32_t m = block_magnitude(v[e]);
      if (e * 256 < pad) {
        *reinterpret_cast<uint2*>(codes + e * 256) = ckpt_pack8(v[e], m);
        if ((lane & 3) == 0) scales[e * (256 / kCkptBlock)] = uint8_t(ckpt_scale(m));
      }
    }
  }
}

// One value per lane, a block per warp, kRun consecutive blocks at a time.
constexpr int kRun = 8;

template <bool BF16>
__global__ void __launch_bounds__(kThreads) k_encode_narrow(EncodeArgs a, Divisor per_row, int64_t blocks) {
  const int lane = threadIdx.x & 31;
  const int64_t step = int64_t(gridDim.x) * (kThreads / 32) * kRun;
  for (int64_t b0 = (int64_t(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32) * kRun; b0 < blocks; b0 += step) {
    int64_t row = divide(b0, per_row), blk = b0 - row * per_row.d;
    float v[kRun];
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const int64_t col = blk * kCkptBlock + lane;
      v[i] = b0 + i < blocks && col < a.cols ? load_elem(a.x, row * a.ldx + col, BF16) : 0.0f;
      if (++blk == per_row.d) blk = 0, ++row;
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      if (b0 + i >= blocks) continue;
      const uint32_t sc = ckpt_scale(__reduce_max_sync(0xFFFFFFFFu, mag_bits(v[i])));
      a.codes[(b0 + i) * kCkptBlock + lane] = int8_t(ckpt_code(v[i], ckpt_inv_step(sc)));
      if (lane == 0) a.scales[b0 + i] = uint8_t(sc);
    }
  }
}

// Runs as in k_encode_wide, for rows of out that start on 16-byte boundaries.  PLAIN: the values as they are.
template <bool BF16, bool PLAIN>
__global__ void __launch_bounds__(kThreads) k_decode_wide(DecodeArgs a, Divisor per_row, int64_t nb, int64_t runs) {
  const int lane = threadIdx.x & 31;
  const int64_t step = int64_t(gridDim.x) * (kThreads / 32);
  for (int64_t i = int64_t(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32; i < runs; i += step) {
    const int64_t row = divide(i, per_row), c0 = (i - row * per_row.d) * kRunCols + lane * 8;
    const int8_t* codes = a.codes + row * nb * kCkptBlock + c0;
    const uint8_t* scales = a.scales + row * nb + c0 / kCkptBlock;
    char* out = static_cast<char*>(a.out) + (row * a.ldo + c0) * (BF16 ? 2 : 4);
    const int64_t left = a.cols - c0;
    uint2 w[kVec];
    uint32_t sc[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      w[e] = make_uint2(0, 0);
      sc[e] = 1;
      if (e * 256 < left) {
        w[e] = __ldg(reinterpret_cast<const uint2*>(codes + e * 256));
        sc[e] = __ldg(scales + e * (256 / kCkptBlock));
      }
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      if (e * 256 >= left) continue;
      const bool full = e * 256 + 8 <= left;
      if (PLAIN && BF16 && full) {
        const uint32_t st = ckpt_step_bf16x2(sc[e]);
        const uint2 lo = decode4_bf16(w[e].x, st), hi = decode4_bf16(w[e].y, st);
        *reinterpret_cast<uint4*>(out + e * 512) = make_uint4(lo.x, lo.y, hi.x, hi.y);
        continue;
      }
      Pair p[4];
      float v[8];
      ckpt_pairs4(w[e].x, sc[e], p);
      ckpt_pairs4(w[e].y, sc[e], p + 2);
      floats8(p, v);
      if (!PLAIN) {
        if (a.gamma != nullptr || a.beta != nullptr) {
          const int64_t c = c0 + e * 256;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (c + k < a.cols)
              v[k] = fmaf(v[k], a.gamma ? load_elem(a.gamma, c + k, a.param_bf16) : 1.0f,
                          a.beta ? load_elem(a.beta, c + k, a.param_bf16) : 0.0f);
        }
        apply_act(v, a.act);
      }
      if (full) {
        store8(out, e * 256, BF16, v);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (e * 256 + k < left) store_elem(out, e * 256 + k, BF16, v[k]);
      }
    }
  }
}

// One value per lane, a block per warp, kRun consecutive blocks at a time.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) k_decode_narrow(DecodeArgs a, Divisor per_row, int64_t blocks) {
  const int lane = threadIdx.x & 31;
  const int64_t step = int64_t(gridDim.x) * (kThreads / 32) * kRun;
  for (int64_t b0 = (int64_t(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32) * kRun; b0 < blocks; b0 += step) {
    float v[kRun];
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      v[i] = 0.0f;
      if (b0 + i < blocks)
        v[i] = float(__ldg(a.codes + (b0 + i) * kCkptBlock + lane)) * ckpt_step(__ldg(a.scales + b0 + i));
    }
    int64_t row = divide(b0, per_row), blk = b0 - row * per_row.d;
    if (a.gamma != nullptr || a.beta != nullptr) {
      int64_t j = blk;
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        const int64_t col = j * kCkptBlock + lane;
        if (col < a.cols)
          v[i] = fmaf(v[i], a.gamma ? load_elem(a.gamma, col, a.param_bf16) : 1.0f,
                      a.beta ? load_elem(a.beta, col, a.param_bf16) : 0.0f);
        if (++j == per_row.d) j = 0;
      }
    }
    apply_act(v, a.act);
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const int64_t col = blk * kCkptBlock + lane;
      if (b0 + i < blocks && col < a.cols) store_elem(a.out, row * a.ldo + col, BF16, v[i]);
      if (++blk == per_row.d) blk = 0, ++row;
    }
  }
}

bool wide_rows(const void* p, int64_t ld, int64_t rows, int bf16) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows <= 1 || ld * (bf16 ? 2 : 4) % 16 == 0);
}

// As many CTAs as the device holds, or as the items fill.
template <typename Kernel>
cudaError_t grid_for(Kernel kernel, LayerGrid& cache, int64_t items, int per_block, unsigned* grid) {
  int cap = 0;
  const cudaError_t e = layer_grid(cache, reinterpret_cast<const void*>(kernel), kThreads, 0, 0, &cap);
  const int64_t want = (items + per_block - 1) / per_block;
  *grid = unsigned(want < cap ? want : cap);
  return e;
}

}  // namespace

cudaError_t launch_ckpt_encode(const EncodeArgs& in, cudaStream_t s) {
  static LayerGrid cache[4];
  EncodeArgs a = in;
  if (a.rows > 1 && a.ldx == a.cols && a.cols % kCkptBlock == 0) a.ldx = a.cols *= a.rows, a.rows = 1;  // one long row
  const int64_t nb = (a.cols + kCkptBlock - 1) / kCkptBlock;
  unsigned grid;
  if (wide_rows(a.x, a.ldx, a.rows, a.x_bf16)) {
    const int64_t per = (nb * kCkptBlock + kRunCols - 1) / kRunCols, runs = a.rows * per;
    const auto kernel = a.x_bf16 ? k_encode_wide<true> : k_encode_wide<false>;
    const cudaError_t e = grid_for(kernel, cache[a.x_bf16], runs, kThreads / 32, &grid);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kThreads, 0, s>>>(a, make_divisor(per, runs), nb, runs);
  } else {
    const int64_t blocks = a.rows * nb;
    const auto kernel = a.x_bf16 ? k_encode_narrow<true> : k_encode_narrow<false>;
    const cudaError_t e = grid_for(kernel, cache[2 + a.x_bf16], blocks, kThreads / 32 * kRun, &grid);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kThreads, 0, s>>>(a, make_divisor(nb, blocks), blocks);
  }
  return cudaGetLastError();
}

cudaError_t launch_ckpt_decode(const DecodeArgs& in, cudaStream_t s) {
  static LayerGrid cache[6];
  DecodeArgs a = in;
  const bool plain = a.act == LOCO_ACT_NONE && a.gamma == nullptr && a.beta == nullptr;
  if (a.rows > 1 && a.ldo == a.cols && a.cols % kCkptBlock == 0 && a.gamma == nullptr && a.beta == nullptr)
    a.ldo = a.cols *= a.rows, a.rows = 1;  // one long row
  const int64_t nb = (a.cols + kCkptBlock - 1) / kCkptBlock;
  unsigned grid;
  if (wide_rows(a.out, a.ldo, a.rows, a.out_bf16)) {
    const int64_t per = (a.cols + kRunCols - 1) / kRunCols, runs = a.rows * per;
    const auto kernel = a.out_bf16 ? (plain ? k_decode_wide<true, true> : k_decode_wide<true, false>)
                                   : (plain ? k_decode_wide<false, true> : k_decode_wide<false, false>);
    const cudaError_t e = grid_for(kernel, cache[a.out_bf16 * 2 + plain], runs, kThreads / 32, &grid);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kThreads, 0, s>>>(a, make_divisor(per, runs), nb, runs);
  } else {
    const int64_t blocks = a.rows * nb;
    const auto kernel = a.out_bf16 ? k_decode_narrow<true> : k_decode_narrow<false>;
    const cudaError_t e = grid_for(kernel, cache[4 + a.out_bf16], blocks, kThreads / 32 * kRun, &grid);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kThreads, 0, s>>>(a, make_divisor(nb, blocks), blocks);
  }
  return cudaGetLastError();
}

}  // namespace loco
