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

// Eight values per thread and step, two steps in flight; groups of 8 values number nb*4 per row
// (those past cols are padding).  All 32 lanes stay in the loop together.
constexpr int kUnroll = 2;

template <bool BF16>
__global__ void __launch_bounds__(kThreads) k_encode_wide(EncodeArgs a, Divisor per_row, int64_t groups) {
  for (int64_t g0 = (int64_t(blockIdx.x) * kUnroll) * kThreads + threadIdx.x; g0 - (threadIdx.x & 31) < groups;
       g0 += int64_t(gridDim.x) * kUnroll * kThreads) {
    float v[kUnroll][8];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int64_t g = g0 + i * kThreads;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i][k] = 0.0f;
      if (g >= groups) continue;
      const int64_t row = divide(g, per_row), col = (g - row * per_row.d) * 8;
      if (col + 8 <= a.cols) {
        load8(a.x, row * a.ldx + col, BF16, v[i]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (col + k < a.cols) v[i][k] = load_elem(a.x, row * a.ldx + col + k, BF16);
      }
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int64_t g = g0 + i * kThreads;
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) m = max(m, mag_bits(v[i][k]));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      if (g >= groups) continue;
      reinterpret_cast<uint2*>(a.codes)[g] = ckpt_pack8(v[i], m);
      if ((g & 3) == 0) a.scales[g >> 2] = uint8_t(ckpt_scale(m));
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

// Sixteen codes per thread (half a block), for rows of out that start on 16-byte boundaries.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) k_decode_wide(DecodeArgs a, Divisor per_row, int64_t halves) {
  const int64_t step = int64_t(gridDim.x) * kThreads;
  for (int64_t h = int64_t(blockIdx.x) * kThreads + threadIdx.x; h < halves; h += step) {
    const int64_t row = divide(h, per_row), col = (h - row * per_row.d) * 16;
    if (col >= a.cols) continue;
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(a.codes) + h);
    const float st = ckpt_step(__ldg(a.scales + (h >> 1)));
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    const int64_t at = row * a.ldo + col;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t c = col + i * 8;
      float v[8];
      ckpt_unpack4(u[2 * i], st, v);
      ckpt_unpack4(u[2 * i + 1], st, v + 4);
      if (a.gamma != nullptr || a.beta != nullptr) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (c + k < a.cols)
            v[k] = fmaf(v[k], a.gamma ? load_elem(a.gamma, c + k, a.param_bf16) : 1.0f,
                        a.beta ? load_elem(a.beta, c + k, a.param_bf16) : 0.0f);
      }
      apply_act8(v, a.act);
      if (c + 8 <= a.cols) {
        store8(a.out, at + i * 8, BF16, v);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (c + k < a.cols) store_elem(a.out, at + i * 8 + k, BF16, v[k]);
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
    apply_act8(v, a.act);
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

cudaError_t grid_for(int64_t items, int per_block, unsigned* grid) {
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int64_t want = (items + per_block - 1) / per_block, most = int64_t(sms) * 8;
  *grid = unsigned(want < most ? want : most);
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_ckpt_encode(const EncodeArgs& in, cudaStream_t s) {
  EncodeArgs a = in;
  if (a.rows > 1 && a.ldx == a.cols && a.cols % kCkptBlock == 0) a.ldx = a.cols *= a.rows, a.rows = 1;  // one long row
  const int64_t nb = (a.cols + kCkptBlock - 1) / kCkptBlock;
  unsigned grid;
  cudaError_t e;
  if (wide_rows(a.x, a.ldx, a.rows, a.x_bf16)) {
    const int64_t groups = a.rows * nb * 4;
    if ((e = grid_for(groups, kThreads * kUnroll, &grid)) != cudaSuccess) return e;
    (a.x_bf16 ? k_encode_wide<true> : k_encode_wide<false>)<<<grid, kThreads, 0, s>>>(
        a, make_divisor(nb * 4, groups + int64_t(kThreads) * kUnroll), groups);
  } else {
    if ((e = grid_for(a.rows * nb, kThreads / 32 * kRun, &grid)) != cudaSuccess) return e;
    (a.x_bf16 ? k_encode_narrow<true> : k_encode_narrow<false>)<<<grid, kThreads, 0, s>>>(
        a, make_divisor(nb, a.rows * nb), a.rows * nb);
  }
  return cudaGetLastError();
}

cudaError_t launch_ckpt_decode(const DecodeArgs& in, cudaStream_t s) {
  DecodeArgs a = in;
  if (a.rows > 1 && a.ldo == a.cols && a.cols % kCkptBlock == 0 && a.gamma == nullptr && a.beta == nullptr)
    a.ldo = a.cols *= a.rows, a.rows = 1;  // one long row
  const int64_t nb = (a.cols + kCkptBlock - 1) / kCkptBlock;
  unsigned grid;
  cudaError_t e;
  if (wide_rows(a.out, a.ldo, a.rows, a.out_bf16)) {
    const int64_t halves = a.rows * nb * 2;
    if ((e = grid_for(halves, kThreads, &grid)) != cudaSuccess) return e;
    (a.out_bf16 ? k_decode_wide<true> : k_decode_wide<false>)<<<grid, kThreads, 0, s>>>(a, make_divisor(nb * 2, halves),
                                                                                       halves);
  } else {
    if ((e = grid_for(a.rows * nb, kThreads / 32 * kRun, &grid)) != cudaSuccess) return e;
    (a.out_bf16 ? k_decode_narrow<true> : k_decode_narrow<false>)<<<grid, kThreads, 0, s>>>(
        a, make_divisor(nb, a.rows * nb), a.rows * nb);
  }
  return cudaGetLastError();
}

}  // namespace loco
