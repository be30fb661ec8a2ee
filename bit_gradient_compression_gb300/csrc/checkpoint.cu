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

// Eight values per thread; groups of 8 values number nb*4 per row (those past cols are padding).
template <bool BF16>
__global__ void __launch_bounds__(kThreads) k_encode_wide(EncodeArgs a, int64_t groups_per_row, int64_t groups) {
  // every thread of a warp stays in the loop together: the bound is rounded up to a warp's 32 groups
  const int64_t step = int64_t(gridDim.x) * kThreads;
  for (int64_t g = int64_t(blockIdx.x) * kThreads + threadIdx.x; g < (groups + 31) / 32 * 32; g += step) {
    const bool live = g < groups;
    const int64_t row = live ? g / groups_per_row : 0;
    const int64_t col = (g - row * groups_per_row) * 8;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.0f;
    if (live && col + 8 <= a.cols) {
      load8(a.x, row * a.ldx + col, BF16, v);
    } else if (live) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (col + k < a.cols) v[k] = load_elem(a.x, row * a.ldx + col + k, BF16);
    }
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, mag_bits(v[k]));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    if (!live) continue;
    reinterpret_cast<uint2*>(a.codes)[g] = ckpt_pack8(v, m);
    if ((g & 3) == 0) a.scales[g >> 2] = uint8_t(ckpt_scale(m));
  }
}

// One value per lane, a block per warp.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) k_encode_narrow(EncodeArgs a, int64_t nb, int64_t blocks) {
  const int lane = threadIdx.x & 31;
  const int64_t step = int64_t(gridDim.x) * (kThreads / 32);
  for (int64_t b = int64_t(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32; b < blocks; b += step) {
    const int64_t row = b / nb, col = (b - row * nb) * kCkptBlock + lane;
    const float v = col < a.cols ? load_elem(a.x, row * a.ldx + col, BF16) : 0.0f;
    const uint32_t sc = ckpt_scale(__reduce_max_sync(0xFFFFFFFFu, mag_bits(v)));
    a.codes[b * kCkptBlock + lane] = int8_t(ckpt_code(v, ckpt_inv_step(sc)));
    if (lane == 0) a.scales[b] = uint8_t(sc);
  }
}

// Sixteen codes per thread (half a block).  WIDE: rows of out start on 16-byte boundaries.
template <bool BF16, bool WIDE>
__global__ void __launch_bounds__(kThreads) k_decode(DecodeArgs a, int64_t halves_per_row, int64_t halves) {
  const int64_t step = int64_t(gridDim.x) * kThreads;
  for (int64_t h = int64_t(blockIdx.x) * kThreads + threadIdx.x; h < halves; h += step) {
    const int64_t row = h / halves_per_row, col = (h - row * halves_per_row) * 16;
    if (col >= a.cols) continue;
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(a.codes) + h);
    const float st = ckpt_step(__ldg(a.scales + (h >> 1)));
    float v[16];
    ckpt_unpack4(w.x, st, v);
    ckpt_unpack4(w.y, st, v + 4);
    ckpt_unpack4(w.z, st, v + 8);
    ckpt_unpack4(w.w, st, v + 12);
    if (a.gamma != nullptr || a.beta != nullptr) {
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if (col + k < a.cols)
          v[k] = fmaf(v[k], a.gamma ? load_elem(a.gamma, col + k, a.param_bf16) : 1.0f,
                      a.beta ? load_elem(a.beta, col + k, a.param_bf16) : 0.0f);
    }
    if (a.act != LOCO_ACT_NONE) {
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] = act_value(v[k], a.act);
    }
    const int64_t at = row * a.ldo + col;
    if (WIDE && col + 16 <= a.cols) {
      store8(a.out, at, BF16, v);
      store8(a.out, at + 8, BF16, v + 8);
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if (col + k < a.cols) store_elem(a.out, at + k, BF16, v[k]);
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

cudaError_t launch_ckpt_encode(const EncodeArgs& a, cudaStream_t s) {
  const int64_t nb = (a.cols + kCkptBlock - 1) / kCkptBlock;
  unsigned grid;
  cudaError_t e;
  if (wide_rows(a.x, a.ldx, a.rows, a.x_bf16)) {
    const int64_t groups = a.rows * nb * 4;
    if ((e = grid_for(groups, kThreads, &grid)) != cudaSuccess) return e;
    (a.x_bf16 ? k_encode_wide<true> : k_encode_wide<false>)<<<grid, kThreads, 0, s>>>(a, nb * 4, groups);
  } else {
    if ((e = grid_for(a.rows * nb, kThreads / 32, &grid)) != cudaSuccess) return e;
    (a.x_bf16 ? k_encode_narrow<true> : k_encode_narrow<false>)<<<grid, kThreads, 0, s>>>(a, nb, a.rows * nb);
  }
  return cudaGetLastError();
}

cudaError_t launch_ckpt_decode(const DecodeArgs& a, cudaStream_t s) {
  const int64_t nb = (a.cols + kCkptBlock - 1) / kCkptBlock, halves = a.rows * nb * 2;
  unsigned grid;
  const cudaError_t e = grid_for(halves, kThreads, &grid);
  if (e != cudaSuccess) return e;
  if (wide_rows(a.out, a.ldo, a.rows, a.out_bf16))
    (a.out_bf16 ? k_decode<true, true> : k_decode<false, true>)<<<grid, kThreads, 0, s>>>(a, nb * 2, halves);
  else
    (a.out_bf16 ? k_decode<true, false> : k_decode<false, false>)<<<grid, kThreads, 0, s>>>(a, nb * 2, halves);
  return cudaGetLastError();
}

}  // namespace loco
