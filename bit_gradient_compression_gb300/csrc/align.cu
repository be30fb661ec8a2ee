// A bf16 matrix copied to rows that start on 16-byte boundaries, as the tensor
// memory accelerator wants a linear layer's operands.
//
// Bound by memory: 2 bytes read and 2 written a value.  A warp takes runs of 1024
// columns of a row, a lane 8 of every 256, with all its loads in flight.  Eight
// values that start on no 16-byte boundary are put together from the aligned
// sixteen bytes on either side (the upper ones are the next lane's lower ones,
// from L1); only where those would leave the matrix, at its very beginning and
// end, they go element by element.
#include "layers_common.cuh"

namespace loco {

namespace {

constexpr int kThreads = 256, kVec = 4, kRunCols = kVec * 256;

__global__ void __launch_bounds__(kThreads) k_align(AlignArgs a, Divisor per_row, int64_t runs) {
  const int lane = threadIdx.x & 31;
  const char* lo = static_cast<const char*>(a.src);
  const char* hi = lo + ((a.rows - 1) * a.lds + a.cols) * 2;
  const int64_t step = int64_t(gridDim.x) * (kThreads / 32);
  for (int64_t i = int64_t(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32; i < runs; i += step) {
    const int64_t row = divide(i, per_row), c0 = (i - row * per_row.d) * kRunCols + lane * 8, left = a.cols - c0;
    const char* q = lo + (row * a.lds + c0) * 2;
    const uint32_t off = uint32_t(reinterpret_cast<uintptr_t>(q)) & 15u;
    uint4 x[kVec], y[kVec];
    bool safe[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      const char* b = q + e * 512 - off;
      safe[e] = e * 256 < left && b >= lo && b + 32 <= hi;
      if (safe[e]) {
        x[e] = __ldg(reinterpret_cast<const uint4*>(b));
        y[e] = __ldg(reinterpret_cast<const uint4*>(b) + 1);
      }
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      const int n = int(min(left - e * 256, int64_t(8)));
      if (n <= 0) continue;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (safe[e]) v = shifted16(x[e], y[e], off);
      if (!safe[e] || n < 8) {
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t keep = k & 1 ? 0x0000FFFFu : 0xFFFF0000u;  // the other half of the word
          if (k >= n)
            w[k / 2] &= keep;
          else if (!safe[e])
            w[k / 2] |= uint32_t(__ldg(reinterpret_cast<const uint16_t*>(q + e * 512) + k)) << (k & 1 ? 16 : 0);
        }
        v = make_uint4(w[0], w[1], w[2], w[3]);
      }
      *reinterpret_cast<uint4*>(static_cast<char*>(a.dst) + (row * a.ldd + c0 + e * 256) * 2) = v;
    }
  }
}

}  // namespace

cudaError_t launch_align(const AlignArgs& a, cudaStream_t s) {
  static LayerGrid cache;
  const int64_t per = (a.cols + kRunCols - 1) / kRunCols, runs = a.rows * per, want = (runs + kThreads / 32 - 1) / (kThreads / 32);
  int cap = 0;
  const cudaError_t e = layer_grid(cache, reinterpret_cast<const void*>(k_align), kThreads, 0, 0, &cap);
  if (e != cudaSuccess) return e;
  k_align<<<unsigned(want < cap ? want : cap), kThreads, 0, s>>>(a, make_divisor(per, runs), runs);
  return cudaGetLastError();
}

}  // namespace loco
