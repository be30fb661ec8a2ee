// 8-bit activation checkpoints: a matrix to codes and scales, and back through
// an activation or a norm's scale and shift.
//
// Both are single passes bound by memory: bf16 values cost 2 + 1 + 1/32 bytes
// each way.  A block of 32 values spans 4 threads of 8 values (one or two
// 16-byte loads each), whose largest magnitude is two shuffles away.  Rows that
// start on no 16-byte boundary are read and written in aligned pieces all the
// same, shifted together from two of them.
// 16384 x 11008 bf16: encode 89 us (6.1 TB/s, 90 % of a copy's rate), decode 96 us
// (5.7), through SiLU 97 us, through GELU 150 us (bound by the distribution function's arithmetic);
// fp32 encode 135 us (6.7).  16384 x 4095 bf16: encode 85 us, decode 58 us.
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

template <bool BF16, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) k_encode(EncodeArgs a, Divisor per_row, int64_t nb, int64_t runs) {
  const int lane = threadIdx.x & 31;
  const int64_t step = int64_t(gridDim.x) * (kThreads / 32);
  const char* lo = static_cast<const char*>(a.x);  // the matrix in memory
  const char* hi = lo + ((a.rows - 1) * a.ldx + a.cols) * (BF16 ? 2 : 4);
  for (int64_t i = int64_t(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32; i < runs; i += step) {
    const int64_t row = divide(i, per_row), c0 = (i - row * per_row.d) * kRunCols + lane * 8;
    const char* x = static_cast<const char*>(a.x) + (row * a.ldx + c0) * (BF16 ? 2 : 4);
    int8_t* codes = a.codes + row * nb * kCkptBlock + c0;
    uint8_t* scales = a.scales + row * nb + c0 / kCkptBlock;
    const int64_t left = a.cols - c0, pad = nb * kCkptBlock - c0;  // columns from the lane's first on
    float v[kVec][8];
    const auto load = [&](int e) {
      if (ALIGNED)
        load8(x, e * 256, BF16, v[e]);
      else
        load8_any<BF16>(x + e * 256 * (BF16 ? 2 : 4), lo, hi, v[e]);
    };
    if (left >= kRunCols - 256 + 8) {
#pragma unroll
      for (int e = 0; e < kVec; ++e) load(e);
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        if (left >= e * 256 + 8) {
          load(e);
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

// The sixteen bytes (of bf16; thirty-two of fp32) that end `off` bytes into a lane's eight values: the
// previous lane's last ones before its own.  w: the lane's words, p: the previous lane's.
template <int N>
__device__ __forceinline__ void joined(const uint32_t (&w)[N], const uint32_t (&p)[N], uint32_t off, uint32_t (&r)[N]) {
  // words 4 - off/4 of the previous lane and on, the shift of a half word last
  uint32_t t[N + 5];
#pragma unroll
  for (int i = 0; i < 4; ++i) t[i] = p[N - 4 + i];
#pragma unroll
  for (int i = 0; i < N; ++i) t[4 + i] = w[i];
  // the window starts (16 - off) bytes into t
  const uint32_t s = 16 - off;
#pragma unroll
  for (int i = 0; i < N + 2; ++i) t[i] = s & 8 ? t[i + 2] : t[i];
#pragma unroll
  for (int i = 0; i < N + 1; ++i) t[i] = s & 4 ? t[i + 1] : t[i];
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = __byte_perm(t[i], t[i + 1], s & 2 ? 0x5432 : 0x3210);
}

// Runs as in k_encode.  PLAIN: the values as they are.  Where the rows of out start on no 16-byte
// boundary, a lane writes the aligned bytes that end inside its values, the first of them the previous
// lane's; what has no neighbour to write it goes element by element.
template <bool BF16, bool PLAIN, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, ALIGNED ? 4 : 3) k_decode(DecodeArgs a, Divisor per_row, int64_t nb, int64_t runs) {
  constexpr int kWords = BF16 ? 4 : 8, kSize = BF16 ? 2 : 4;
  const int lane = threadIdx.x & 31;
  const int64_t step = int64_t(gridDim.x) * (kThreads / 32);
  for (int64_t i = int64_t(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32; i < runs; i += step) {
    const int64_t row = divide(i, per_row), c0 = (i - row * per_row.d) * kRunCols + lane * 8;
    const int8_t* codes = a.codes + row * nb * kCkptBlock + c0;
    const uint8_t* scales = a.scales + row * nb + c0 / kCkptBlock;
    char* out = static_cast<char*>(a.out) + (row * a.ldo + c0) * kSize;
    const int64_t left = a.cols - c0;
    const uint32_t off = ALIGNED ? 0 : uint32_t(reinterpret_cast<uintptr_t>(out)) & 15u;  // the same in all lanes
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
    uint32_t before[kWords];  // the previous vector's words
#pragma unroll
    for (int k = 0; k < kWords; ++k) before[k] = 0;
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      if (ALIGNED && e * 256 >= left) continue;
      uint32_t u[kWords];
      if (PLAIN && BF16) {
        const uint32_t st = ckpt_step_bf16x2(sc[e]);
        const uint2 lo = decode4_bf16(w[e].x, st), hi = decode4_bf16(w[e].y, st);
        u[0] = lo.x, u[1] = lo.y, u[2] = hi.x, u[3] = hi.y;
      } else {
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
#pragma unroll
        for (int k = 0; k < kWords; ++k) u[k] = BF16 ? pack_bf16x2(v[2 * k % 8], v[(2 * k + 1) % 8]) : __float_as_uint(v[k]);
      }
      const auto element = [&](int k) {
        if (BF16)
          reinterpret_cast<uint16_t*>(out + e * 512)[k] = uint16_t(u[k / 2 % kWords] >> (k & 1 ? 16 : 0));
        else
          reinterpret_cast<uint32_t*>(out + e * 1024)[k] = u[k % kWords];
      };
      const bool full = e * 256 + 8 <= left;
      if (ALIGNED || off == 0) {
        if (full) {
          uint4* o = reinterpret_cast<uint4*>(out + e * 256 * kSize);
          o[0] = make_uint4(u[0], u[1], u[2], u[3]);
          if (!BF16) o[1] = make_uint4(u[kWords - 4], u[kWords - 3], u[kWords - 2], u[kWords - 1]);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (e * 256 + k < left) element(k);
        }
      } else if constexpr (!ALIGNED) {
        uint32_t prev[kWords], r[kWords];
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
          prev[k] = 0;
          if (k >= kWords - 4) prev[k] = __shfl_sync(0xFFFFFFFFu, lane == 31 ? before[k] : u[k], (lane + 31) & 31);
          before[k] = u[k];
        }
        joined(u, prev, off, r);
        const bool has_prev = e > 0 || lane > 0, has_next = (e + 1 < kVec || lane < 31) && e * 256 + 16 <= left;
        const int tail = int(off) / kSize;  // elements after the lane's last boundary
        if (full && has_prev) {
          uint4* o = reinterpret_cast<uint4*>(out + e * 256 * kSize - off);
          o[0] = make_uint4(r[0], r[1], r[2], r[3]);
          if (!BF16) o[1] = make_uint4(r[kWords - 4], r[kWords - 3], r[kWords - 2], r[kWords - 1]);
        }
        // not written by this lane's pieces or the next one's: all of a lane that is not full, the head of a
        // run's first lane, the tail of a lane whose next is not full
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const bool mine = !full ? e * 256 + k < left : (!has_prev && k < 8 - tail) || (!has_next && k >= 8 - tail);
          if (mine) element(k);
        }
      }
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
  const bool aligned = wide_rows(a.x, a.ldx, a.rows, a.x_bf16);
  const int64_t per = (nb * kCkptBlock + kRunCols - 1) / kRunCols, runs = a.rows * per;
  const auto kernel = a.x_bf16 ? (aligned ? k_encode<true, true> : k_encode<true, false>)
                               : (aligned ? k_encode<false, true> : k_encode<false, false>);
  unsigned grid;
  const cudaError_t e = grid_for(kernel, cache[a.x_bf16 * 2 + aligned], runs, kThreads / 32, &grid);
  if (e != cudaSuccess) return e;
  kernel<<<grid, kThreads, 0, s>>>(a, make_divisor(per, runs), nb, runs);
  return cudaGetLastError();
}

cudaError_t launch_ckpt_decode(const DecodeArgs& in, cudaStream_t s) {
  static LayerGrid cache[8];
  DecodeArgs a = in;
  const bool plain = a.act == LOCO_ACT_NONE && a.gamma == nullptr && a.beta == nullptr;
  if (a.rows > 1 && a.ldo == a.cols && a.cols % kCkptBlock == 0 && a.gamma == nullptr && a.beta == nullptr)
    a.ldo = a.cols *= a.rows, a.rows = 1;  // one long row
  const int64_t nb = (a.cols + kCkptBlock - 1) / kCkptBlock;
  const bool aligned = wide_rows(a.out, a.ldo, a.rows, a.out_bf16);
  const int64_t per = (a.cols + kRunCols - 1) / kRunCols, runs = a.rows * per;
  const auto kernel = a.out_bf16 ? (plain ? (aligned ? k_decode<true, true, true> : k_decode<true, true, false>)
                                          : (aligned ? k_decode<true, false, true> : k_decode<true, false, false>))
                                 : (plain ? (aligned ? k_decode<false, true, true> : k_decode<false, true, false>)
                                          : (aligned ? k_decode<false, false, true> : k_decode<false, false, false>));
  unsigned grid;
  const cudaError_t e = grid_for(kernel, cache[a.out_bf16 * 4 + plain * 2 + aligned], runs, kThreads / 32, &grid);
  if (e != cudaSuccess) return e;
  kernel<<<grid, kThreads, 0, s>>>(a, make_divisor(per, runs), nb, runs);
  return cudaGetLastError();
}

}  // namespace loco
