// Internal interface between the layers' entry points (layers_abi.cu) and the
// launchers of their kernels.  Not installed; the public interface is include/loco.h.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace loco {

constexpr int kCkptBlock = 32;

// Types of elements and parameters: 1 bf16, 0 fp32 (the values of loco_dtype).
struct EncodeArgs {
  const void* x;
  int64_t ldx, rows, cols;
  int x_bf16;
  int8_t* codes;
  uint8_t* scales;
};

struct DecodeArgs {
  const int8_t* codes;
  const uint8_t* scales;
  int64_t rows, cols, ldo;
  int act;
  const void* gamma;
  const void* beta;
  int param_bf16;
  void* out;
  int out_bf16;
};

struct NormFwdArgs {
  const void* x;
  const void* gamma;
  const void* beta;
  void* y;
  float* mean;
  float* rstd;
  int8_t* codes;
  uint8_t* scales;
  int64_t ldx, ldy, rows, cols;
  float eps;
  int rms, x_bf16, y_bf16, param_bf16;
};

// Most partial sums of dgamma/dbeta that the backward pass writes (one per CTA).
constexpr int kNormPartials = 608;

struct NormBwdArgs {
  const void* dy;
  const void* x;
  const int8_t* codes;
  const uint8_t* scales;
  const float* mean;
  const float* rstd;
  const void* gamma;
  const void* residual;
  void* dx;
  void* dgamma;
  void* dbeta;
  float* partials;  // [CTAs][2][cols]
  int64_t lddy, ldx, ldr, lddx, rows, cols;
  int rms, x_bf16, y_bf16, param_bf16, grad_bf16;
};

// One product D[n][m] = sum_k A[m][k] * B[n][k] with its epilogue.  m runs along
// the output's contiguous columns, n along its rows.
struct LinearArgs {
  // operands: memory [m][k] with k contiguous, or ("mn") [k][m] with m contiguous
  const void* a;
  const void* b;
  int64_t lda, ldb;
  int a_mn, b_mn;
  const int8_t* a_codes;    // A from a checkpoint [k][m] (then a is null, a_mn = 1)
  const uint8_t* a_scales;
  int64_t M, N, K;
  // epilogue, in this order
  const void* col_scale;    // v *= col_scale[m]
  const void* col_shift;    // v += col_shift[m] * row_sum[n]
  const float* row_sum;
  const void* bias;         // v += bias[m]
  int param_bf16;
  int8_t* save_codes;       // checkpoint of v, [n][m]
  uint8_t* save_scales;
  int act;                  // v = act(v)
  const int8_t* z_codes;    // v *= act'(z), z [n][m] from its checkpoint (then act is not applied)
  const uint8_t* z_scales;
  const void* residual;     // v += residual[n][m]
  void* out;
  int64_t ldr, ldo;
  int out_bf16;
};

struct AlignArgs {
  const void* src;          // [rows, cols] bf16
  int64_t lds, rows, cols;
  void* dst;                // on a 16-byte boundary, ldd a multiple of 8
  int64_t ldd;
};

struct ColSumArgs {
  const void* x;            // [rows, cols] bf16
  int64_t ldx, rows, cols;
  float* sum_f32;           // [cols] fp32 or null
  void* out;                // [cols] of out_bf16 or null
  int out_bf16;
};

cudaError_t launch_ckpt_encode(const EncodeArgs& a, cudaStream_t s);
cudaError_t launch_ckpt_decode(const DecodeArgs& a, cudaStream_t s);
cudaError_t launch_norm_forward(const NormFwdArgs& a, cudaStream_t s);
cudaError_t launch_norm_backward(const NormBwdArgs& a, cudaStream_t s);
cudaError_t launch_align(const AlignArgs& a, cudaStream_t s);
cudaError_t launch_linear(const LinearArgs& a, cudaStream_t s);
cudaError_t launch_col_sum(const ColSumArgs& a, cudaStream_t s);
cudaError_t read_linear_timeouts(int64_t* count);

// Resident CTAs of one kernel on each device (0: not asked yet there).
struct LayerGrid {
  static constexpr int kDevices = 64;
  std::atomic<int> cap[kDevices];
};

// CTAs of the kernel that the current device holds at once, launched with smem_bytes of dynamic
// shared memory; smem_most is the most that any launch of this kernel asks for.
cudaError_t layer_grid(LayerGrid& cache, const void* kernel, int threads, size_t smem_bytes, size_t smem_most, int* cap);

// SMs of the current device (asked once per device).
cudaError_t sm_count(int* sms);

}  // namespace loco
