// Internal interface between the entry points of joins, log probabilities and many-tensor
// optimizer steps (steps_abi.cu) and the launchers of their kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "layers_internal.h"

namespace loco {

// Types of elements: 1 bf16, 0 fp32 (the values of loco_dtype).
struct JoinFwdArgs {
  const void* x;
  const void* y;
  const void* post_gamma;
  const void* post_beta;
  const void* gate;
  const float* row_gate;
  const void* gamma;
  const void* beta;
  void* h;
  void* u;
  float* stats;  // [4][rows]
  int64_t ldx, ldy, ldh, ldu, rows, cols;
  float eps, a, s;
  int rms, post, x_bf16, y_bf16, param_bf16;
};

// Most partial sums of the parameters' gradients that the backward pass writes (one per CTA), and the
// sums of each: of c yh, of c (without the gate), of du hh and of du.
constexpr int kJoinPartials = 608;
constexpr int kJoinSums = 4;

struct JoinBwdArgs {
  const void* dh;
  const void* du;
  const void* h;
  const void* y;
  const float* stats;
  const void* post_gamma;
  const void* post_beta;
  const void* gate;
  const float* row_gate;
  const void* gamma;
  void* dx;
  void* dy;
  void* dpost_gamma;
  void* dpost_beta;
  void* dgate;
  float* drow_gate;
  void* dgamma;
  void* dbeta;
  float* partials;  // [CTAs][kJoinSums][cols]; null: no gradient of a parameter
  int64_t lddh, lddu, ldh, ldy, lddx, lddy, rows, cols;
  float a, s;
  int rms, post, x_bf16, y_bf16, param_bf16, grad_bf16;
};

struct LogprobFwdArgs {
  const void* logits;
  int64_t ld, rows, vocab;
  float scale;
  const int64_t* targets;
  float* logp;
  float* lse;
  float* entropy;
  int64_t* top_ids;
  float* top_logp;
  int top, bf16;
};

struct LogprobBwdArgs {
  const void* logits;
  int64_t ld, rows, vocab;
  float scale;
  const int64_t* targets;
  const float* lse;
  const float* entropy;
  const float* dlogp;
  const float* dentropy;
  void* dlogits;
  int64_t ldd;
  int bf16;
};

// One tensor of an optimizer step as its kernel reads it.
struct AdamTensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* m_steps;
  float* v_steps;
  uint16_t* copy;
  int64_t n;
  float c1, lr_wd;
  uint32_t key;  // of its dither: mix(mix(mix(dither) ^ lo32(t)) ^ index)
  uint32_t wide; // every buffer takes vectors of four elements
};

// Tensors of one launch: they travel in the kernel's parameters (32764 bytes at most).
constexpr int kAdamFew = 24, kAdamMany = 384;

struct AdamTensorsArgs {
  float beta1, beta2, one_minus_beta1, one_minus_beta2, c2, eps;
  float neg_zero;  // -0.0f, unknown when the kernel is compiled
  int eps_inside_sqrt;
  const float* grad_scale;
};

// Kernel parameters: tensors and the first unit (256 elements) of each; first[count] is the total.
template <int MAX>
struct AdamTensorList {
  AdamTensorsArgs a;
  int count;
  uint32_t first[MAX + 1];
  AdamTensor t[MAX];
};
static_assert(sizeof(AdamTensorList<kAdamMany>) <= 32764, "a kernel's parameters");

struct AdamTensorsKind {
  int bits, p_bf16, g_bf16, dither;
};

// The hash behind the dither, on 32 bits: multiplications by the fractions of the roots of 2 and 3.
__host__ __device__ inline uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}

// Waits of a cluster's CTAs for one another that ran out, on the current device.
cudaError_t read_join_forward_timeouts(int64_t* count);
cudaError_t read_join_backward_timeouts(int64_t* count);

cudaError_t launch_join_forward(const JoinFwdArgs& a, cudaStream_t s);
cudaError_t launch_join_backward(const JoinBwdArgs& a, cudaStream_t s);
cudaError_t launch_logprob_forward(const LogprobFwdArgs& a, cudaStream_t s);
cudaError_t launch_logprob_backward(const LogprobBwdArgs& a, cudaStream_t s);
template <int MAX>
cudaError_t launch_adam_tensors(const AdamTensorList<MAX>& list, const AdamTensorsKind& kind, cudaStream_t s);
cudaError_t launch_state_decode(int second, const void* codes, const float* steps, int64_t n, void* out, int out_bf16,
                                cudaStream_t s);

}  // namespace loco
