// Device helpers of the layer kernels: element access, activations, and the
// arithmetic of 8-bit checkpoints.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "layers_internal.h"
#include "loco.h"

namespace loco {

// Division of indexes below 2^31 by one divisor: n / d = (n * m) >> (31 + l) with 2^(l-1) < d <= 2^l
// and m = ceil(2^(31+l) / d) < 2^32, exact because n * (m * d - 2^(31+l)) < 2^31 * 2^l.  Larger
// ranges divide in 64 bits.
struct Divisor {
  uint32_t m;
  int shift;
  bool wide;
  int64_t d;
};
inline Divisor make_divisor(int64_t d, int64_t range) {
  Divisor v{0, 0, range > 0x7FFFFFFF, d};
  if (!v.wide) {
    int l = 0;
    while ((int64_t(1) << l) < d) ++l;
    v.shift = 31 + l;
    v.m = uint32_t(((uint64_t(1) << v.shift) + uint64_t(d) - 1) / uint64_t(d));
  }
  return v;
}
__device__ __forceinline__ int64_t divide(int64_t n, const Divisor& v) {
  return v.wide ? n / v.d : int64_t((uint64_t(uint32_t(n)) * v.m) >> v.shift);
}

__device__ __forceinline__ float bf16_bits_to_f32(uint32_t b) { return __uint_as_float(b << 16); }
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Pairs of fp32 values in one register pair: one instruction for two sums, products or both.
struct Pair {
  unsigned long long u;
};
__device__ __forceinline__ Pair pair(float lo, float hi) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p.u) : "f"(lo), "f"(hi));
  return p;
}
__device__ __forceinline__ float2 halves(Pair p) {
  float2 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(p.u));
  return v;
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(a.u), "l"(b.u));
  return r;
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(a.u), "l"(b.u));
  return r;
}
__device__ __forceinline__ Pair fma(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.u) : "l"(a.u), "l"(b.u), "l"(c.u));
  return r;
}
__device__ __forceinline__ Pair widen(uint32_t bf16x2) {
  return pair(__uint_as_float(bf16x2 << 16), __uint_as_float(bf16x2 & 0xFFFF0000u));
}
// Eight values as four pairs.
__device__ __forceinline__ void widen8(uint4 w, Pair v[4]) {
  v[0] = widen(w.x), v[1] = widen(w.y), v[2] = widen(w.z), v[3] = widen(w.w);
}
__device__ __forceinline__ void pairs8(const float f[8], Pair v[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = pair(f[2 * k], f[2 * k + 1]);
}
__device__ __forceinline__ void floats8(const Pair v[4], float f[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 h = halves(v[k]);
    f[2 * k] = h.x, f[2 * k + 1] = h.y;
  }
}

// Shared memory by its 32-bit address: sixteen or eight bytes in, sixteen out.
__device__ __forceinline__ void copy_to_shared16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_to_shared8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 shared16(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(src) : "memory");
  return v;
}
__device__ __forceinline__ uint2 shared8(uint32_t src) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(src) : "memory");
  return v;
}
__device__ __forceinline__ void to_shared16(uint32_t dst, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// One element of an array of bf16 or fp32 (a uniform branch on the type).
__device__ __forceinline__ float load_elem(const void* p, int64_t i, int bf16) {
  return bf16 ? bf16_bits_to_f32(__ldg(static_cast<const uint16_t*>(p) + i)) : __ldg(static_cast<const float*>(p) + i);
}
__device__ __forceinline__ void store_elem(void* p, int64_t i, int bf16, float v) {
  if (bf16)
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(p)[i] = v;
}

// One element of an array that the same kernel may write (an output that is also the residual).
__device__ __forceinline__ float load_elem_rw(const void* p, int64_t i, int bf16) {
  return bf16 ? bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}

// Eight consecutive elements through 16-byte accesses (the address is 16-byte aligned).
template <bool RW = false>
__device__ __forceinline__ void load8(const void* p, int64_t i, int bf16, float v[8]) {
  if (bf16) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint4 w = RW ? *q : __ldg(q);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(u[k] << 16);
      v[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
    }
  } else {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = RW ? q[0] : __ldg(q), b = RW ? q[1] : __ldg(q + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}
__device__ __forceinline__ void store8(void* p, int64_t i, int bf16, const float v[8]) {
  if (bf16) {
    uint4 w;
    w.x = pack_bf16x2(v[0], v[1]), w.y = pack_bf16x2(v[2], v[3]);
    w.z = pack_bf16x2(v[4], v[5]), w.w = pack_bf16x2(v[6], v[7]);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = w;
  } else {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// Sixteen bytes that begin `off` bytes (a multiple of 2) into x and run on into y.
__device__ __forceinline__ uint4 shifted16(uint4 x, uint4 y, uint32_t off) {
  uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
  for (int i = 0; i < 6; ++i) w[i] = off & 8 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = off & 4 ? w[i + 1] : w[i];
  const uint32_t pick = off & 2 ? 0x5432u : 0x3210u;
  return make_uint4(__byte_perm(w[0], w[1], pick), __byte_perm(w[1], w[2], pick), __byte_perm(w[2], w[3], pick),
                    __byte_perm(w[3], w[4], pick));
}

// Eight elements from any place, where [lo, hi) is the matrix in memory: put together from the aligned
// sixteen bytes around them, or element by element where those would leave the matrix.
template <bool BF16>
__device__ __forceinline__ void load8_any(const char* q, const char* lo, const char* hi, float v[8]) {
  constexpr int kBytes = BF16 ? 16 : 32;
  const uint32_t off = uint32_t(reinterpret_cast<uintptr_t>(q)) & 15u;
  const char* b = q - off;
  if (b >= lo && b + kBytes + (off ? 16 : 0) <= hi) {
    const uint4* p = reinterpret_cast<const uint4*>(b);
    const uint4* last = p + (kBytes / 16 - (off ? 0 : 1));
    if (BF16) {
      const uint4 w = shifted16(__ldg(p), __ldg(last), off);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        v[2 * k] = __uint_as_float(u[k] << 16), v[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
    } else {
      const uint4 x = __ldg(p), y = __ldg(p + 1), z = __ldg(last);
      const uint4 a = shifted16(x, y, off), c = shifted16(y, z, off);
      v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y), v[2] = __uint_as_float(a.z), v[3] = __uint_as_float(a.w);
      v[4] = __uint_as_float(c.x), v[5] = __uint_as_float(c.y), v[6] = __uint_as_float(c.z), v[7] = __uint_as_float(c.w);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = load_elem(q, k, BF16);
  }
}

// ---------------------------------------------------------------------------
// 8-bit checkpoints: a block of 32 values shares the step 2^e, e = max(floor(log2 A) - 6, -126).
// The exponent field of A's bits is floor(log2 A) + 127 (0 for a subnormal A), so the scale byte
// e + 127 needs no logarithm, and 2^-e and 2^e are built from it: products with them are exact.
// ---------------------------------------------------------------------------
constexpr uint32_t kCkptBad = 255;  // a block with a NaN or an infinity

// Magnitude bits order like the magnitudes, with infinity and then NaN on top.
__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t ckpt_scale(uint32_t amax_bits) {
  const int f = int(amax_bits >> 23);
  return f == 255 ? kCkptBad : uint32_t(max(f - 6, 1));
}
// 2^-e, or 0 for a bad block (whose codes are then all 0).
__device__ __forceinline__ float ckpt_inv_step(uint32_t scale) {
  return scale == kCkptBad ? 0.0f : __uint_as_float((254u - scale) << 23);
}
// 2^e, or NaN for a bad block.
__device__ __forceinline__ float ckpt_step(uint32_t scale) {
  return __uint_as_float(scale == kCkptBad ? 0x7FC00000u : scale << 23);
}
// The code of v: rint_even(v * inv) clamped to [-127, 127]; 0 for a NaN product (a bad block's).
__device__ __forceinline__ int ckpt_code(float v, float inv) {
  return __float2int_rn(fminf(fmaxf(inv == 0.0f ? 0.0f : v * inv, -127.0f), 127.0f));
}
// Bits of the largest magnitude of a block of which four neighbouring lanes hold eight values each.
__device__ __forceinline__ uint32_t block_magnitude(const float v[8]) {
  uint32_t m = mag_bits(v[0]);
#pragma unroll
  for (int k = 1; k < 8; ++k) m = max(m, mag_bits(v[k]));
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  return max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
}
// Eight codes of a block whose largest magnitude has the bits `amax`.  v * 2^-e is exact, so adding
// 1.5 * 2^23 in one fused operation rounds it to an integer (halves to even) whose low byte is the
// code.  Only a block with A >= 127.5 * 2^e can round past +-127, and only a bad block holds NaN or
// infinity: those few take the clamped way.
__device__ __forceinline__ uint2 ckpt_pack8(const float v[8], uint32_t amax) {
  const float inv = ckpt_inv_step(ckpt_scale(amax));
  uint32_t b[8];
  if ((amax & 0x7FFFFFu) < 0x7F0000u && amax < 0x7F800000u) {
#pragma unroll
    for (int k = 0; k < 8; ++k) b[k] = __float_as_uint(fmaf(v[k], inv, 12582912.0f));
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) b[k] = uint32_t(ckpt_code(v[k], inv));
  }
  return make_uint2(__byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410));
}
// Four codes of a word as floats (exact): each byte, offset to unsigned, is placed in the low
// mantissa bits of 2^23 and the offset subtracted.
__device__ __forceinline__ void ckpt_unpack4(uint32_t w, float step, float v[4]) {
  const uint32_t u = w ^ 0x80808080u;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    v[k] = (__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 | k)) - 8388736.0f) * step;
}

// Four codes of a word under a scale byte as two pairs.
__device__ __forceinline__ void ckpt_pairs4(uint32_t w, uint32_t scale, Pair v[2]) {
  const float st = ckpt_step(scale);
  const Pair off = pair(-8388736.0f, -8388736.0f), st2 = pair(st, st);
  const uint32_t u = w ^ 0x80808080u;
#pragma unroll
  for (int k = 0; k < 2; ++k)
    v[k] = (pair(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 | 2 * k)),
                 __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7441 | 2 * k))) + off) * st2;
}

// Four codes as four bf16, with no detour over fp32.  Under the exponent of 2^7 a bf16's seven
// mantissa bits count whole units: 0x4300 | (c & 0x7F) is 128 + (c & 0x7F) and 0x4300 | (c & 0x80) is
// 128 or, for a negative code, 256, so their difference is the code, and its product with a power of
// two is exact.
__device__ __forceinline__ uint2 decode4_bf16(uint32_t w, uint32_t step_bf16x2) {
  uint32_t r[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t u = __byte_perm(w, 0x43u, i ? 0x4342 : 0x4140);
    asm("{\n\t.reg .b32 d;\n\tsub.rn.bf16x2 d, %1, %2;\n\tmul.rn.bf16x2 %0, d, %3;\n\t}"
        : "=r"(r[i])
        : "r"(u & 0xFF7FFF7Fu), "r"(u & 0xFF80FF80u), "r"(step_bf16x2));
  }
  return make_uint2(r[0], r[1]);
}
// 2^e twice in bf16 (NaN for a bad block).
__device__ __forceinline__ uint32_t ckpt_step_bf16x2(uint32_t scale) {
  return scale == kCkptBad ? 0x7FC07FC0u : scale * 0x00800080u;
}

// ---------------------------------------------------------------------------
// Activations and their slopes, in fp32.  2^x and 1/x are the hardware's approximations (2 and 1 units
// of the last place) on arguments and results that may be flushed to zero: a term below 2^-126 beside
// 1, or a sigmoid below it.  A NaN stays one through every activation and slope.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float exp2_f(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp_f(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
constexpr float kLog2E = 1.4426950408889634f;
__device__ __forceinline__ float sigmoid_f(float v) { return rcp_f(1.0f + exp2_f(v * -kLog2E)); }

constexpr float kGeluK2 = 1.5957691216057308f;  // 2 sqrt(2/pi)
constexpr float kGeluC = 0.044715f;

// The normal distribution function at v and, through `e`, exp(-v^2 / 2).  Its lower tail is t P(t) exp(-v^2 / 2)
// with t = 1 / (1 + 0.3 |v|), P of degree 7: the tail times exp(v^2 / 2) is smooth in t down to t = 0, and the
// coefficients make the largest relative error over |v| <= 13.3 (where the tail leaves the normal numbers)
// smallest, 1.2e-7 (Remez exchange in 64 bits).  So the error is relative in the tail too: (26 + 1.13 v^2) 2^-24
// at most, the second part from rounding the exponent.  (Five terms with an absolute bound of 1.5e-7 were off
// by 5e-5 at -3 and 4e-3 at -6.)
__device__ __forceinline__ float normal_cdf(float v, float* e) {
  const float t = rcp_f(fmaf(fabsf(v), 0.3f, 1.0f));
  *e = exp2_f(v * v * (-0.5f * kLog2E));
  float q = fmaf(t, 0.0360362083f, -0.158713222f);
  q = fmaf(t, q, 0.208963946f);
  q = fmaf(t, q, -0.0560953282f);
  q = fmaf(t, q, 0.129843146f);
  q = fmaf(t, q, 0.099523142f);
  q = fmaf(t, q, 0.120816886f);
  q = fmaf(t, q, 0.119625174f);
  q *= t * *e;  // the tail
  return v > 0.0f ? 1.0f - q : q;
}

__device__ __forceinline__ float act_value(float v, int act) {
  switch (act) {
    case LOCO_ACT_RELU: return v <= 0.0f ? 0.0f : v;
    case LOCO_ACT_GELU: {
      float e;
      return v * normal_cdf(v, &e);
    }
    case LOCO_ACT_GELU_TANH: {
      // (1 + tanh u) / 2 = sigmoid(2u); beyond |v| = 20 it is 0 or 1 in fp32
      const float c = fminf(fmaxf(v, -20.0f), 20.0f);
      return v * sigmoid_f(c * fmaf(c * c, kGeluK2 * kGeluC, kGeluK2));
    }
    case LOCO_ACT_SILU: return v * sigmoid_f(v);
    default: return v;
  }
}

__device__ __forceinline__ float act_slope(float v, int act) {
  switch (act) {
    case LOCO_ACT_RELU: return v > 0.0f ? 1.0f : (v == v ? 0.0f : v);
    case LOCO_ACT_GELU: {
      float e;
      const float p = normal_cdf(v, &e);
      return fmaf(v * 0.3989422804014327f, e, p);
    }
    case LOCO_ACT_GELU_TANH: {
      const float c = fminf(fmaxf(v, -20.0f), 20.0f), q = c * c;
      const float s = sigmoid_f(c * fmaf(q, kGeluK2 * kGeluC, kGeluK2));
      const float d = fmaf(c * s * (1.0f - s), fmaf(q, 3.0f * kGeluK2 * kGeluC, kGeluK2), s);
      return v == v ? d : v;
    }
    case LOCO_ACT_SILU: {
      const float s = sigmoid_f(v);
      return s * fmaf(v, 1.0f - s, 1.0f);
    }
    default: return 1.0f;
  }
}

// v = act(v) and v *= act'(z) for N values, with the choice made once.
template <int N>
__device__ __forceinline__ void apply_act(float (&v)[N], int act) {
#define LOCO_EACH(A)               \
  case A:                          \
    _Pragma("unroll") for (int k = 0; k < N; ++k) v[k] = act_value(v[k], A); \
    break
  switch (act) {
    LOCO_EACH(LOCO_ACT_RELU);
    LOCO_EACH(LOCO_ACT_GELU);
    LOCO_EACH(LOCO_ACT_GELU_TANH);
    LOCO_EACH(LOCO_ACT_SILU);
    default: break;
  }
#undef LOCO_EACH
}
template <int N>
__device__ __forceinline__ void mul_slope(float (&v)[N], const float (&z)[N], int act) {
#define LOCO_EACH(A)               \
  case A:                          \
    _Pragma("unroll") for (int k = 0; k < N; ++k) v[k] *= act_slope(z[k], A); \
    break
  switch (act) {
    LOCO_EACH(LOCO_ACT_RELU);
    LOCO_EACH(LOCO_ACT_GELU);
    LOCO_EACH(LOCO_ACT_GELU_TANH);
    LOCO_EACH(LOCO_ACT_SILU);
    default: break;
  }
#undef LOCO_EACH
}

}  // namespace loco
