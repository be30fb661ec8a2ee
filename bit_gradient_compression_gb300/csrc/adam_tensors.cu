// One Adam(W) step over many tensors, with states in 32 bits or in 8.
//
// A unit is 256 elements of one tensor: the elements that share an 8-bit state's step, and the work
// of one warp at a time.  The tensors' addresses and the first unit of each come in the kernel's
// parameters, so a step needs no table in device memory and no launch per tensor; a warp finds the
// tensor of its units by bisection.
//
// 8-bit states (the layout and the rounding are stated at loco_adam_tensors): codes become values by
// one product, the new values' largest magnitude is one warp reduction, and the new codes are the low
// bytes of x + d + 1.5 * 2^23.
//
// Every product and sum is rounded on its own, as in loco_adam_step.
//
// With 32-bit states HBM is the bound: 1.1e9 elements with bf16 gradients 4.60 ms, 6.7 TB/s, a copy's rate.  With 8-bit
// states the arithmetic is, 16 bytes and about 100 instructions an element: 1.41e9 elements, dithered, with bf16 copies 4.7
// ms, 4.8 TB/s (71 % of a copy's rate, issuing in 74 % of the cycles), and 1.3 ms for decoding both states to bf16, 6.4
// TB/s.  A block's 353712 elements take 7 us with their decodes on the device, less than the host's part of the calls.
#include "device_common.cuh"
#include "layers_common.cuh"
#include "steps_internal.h"

namespace loco {

namespace {

constexpr int kUnit = LOCO_STATE_BLOCK;
constexpr int kThreadsAdam = 256;
constexpr int kGroup = 8;  // most consecutive units of a warp

struct Elem4 {
  float f[4];
};

// Four consecutive elements (the address takes one access).
template <bool BF16>
__device__ __forceinline__ Elem4 load4(const void* p, int64_t i) {
  Elem4 r;
  if (BF16) {
    const uint2 w = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i));
    r.f[0] = bf16lo_to_f32(w.x), r.f[1] = bf16hi_to_f32(w.x), r.f[2] = bf16lo_to_f32(w.y), r.f[3] = bf16hi_to_f32(w.y);
  } else {
    const float4 w = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i));
    r.f[0] = w.x, r.f[1] = w.y, r.f[2] = w.z, r.f[3] = w.w;
  }
  return r;
}
__device__ __forceinline__ void store4(float* p, int64_t i, const Elem4& v) {
  __stcs(reinterpret_cast<float4*>(p + i), make_float4(v.f[0], v.f[1], v.f[2], v.f[3]));
}
__device__ __forceinline__ void store4_bf16(uint16_t* p, int64_t i, uint32_t lo, uint32_t hi) {
  __stcs(reinterpret_cast<uint2*>(p + i), make_uint2(lo, hi));
}

// Upper half of p's bits after the dither (a NaN stays one).
__device__ __forceinline__ uint32_t bf16_dithered(float p, uint32_t r) {
  const uint32_t b = __float_as_uint(p);
  return p == p ? (b + (r >> 16)) >> 16 : (b >> 16) | 0x40u;
}

// Products of pairs that feed sums: a packed product alone would be joined with the sum into one rounding, a fused
// one with -0 (which the compiler does not know) is rounded like a product and stays.
struct Rounded {
  Pair none;
  __device__ __forceinline__ Pair mul(Pair a, Pair b) const { return fma(a, b, none); }
};
__device__ __forceinline__ Pair both(float v) { return pair(v, v); }

// Correctly rounded square roots and quotients of pairs by Newton's iteration on fused multiply-adds, after P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor" (1990), and M. Cornea, R. Golliver and
// P. Markstein, "Correctness proofs outline for Newton-Raphson based floating-point divide and square root algorithms"
// (1999): from an approximation y of 1/b, one step makes it the rounded reciprocal, and q + (a - b q) y, whose remainder
// a - b q is exact, the rounded quotient; likewise g + (v - g^2) h for the root, h of 1 / (2 sqrt(v)).  They hold where
// nothing is lost to the ends of the exponent's range: see `extreme`.  The tests compare steps over every root of [1, 4),
// each the denominator of several quotients, with the IEEE operations.
// With them a step with 8-bit states takes about 100 instructions an element instead of 111.
__device__ __forceinline__ float rsqrt_approx(float v) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ Pair sqrt_pair(Pair v) {
  const float2 f = halves(v);
  const Pair y = pair(rsqrt_approx(f.x), rsqrt_approx(f.y));
  Pair g = v * y, h = y * both(-0.5f);
  const Pair r = fma(g, h, both(0.5f));
  g = fma(g, r, g), h = fma(h, r, h);
  return fma(fma(g, g, v * both(-1.0f)), h, g);
}
__device__ __forceinline__ Pair div_pair(Pair a, Pair b) {
  const float2 f = halves(b);
  const Pair less = b * both(-1.0f), y0 = pair(rcp_f(f.x), rcp_f(f.y));
  const Pair y = fma(y0, fma(less, y0, both(1.0f)), y0);
  const Pair q = a * y;
  return fma(fma(less, q, a), y, q);
}
// Whether one of m, v and the denominator is neither zero nor far enough from the ends of the exponent's range for
// sqrt_pair (of v > 0) and div_pair: the last place of a remainder, 2^-47 of v or of m, must not be below 2^-149, nor
// a quotient's exponent out of range.  sqrt_pair of an infinite v is NaN, and so is its denominator: what is not a number
// within the range counts as extreme.
constexpr float kSmall = 8.67361738e-19f, kLarge = 1.15292150e18f;  // 2^-60, 2^60
constexpr float kSmallSquare = 7.88860905e-31f;                     // 2^-100
__device__ __forceinline__ bool extreme(float m, float v, float den) {
  return (fabsf(m) < kSmall && m != 0.0f) || fabsf(m) > kLarge || (v < kSmallSquare && v != 0.0f) ||
         !(den >= kSmall && den <= kLarge);
}

// d = (b - 127.5) / 256 of byte 0 or 1 of the random bits, exact: the byte under the exponent of 2^7, where it counts
// 256ths, less 2^7 + 127.5 / 256.
__device__ __forceinline__ Pair dither_of(uint32_t r0, uint32_t r1, int byte) {
  const uint32_t pick = byte ? 0x7414u : 0x7404u;
  return pair(__uint_as_float(__byte_perm(r0, 0x43000000u, pick)), __uint_as_float(__byte_perm(r1, 0x43000000u, pick))) +
         both(-128.498046875f);
}

__device__ __forceinline__ void store_pairs(float* p, int64_t i, Pair a, Pair b) {
  const float2 x = halves(a), y = halves(b);
  __stcs(reinterpret_cast<float4*>(p + i), make_float4(x.x, x.y, y.x, y.y));
}
__device__ __forceinline__ float of(const Pair* v, int j) { return j % 2 ? halves(v[j / 2]).y : halves(v[j / 2]).x; }
__device__ __forceinline__ uint32_t low_bytes(const uint32_t* c) {
  return __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
}
template <bool B>
struct Flag {
  static constexpr bool value = B;
};

__device__ __forceinline__ float largest(float a, float b) {  // of two magnitudes; NaN where one is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 1/step and the step of a block whose largest magnitude has the bits `top`, for `most` codes: 1/step is 0 for a block
// that is held as zeros, or as NaN.
__device__ __forceinline__ void state_step(uint32_t top, float most, float* inv, float* step) {
  const float a = __uint_as_float(top);
  const bool bad = top >= 0x7F800000u;
  const float i = __fdiv_rn(most, a);
  const bool some = !bad && i <= 3.402823466e38f;  // (0 and what is too small for 1/step: zeros)
  *inv = some ? i : 0.0f;
  *step = bad ? __uint_as_float(0x7FC00000u) : some ? __fdiv_rn(a, most) : 0.0f;
}

// A whole unit of a tensor whose buffers take vectors: elements lane * 4 + k + 128 * q.  32-bit states are loaded where
// they are needed.  8-bit ones take so much arithmetic that the next unit has to be on its way meanwhile: a thread copies
// its own pieces to shared memory (cp.async; nobody else reads them, so no barrier is needed).
template <bool PBF16, bool GBF16>
struct Staged {
  static constexpr int kP = PBF16 ? 1 : 2, kG = GBF16 ? 1 : 2, kPieces = kP + kG + 1;  // of sixteen bytes; the last are codes
  static constexpr uint32_t kPiece = kThreadsAdam * 16, kStage = kPieces * kPiece;

  __device__ static __forceinline__ void copy(uint32_t to, const AdamTensor& t, uint32_t unit, int lane) {
    const int64_t i = int64_t(unit) * kUnit + lane * 4;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (PBF16)
        copy_to_shared8(to + q * 8, static_cast<const uint16_t*>(t.p) + i + q * 128);
      else
        copy_to_shared16(to + q * kPiece, static_cast<const float*>(t.p) + i + q * 128);
      if (GBF16)
        copy_to_shared8(to + kP * kPiece + q * 8, static_cast<const uint16_t*>(t.g) + i + q * 128);
      else
        copy_to_shared16(to + (kP + q) * kPiece, static_cast<const float*>(t.g) + i + q * 128);
      copy4(to + (kP + kG) * kPiece + q * 4, static_cast<const int8_t*>(t.m) + i + q * 128);
      copy4(to + (kP + kG) * kPiece + 8 + q * 4, static_cast<const uint8_t*>(t.v) + i + q * 128);
    }
  }
  __device__ static __forceinline__ void copy4(uint32_t to, const void* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
  }
  // A unit whose buffers take no vectors, or a tensor's last: elements lane + 32 * j in the places of a thread's eight, 0
  // past the end.
  __device__ static __forceinline__ void put(uint32_t to, const AdamTensor& t, int64_t e0, int left, int lane) {
    put_eight<PBF16>(to, t.p, e0, left, lane);
    put_eight<GBF16>(to + kP * kPiece, t.g, e0, left, lane);
    uint32_t c[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c[j / 4] |= uint32_t(static_cast<const uint8_t*>(t.m)[e0 + lane + 32 * j]) << (j % 4 * 8);
      c[2 + j / 4] |= uint32_t(static_cast<const uint8_t*>(t.v)[e0 + lane + 32 * j]) << (j % 4 * 8);
    }
    to_shared16(to + (kP + kG) * kPiece, make_uint4(c[0], c[1], c[2], c[3]));
  }
  template <bool BF16>
  __device__ static __forceinline__ void put_eight(uint32_t to, const void* p, int64_t e0, int left, int lane) {
    uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int o = lane + 32 * j;
      if (o >= left) continue;
      if (BF16)
        w[j / 2] |= uint32_t(static_cast<const uint16_t*>(p)[e0 + o]) << (j % 2 * 16);
      else
        w[j] = static_cast<const uint32_t*>(p)[e0 + o];
    }
    to_shared16(to, make_uint4(w[0], w[1], w[2], w[3]));
    if (!BF16) to_shared16(to + kPiece, make_uint4(w[4], w[5], w[6], w[7]));
  }
  // Half q of the unit, elements lane * 4 + 128 * q: few registers at a time.  Codes become the floats 2^23 + code (and
  // 128 for a signed one).
  __device__ static __forceinline__ void half(uint32_t at, int q, float* p, float* g, float* m, float* v) {
    four<PBF16>(at, q, p);
    four<GBF16>(at + kP * kPiece, q, g);
    const uint32_t c = at + (kP + kG) * kPiece + q * 4;
    const uint32_t mw = word(c) ^ 0x80808080u, vw = word(c + 8);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      m[k] = __uint_as_float(__byte_perm(mw, kTwo23Bits, 0x7440 | k));
      v[k] = __uint_as_float(__byte_perm(vw, kTwo23Bits, 0x7440 | k));
    }
  }
  __device__ static __forceinline__ uint32_t word(uint32_t at) {
    uint32_t w;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(at) : "memory");
    return w;
  }
  template <bool BF16>
  __device__ static __forceinline__ void four(uint32_t at, int q, float* f) {
    if (BF16) {
      const uint2 w = shared8(at + q * 8);
      f[0] = bf16lo_to_f32(w.x), f[1] = bf16hi_to_f32(w.x), f[2] = bf16lo_to_f32(w.y), f[3] = bf16hi_to_f32(w.y);
    } else {
      const uint4 w = shared16(at + q * kPiece);
      f[0] = __uint_as_float(w.x), f[1] = __uint_as_float(w.y), f[2] = __uint_as_float(w.z), f[3] = __uint_as_float(w.w);
    }
  }
};

template <int BITS, bool PBF16, bool GBF16, bool DITHER, int MAX>
__global__ void __launch_bounds__(kThreadsAdam, BITS == 32 ? 2 : 3) k_step_tensors(const __grid_constant__ AdamTensorList<MAX> l, uint32_t group) {
  extern __shared__ __align__(128) uint8_t ring[];  // two stages
  using Stage = Staged<PBF16, GBF16>;
  const uint32_t base = smem_addr(ring) + threadIdx.x * 16;
  const int lane = threadIdx.x & 31;
  const uint32_t units = l.first[l.count];
  const uint32_t warps = gridDim.x * (kThreadsAdam / 32);
  const float scale = l.a.grad_scale != nullptr ? __ldg(l.a.grad_scale) : 1.0f;
  const Rounded rn{both(l.a.neg_zero)};
  // (units are below 2^31)
  for (uint32_t u0 = (blockIdx.x * (kThreadsAdam / 32) + threadIdx.x / 32) * group; u0 < units; u0 += warps * group) {
    int lo = 0, hi = l.count;  // first[lo] <= u0 < first[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (l.first[mid] <= u0)
        lo = mid;
      else
        hi = mid;
    }
    const uint32_t end = min(u0 + group, units);
    uint32_t slot = 0;                // of the unit at work
    bool here = false;                // it has been asked for
    float m_next = 0.0f, v_next = 0.0f;
    for (uint32_t u = u0; u < end; ++u) {
      while (u >= l.first[lo + 1]) ++lo;
      const AdamTensor& t = l.t[lo];
      const uint32_t b = u - l.first[lo];       // the unit within its tensor
      const int64_t e0 = int64_t(b) * kUnit;
      const int left = t.n - e0 < kUnit ? int(t.n - e0) : kUnit;
      const bool wide = t.wide && left == kUnit;
      // element j of a lane: lane * 4 + j % 4 + j / 4 * 128 (wide), else lane + 32 * j; past the end everything is 0
      Pair ms{}, vs{};
      if constexpr (BITS == 8) {
        const auto ask = [&](uint32_t unit, uint32_t to) {
          Stage::copy(base + to * Stage::kStage, t, unit, lane);
          m_next = t.m_steps[unit], v_next = t.v_steps[unit];
        };
        if (wide) {
          if (!here) {
            ask(b, slot);
            cp_async_commit();
          }
          ms = both(m_next), vs = both(v_next);
          here = u + 1 < end && u + 1 < l.first[lo + 1] && t.n - e0 >= 2 * kUnit;
          if (here) ask(b + 1, slot ^ 1);
          cp_async_commit();
          cp_async_wait<1>();
        } else {
          here = false;
          Stage::put(base + slot * Stage::kStage, t, e0, left, lane);
          ms = both(t.m_steps[b]), vs = both(t.v_steps[b]);
        }
        slot ^= 1;
      }
      Pair p[4], m[4], v[4];  // v: the root with 8-bit states
      // The whole step; EXACT with the IEEE square roots and quotients, which are right at every exponent.  Returns
      // whether it may not be right without them.
      const auto step = [&](auto exact) {
        constexpr bool EXACT = decltype(exact)::value;
        float pf[8], gf[8], mf[8], vf[8];
        if constexpr (BITS == 32) {
          if (wide) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const int64_t i = e0 + q * 128 + lane * 4;
              const Elem4 pv = load4<PBF16>(t.p, i), gv = load4<GBF16>(t.g, i), mv = load4<false>(t.m, i), vv = load4<false>(t.v, i);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                pf[q * 4 + k] = pv.f[k], gf[q * 4 + k] = gv.f[k], mf[q * 4 + k] = mv.f[k], vf[q * 4 + k] = vv.f[k];
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int o = lane + 32 * j;
              const bool in = o < left;
              pf[j] = in ? load_elem_rw(t.p, e0 + o, PBF16) : 0.0f;
              gf[j] = in ? load_elem(t.g, e0 + o, GBF16) : 0.0f;
              mf[j] = in ? static_cast<const float*>(t.m)[e0 + o] : 0.0f;
              vf[j] = in ? static_cast<const float*>(t.v)[e0 + o] : 0.0f;
            }
          }
        }
        bool odd = l.a.eps_inside_sqrt != 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (BITS == 8) {
            if (j % 2 == 0)
              Stage::half(base + (slot ^ 1) * Stage::kStage, j / 2, pf + 2 * j, gf + 2 * j, mf + 2 * j, vf + 2 * j);
          }
          Pair m2 = pair(mf[2 * j], mf[2 * j + 1]), v2 = pair(vf[2 * j], vf[2 * j + 1]), p2 = pair(pf[2 * j], pf[2 * j + 1]);
          if constexpr (BITS == 8) {
            m2 = rn.mul(m2 + both(-8388736.0f), ms);
            v2 = rn.mul(v2 + both(-8388608.0f), vs);
            v2 = rn.mul(v2, v2);
          }
          const Pair g2 = rn.mul(pair(gf[2 * j], gf[2 * j + 1]), both(scale));
          p2 = p2 + rn.mul(both(-t.lr_wd), p2);
          m2 = rn.mul(both(l.a.beta1), m2) + rn.mul(both(l.a.one_minus_beta1), g2);
          v2 = rn.mul(both(l.a.beta2), v2) + rn.mul(both(l.a.one_minus_beta2), rn.mul(g2, g2));
          const float2 mx = halves(m2), vx = halves(v2);
          Pair root, den, q;
          if constexpr (EXACT) {
            root = pair(sqrt_zsel(vx.x), sqrt_zsel(vx.y));
            den = rn.mul(root, both(l.a.c2)) + both(l.a.eps);
            if (l.a.eps_inside_sqrt) {
              const float2 x = halves(rn.mul(v2, both(l.a.c2)) + both(l.a.eps));
              den = pair(sqrt_zsel(x.x), sqrt_zsel(x.y));
            }
            const float2 d = halves(den);
            q = pair(div_zsel(mx.x, d.x), div_zsel(mx.y, d.y));
          } else {
            const float2 s = halves(sqrt_pair(v2));
            root = pair(vx.x != 0.0f ? s.x : 0.0f, vx.y != 0.0f ? s.y : 0.0f);
            den = rn.mul(root, both(l.a.c2)) + both(l.a.eps);
            const float2 d = halves(den);
            odd |= extreme(mx.x, vx.x, d.x) || extreme(mx.y, vx.y, d.y);
            q = div_pair(m2, den);
          }
          p[j] = p2 + rn.mul(both(-t.c1), q), m[j] = m2, v[j] = BITS == 8 ? root : v2;
        }
        return odd;
      };
      if (step(Flag<false>())) step(Flag<true>());
      uint32_t r[8];
      const auto draw = [&]() {
        const uint32_t key = mix32(t.key ^ uint32_t(uint64_t(e0) >> 32));
#pragma unroll
        for (int j = 0; j < 8; ++j)
          r[j] = mix32((uint32_t(e0) + (wide ? uint32_t(lane * 4 + j % 4 + j / 4 * 128) : uint32_t(lane + 32 * j))) ^ key);
      };
      if constexpr (DITHER && PBF16) draw();
      // parameters, and 32-bit states
      if (wide) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int64_t i = e0 + q * 128 + lane * 4;
          const float2 lo2 = halves(p[2 * q]), hi2 = halves(p[2 * q + 1]);
          if constexpr (BITS == 32) {
            store_pairs(static_cast<float*>(t.m), i, m[2 * q], m[2 * q + 1]);
            store_pairs(static_cast<float*>(t.v), i, v[2 * q], v[2 * q + 1]);
          }
          const uint32_t near0 = pack_bf16x2(lo2.x, lo2.y), near1 = pack_bf16x2(hi2.x, hi2.y);
          if constexpr (PBF16) {
            if constexpr (DITHER)
              store4_bf16(static_cast<uint16_t*>(t.p), i, bf16_dithered(lo2.x, r[q * 4]) | bf16_dithered(lo2.y, r[q * 4 + 1]) << 16,
                          bf16_dithered(hi2.x, r[q * 4 + 2]) | bf16_dithered(hi2.y, r[q * 4 + 3]) << 16);
            else
              store4_bf16(static_cast<uint16_t*>(t.p), i, near0, near1);
          } else {
            store_pairs(static_cast<float*>(t.p), i, p[2 * q], p[2 * q + 1]);
            if (t.copy != nullptr) store4_bf16(t.copy, i, near0, near1);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int o = lane + 32 * j;
          if (o >= left) continue;
          const float x = of(p, j);
          if constexpr (BITS == 32) static_cast<float*>(t.m)[e0 + o] = of(m, j), static_cast<float*>(t.v)[e0 + o] = of(v, j);
          if constexpr (PBF16 && DITHER)
            static_cast<uint16_t*>(t.p)[e0 + o] = uint16_t(bf16_dithered(x, r[j]));
          else
            store_elem(t.p, e0 + o, PBF16, x);
          if (!PBF16 && t.copy != nullptr) store_elem(t.copy, e0 + o, 1, x);
        }
      }
      if constexpr (BITS == 8) {
        float mtop = 0.0f, vtop = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 mf = halves(m[j]), vf = halves(v[j]);
          mtop = largest(mtop, largest(fabsf(mf.x), fabsf(mf.y))), vtop = largest(vtop, largest(vf.x, vf.y));
        }
        // (magnitude bits order like magnitudes, NaN on top)
        float minv, vinv, mstep, vstep;
        state_step(__reduce_max_sync(0xFFFFFFFFu, mag_bits(mtop)), 127.0f, &minv, &mstep);
        state_step(__reduce_max_sync(0xFFFFFFFFu, mag_bits(vtop)), 255.0f, &vinv, &vstep);
        if constexpr (DITHER && !PBF16) draw();
        uint32_t mc[8], vc[8];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          Pair x = rn.mul(m[j / 2], both(minv)), y = rn.mul(v[j / 2], both(vinv));
          const float2 rf = halves(v[j / 2]);
          if constexpr (DITHER) x = x + dither_of(r[j], r[j + 1], 0), y = y + dither_of(r[j], r[j + 1], 1);
          const float2 xf = halves(x + both(kRoundMagic)), yf = halves(y + both(kRoundMagic));
          constexpr uint32_t kZero = 0x4B400000u;  // the bits of a rounded 0
          mc[j] = __float_as_uint(xf.x), mc[j + 1] = __float_as_uint(xf.y);
          vc[j] = max(__float_as_uint(yf.x), rf.x > 0.0f ? kZero + 1 : kZero);
          vc[j + 1] = max(__float_as_uint(yf.y), rf.y > 0.0f ? kZero + 1 : kZero);
        }
        if (minv == 0.0f) {  // a block held as zeros, or as NaN
#pragma unroll
          for (int j = 0; j < 8; ++j) mc[j] = 0;
        }
        if (vinv == 0.0f) {
#pragma unroll
          for (int j = 0; j < 8; ++j) vc[j] = 0;
        }
        if (lane == 0) t.m_steps[b] = mstep, t.v_steps[b] = vstep;
        if (wide) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int64_t i = e0 + q * 128 + lane * 4;
            __stcs(reinterpret_cast<uint32_t*>(static_cast<int8_t*>(t.m) + i), low_bytes(mc + q * 4));
            __stcs(reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(t.v) + i), low_bytes(vc + q * 4));
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int o = lane + 32 * j;
            static_cast<uint8_t*>(t.m)[e0 + o] = o < left ? uint8_t(mc[j]) : uint8_t(0);
            static_cast<uint8_t*>(t.v)[e0 + o] = o < left ? uint8_t(vc[j]) : uint8_t(0);
          }
        }
      }
    }
  }
}

template <int BITS, bool PBF16, bool GBF16, bool DITHER, int MAX>
cudaError_t run(const AdamTensorList<MAX>& l, cudaStream_t s) {
  static LayerGrid grid;
  int cap = 0;
  constexpr size_t kSmem = BITS == 8 ? 2 * size_t(Staged<PBF16, GBF16>::kStage) : 0;
  const cudaError_t e =
      layer_grid(grid, reinterpret_cast<const void*>(&k_step_tensors<BITS, PBF16, GBF16, DITHER, MAX>), kThreadsAdam, kSmem, kSmem, &cap);
  if (e != cudaSuccess) return e;
  // few units: one to a warp, before any warp takes a second
  constexpr int64_t kCta = kThreadsAdam / 32;
  const int64_t units = l.first[l.count], all = cap * kCta;
  const int group = int(units >= all * kGroup ? kGroup : units <= all ? 1 : units / all);
  const int64_t want = (units + kCta * group - 1) / (kCta * group);
  k_step_tensors<BITS, PBF16, GBF16, DITHER, MAX><<<int(want < cap ? want : cap), kThreadsAdam, kSmem, s>>>(l, group);
  return cudaGetLastError();
}

template <int BITS, bool PBF16, bool DITHER, int MAX>
cudaError_t run_g(const AdamTensorList<MAX>& l, const AdamTensorsKind& k, cudaStream_t s) {
  return k.g_bf16 ? run<BITS, PBF16, true, DITHER, MAX>(l, s) : run<BITS, PBF16, false, DITHER, MAX>(l, s);
}

// out = code * step, or its square: eight values a thread.
template <bool SECOND, bool BF16>
__global__ void __launch_bounds__(256) k_state_decode(const uint2* codes, const float* steps, int64_t n, void* out, bool wide) {
  const int64_t pieces = (n + 7) / 8;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < pieces; i += int64_t(gridDim.x) * 256) {
    const uint2 w = __ldcs(codes + i);
    const Pair step = both(__ldg(steps + (i >> 5)));
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      const uint32_t c = (k < 4 ? w.x : w.y) ^ (SECOND ? 0u : 0x80808080u);
      Pair x = pair(__uint_as_float(__byte_perm(c, kTwo23Bits, 0x7440 | (k & 3))),
                    __uint_as_float(__byte_perm(c, kTwo23Bits, 0x7441 | (k & 3)))) + both(SECOND ? -8388608.0f : -8388736.0f);
      x = x * step;
      if (SECOND) x = x * x;
      const float2 f = halves(x);
      v[k] = f.x, v[k + 1] = f.y;
    }
    if (wide && i * 8 + 8 <= n) {
      if (BF16) {
        __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + i * 8),
               make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
      } else {
        store4(static_cast<float*>(out), i * 8, Elem4{{v[0], v[1], v[2], v[3]}});
        store4(static_cast<float*>(out), i * 8 + 4, Elem4{{v[4], v[5], v[6], v[7]}});
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (i * 8 + k < n) store_elem(out, i * 8 + k, BF16, v[k]);
    }
  }
}

template <bool SECOND, bool BF16>
cudaError_t run_decode(const void* codes, const float* steps, int64_t n, void* out, cudaStream_t s) {
  static LayerGrid grid;
  int cap = 0;
  const cudaError_t e = layer_grid(grid, reinterpret_cast<const void*>(&k_state_decode<SECOND, BF16>), 256, 0, 0, &cap);
  if (e != cudaSuccess) return e;
  const int64_t want = ((n + 7) / 8 + 255) / 256;
  const bool wide = reinterpret_cast<uintptr_t>(out) % 16 == 0;
  k_state_decode<SECOND, BF16><<<int(want < cap ? want : cap), 256, 0, s>>>(static_cast<const uint2*>(codes), steps, n, out, wide);
  return cudaGetLastError();
}

}  // namespace

template <int MAX>
cudaError_t launch_adam_tensors(const AdamTensorList<MAX>& l, const AdamTensorsKind& k, cudaStream_t s) {
  if (k.bits == 32) {
    if (!k.p_bf16) return run_g<32, false, false, MAX>(l, k, s);
    return k.dither ? run_g<32, true, true, MAX>(l, k, s) : run_g<32, true, false, MAX>(l, k, s);
  }
  if (k.p_bf16) return k.dither ? run_g<8, true, true, MAX>(l, k, s) : run_g<8, true, false, MAX>(l, k, s);
  return k.dither ? run_g<8, false, true, MAX>(l, k, s) : run_g<8, false, false, MAX>(l, k, s);
}
template cudaError_t launch_adam_tensors<kAdamFew>(const AdamTensorList<kAdamFew>&, const AdamTensorsKind&, cudaStream_t);
template cudaError_t launch_adam_tensors<kAdamMany>(const AdamTensorList<kAdamMany>&, const AdamTensorsKind&, cudaStream_t);

cudaError_t launch_state_decode(int second, const void* codes, const float* steps, int64_t n, void* out, int out_bf16,
                                cudaStream_t s) {
  if (second)
    return out_bf16 ? run_decode<true, true>(codes, steps, n, out, s) : run_decode<true, false>(codes, steps, n, out, s);
  return out_bf16 ? run_decode<false, true>(codes, steps, n, out, s) : run_decode<false, false>(codes, steps, n, out, s);
}

}  // namespace loco
