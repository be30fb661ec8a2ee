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

// d = (b - 127.5) / 256 of byte 0 or 1 of the random bits, exact: 2b + 1 in the low bits of 2^14, whose last place is
// 2^-9, less 2^14 + 1/2.
__device__ __forceinline__ Pair dither_of(uint32_t r0, uint32_t r1, int byte) {
  const uint32_t u0 = byte ? r0 >> 7 : r0 << 1, u1 = byte ? r1 >> 7 : r1 << 1;
  return pair(__uint_as_float((u0 & 0x1FEu) | 0x46800001u), __uint_as_float((u1 & 0x1FEu) | 0x46800001u)) + both(-16384.5f);
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

template <int BITS, bool PBF16, bool GBF16, bool DITHER, int MAX>
__global__ void __launch_bounds__(kThreadsAdam, PBF16 && DITHER ? 2 : 3) k_adam_tensors(const __grid_constant__ AdamTensorList<MAX> l, int group) {
  const int lane = threadIdx.x & 31;
  const uint32_t units = l.first[l.count];
  const uint32_t warps = gridDim.x * (kThreadsAdam / 32);
  const float scale = l.a.grad_scale != nullptr ? __ldg(l.a.grad_scale) : 1.0f;
  const Rounded rn{both(l.a.neg_zero)};
  for (uint64_t u0 = uint64_t(blockIdx.x * (kThreadsAdam / 32) + threadIdx.x / 32) * group; u0 < units;
       u0 += uint64_t(warps) * group) {
    int lo = 0, hi = l.count;  // first[lo] <= u0 < first[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (l.first[mid] <= u0)
        lo = mid;
      else
        hi = mid;
    }
    const uint32_t end = uint32_t(u0 + group < units ? u0 + group : units);
    for (uint32_t u = uint32_t(u0); u < end; ++u) {
      while (u >= l.first[lo + 1]) ++lo;
      const AdamTensor& t = l.t[lo];
      const uint32_t b = u - l.first[lo];       // the unit within its tensor
      const int64_t e0 = int64_t(b) * kUnit;
      const int left = t.n - e0 < kUnit ? int(t.n - e0) : kUnit;
      const bool wide = t.wide && left == kUnit;
      // element j of a lane: lane * 4 + j % 4 + j / 4 * 128 (wide), else lane + 32 * j; past the end everything is 0
      float p[8], g[8], m[8], v[8];
      if (wide) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int64_t i = e0 + q * 128 + lane * 4;
          const Elem4 pv = load4<PBF16>(t.p, i), gv = load4<GBF16>(t.g, i);
#pragma unroll
          for (int k = 0; k < 4; ++k) p[q * 4 + k] = pv.f[k], g[q * 4 + k] = gv.f[k];
          if constexpr (BITS == 32) {
            const Elem4 mv = load4<false>(t.m, i), vv = load4<false>(t.v, i);
#pragma unroll
            for (int k = 0; k < 4; ++k) m[q * 4 + k] = mv.f[k], v[q * 4 + k] = vv.f[k];
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int o = lane + 32 * j;
          const bool in = o < left;
          p[j] = in ? load_elem_rw(t.p, e0 + o, PBF16) : 0.0f;
          g[j] = in ? load_elem(t.g, e0 + o, GBF16) : 0.0f;
          if constexpr (BITS == 32) {
            m[j] = in ? static_cast<const float*>(t.m)[e0 + o] : 0.0f;
            v[j] = in ? static_cast<const float*>(t.v)[e0 + o] : 0.0f;
          }
        }
      }
      Pair ms{}, vs{};
      if constexpr (BITS == 8) {
        ms = both(t.m_steps[b]), vs = both(t.v_steps[b]);
        // codes under the exponent of 2^23: the floats 2^23 + code (and 128 for a signed one)
        if (wide) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int64_t i = e0 + q * 128 + lane * 4;
            const uint32_t mw = __ldcs(reinterpret_cast<const uint32_t*>(static_cast<const int8_t*>(t.m) + i)) ^ 0x80808080u;
            const uint32_t vw = __ldcs(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.v) + i));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              m[q * 4 + k] = __uint_as_float(__byte_perm(mw, kTwo23Bits, 0x7440 | k));
              v[q * 4 + k] = __uint_as_float(__byte_perm(vw, kTwo23Bits, 0x7440 | k));
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            m[j] = __uint_as_float(kTwo23Bits | (static_cast<const uint8_t*>(t.m)[e0 + lane + 32 * j] ^ 0x80u));
            v[j] = __uint_as_float(kTwo23Bits | static_cast<const uint8_t*>(t.v)[e0 + lane + 32 * j]);
          }
        }
      }
      float root[8];
      uint32_t mtop = 0, vtop = 0;
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        Pair m2 = pair(m[j], m[j + 1]), v2 = pair(v[j], v[j + 1]), p2 = pair(p[j], p[j + 1]), g2 = pair(g[j], g[j + 1]);
        if constexpr (BITS == 8) {
          m2 = rn.mul(m2 + both(-8388736.0f), ms);
          v2 = rn.mul(v2 + both(-8388608.0f), vs);
          v2 = rn.mul(v2, v2);
        }
        g2 = rn.mul(g2, both(scale));
        p2 = p2 + rn.mul(both(-t.lr_wd), p2);
        m2 = rn.mul(both(l.a.beta1), m2) + rn.mul(both(l.a.one_minus_beta1), g2);
        v2 = rn.mul(both(l.a.beta2), v2) + rn.mul(both(l.a.one_minus_beta2), rn.mul(g2, g2));
        const float2 mf = halves(m2), vf = halves(v2);
        m[j] = mf.x, m[j + 1] = mf.y, v[j] = vf.x, v[j + 1] = vf.y;
        if (BITS == 8 || !l.a.eps_inside_sqrt) root[j] = sqrt_zsel(vf.x), root[j + 1] = sqrt_zsel(vf.y);
        Pair den;
        if (l.a.eps_inside_sqrt) {
          const float2 x = halves(rn.mul(v2, both(l.a.c2)) + both(l.a.eps));
          den = pair(sqrt_zsel(x.x), sqrt_zsel(x.y));
        } else {
          den = rn.mul(pair(root[j], root[j + 1]), both(l.a.c2)) + both(l.a.eps);
        }
        const float2 df = halves(den);
        p2 = p2 + rn.mul(both(-t.c1), pair(div_zsel(mf.x, df.x), div_zsel(mf.y, df.y)));
        const float2 pf = halves(p2);
        p[j] = pf.x, p[j + 1] = pf.y;
        if constexpr (BITS == 8) {
          mtop = max(mtop, max(mag_bits(mf.x), mag_bits(mf.y)));
          vtop = max(vtop, max(__float_as_uint(root[j]), __float_as_uint(root[j + 1])) & 0x7FFFFFFFu);
        }
      }
      uint32_t r[8];
      if constexpr (DITHER) {
        const uint32_t key = mix32(t.key ^ uint32_t(uint64_t(e0) >> 32));
#pragma unroll
        for (int j = 0; j < 8; ++j)
          r[j] = mix32((uint32_t(e0) + (wide ? uint32_t(lane * 4 + j % 4 + j / 4 * 128) : uint32_t(lane + 32 * j))) ^ key);
      }
      if constexpr (BITS == 8) {
        mtop = __reduce_max_sync(0xFFFFFFFFu, mtop);
        vtop = __reduce_max_sync(0xFFFFFFFFu, vtop);
        float minv, vinv, mstep, vstep;
        state_step(mtop, 127.0f, &minv, &mstep);
        state_step(vtop, 255.0f, &vinv, &vstep);
        uint32_t mc[8], vc[8];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          Pair x = rn.mul(pair(m[j], m[j + 1]), both(minv)), y = rn.mul(pair(root[j], root[j + 1]), both(vinv));
          if constexpr (DITHER) x = x + dither_of(r[j], r[j + 1], 0), y = y + dither_of(r[j], r[j + 1], 1);
          const float2 xf = halves(x + both(kRoundMagic)), yf = halves(y + both(kRoundMagic));
          constexpr uint32_t kZero = 0x4B400000u;  // the bits of a rounded 0
          mc[j] = __float_as_uint(xf.x), mc[j + 1] = __float_as_uint(xf.y);
          vc[j] = max(__float_as_uint(yf.x), root[j] > 0.0f ? kZero + 1 : kZero);
          vc[j + 1] = max(__float_as_uint(yf.y), root[j + 1] > 0.0f ? kZero + 1 : kZero);
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
            __stcs(reinterpret_cast<uint32_t*>(static_cast<int8_t*>(t.m) + i),
                   __byte_perm(__byte_perm(mc[q * 4], mc[q * 4 + 1], 0x0040), __byte_perm(mc[q * 4 + 2], mc[q * 4 + 3], 0x0040),
                               0x5410));
            __stcs(reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(t.v) + i),
                   __byte_perm(__byte_perm(vc[q * 4], vc[q * 4 + 1], 0x0040), __byte_perm(vc[q * 4 + 2], vc[q * 4 + 3], 0x0040),
                               0x5410));
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
      if (wide) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int64_t i = e0 + q * 128 + lane * 4;
          const Elem4 pv{{p[q * 4], p[q * 4 + 1], p[q * 4 + 2], p[q * 4 + 3]}};
          if constexpr (BITS == 32) {
            store4(static_cast<float*>(t.m), i, Elem4{{m[q * 4], m[q * 4 + 1], m[q * 4 + 2], m[q * 4 + 3]}});
            store4(static_cast<float*>(t.v), i, Elem4{{v[q * 4], v[q * 4 + 1], v[q * 4 + 2], v[q * 4 + 3]}});
          }
          const uint32_t near0 = pack_bf16x2(pv.f[0], pv.f[1]), near1 = pack_bf16x2(pv.f[2], pv.f[3]);
          if constexpr (PBF16) {
            if constexpr (DITHER)
              store4_bf16(static_cast<uint16_t*>(t.p), i,
                          bf16_dithered(pv.f[0], r[q * 4]) | bf16_dithered(pv.f[1], r[q * 4 + 1]) << 16,
                          bf16_dithered(pv.f[2], r[q * 4 + 2]) | bf16_dithered(pv.f[3], r[q * 4 + 3]) << 16);
            else
              store4_bf16(static_cast<uint16_t*>(t.p), i, near0, near1);
          } else {
            store4(static_cast<float*>(t.p), i, pv);
            if (t.copy != nullptr) store4_bf16(t.copy, i, near0, near1);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int o = lane + 32 * j;
          if (o >= left) continue;
          if constexpr (BITS == 32) static_cast<float*>(t.m)[e0 + o] = m[j], static_cast<float*>(t.v)[e0 + o] = v[j];
          if constexpr (PBF16 && DITHER)
            static_cast<uint16_t*>(t.p)[e0 + o] = uint16_t(bf16_dithered(p[j], r[j]));
          else
            store_elem(t.p, e0 + o, PBF16, p[j]);
          if (!PBF16 && t.copy != nullptr) store_elem(t.copy, e0 + o, 1, p[j]);
        }
      }
    }
  }
}

template <int BITS, bool PBF16, bool GBF16, bool DITHER, int MAX>
cudaError_t run(const AdamTensorList<MAX>& l, cudaStream_t s) {
  static LayerGrid grid;
  int cap = 0;
  const cudaError_t e =
      layer_grid(grid, reinterpret_cast<const void*>(&k_adam_tensors<BITS, PBF16, GBF16, DITHER, MAX>), kThreadsAdam, 0, 0, &cap);
  if (e != cudaSuccess) return e;
  // few units: one to a warp, before any warp takes a second
  constexpr int64_t kCta = kThreadsAdam / 32;
  const int64_t units = l.first[l.count], all = cap * kCta;
  const int group = int(units >= all * kGroup ? kGroup : units <= all ? 1 : units / all);
  const int64_t want = (units + kCta * group - 1) / (kCta * group);
  k_adam_tensors<BITS, PBF16, GBF16, DITHER, MAX><<<int(want < cap ? want : cap), kThreadsAdam, 0, s>>>(l, group);
  return cudaGetLastError();
}

template <int BITS, bool PBF16, bool DITHER, int MAX>
cudaError_t run_g(const AdamTensorList<MAX>& l, const AdamTensorsKind& k, cudaStream_t s) {
  return k.g_bf16 ? run<BITS, PBF16, true, DITHER, MAX>(l, s) : run<BITS, PBF16, false, DITHER, MAX>(l, s);
}

// out = code * step, or its square: four values a thread.
template <bool SECOND, bool BF16>
__global__ void __launch_bounds__(256) k_state_decode(const uint32_t* codes, const float* steps, int64_t n, void* out, bool wide) {
  const int64_t words = (n + 3) / 4;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < words; i += int64_t(gridDim.x) * 256) {
    const uint32_t w = __ldcs(codes + i) ^ (SECOND ? 0u : 0x80808080u);
    const float step = __ldg(steps + i / (kUnit / 4));
    Elem4 v;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v.f[k] = __fmul_rn(__uint_as_float(__byte_perm(w, kTwo23Bits, 0x7440 | k)) - (SECOND ? 8388608.0f : 8388736.0f), step);
      if (SECOND) v.f[k] = __fmul_rn(v.f[k], v.f[k]);
    }
    if (wide && i * 4 + 4 <= n) {
      if (BF16)
        store4_bf16(static_cast<uint16_t*>(out), i * 4, pack_bf16x2(v.f[0], v.f[1]), pack_bf16x2(v.f[2], v.f[3]));
      else
        store4(static_cast<float*>(out), i * 4, v);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i * 4 + k < n) store_elem(out, i * 4 + k, BF16, v.f[k]);
    }
  }
}

template <bool SECOND, bool BF16>
cudaError_t run_decode(const void* codes, const float* steps, int64_t n, void* out, cudaStream_t s) {
  static LayerGrid grid;
  int cap = 0;
  const cudaError_t e = layer_grid(grid, reinterpret_cast<const void*>(&k_state_decode<SECOND, BF16>), 256, 0, 0, &cap);
  if (e != cudaSuccess) return e;
  const int64_t want = ((n + 3) / 4 + 255) / 256;
  const bool wide = reinterpret_cast<uintptr_t>(out) % (BF16 ? 8 : 16) == 0;
  k_state_decode<SECOND, BF16><<<int(want < cap ? want : cap), 256, 0, s>>>(static_cast<const uint32_t*>(codes), steps, n, out, wide);
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
