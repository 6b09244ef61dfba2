// 16-bit elements, and their codes in 8 bits: round(127 v / peak), peak the largest magnitude of the elements that share
// a scale of peak / 127.
#pragma once
#include <cuda_runtime.h>
#include "common.cuh"

namespace nvfp4moe {

// Pairs of BF16 or FP16 elements as FP32.
template <bool kF16>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
  if (kF16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <bool kF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if (kF16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <bool kF16>
__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack16<kF16>(u[i]);
    v[2 * i] = f.x, v[2 * i + 1] = f.y;
  }
}
template <bool kF16>
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack16<kF16>(v[0], v[1]), pack16<kF16>(v[2], v[3]), pack16<kF16>(v[4], v[5]), pack16<kF16>(v[6], v[7]));
}

// Peaks are compared as FP32 bits: infinities, and NaNs behind them, are larger than every number.
__device__ __forceinline__ unsigned magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
// The largest magnitude of 8 elements, as the bits of an element; NaNs and infinities are larger than every number.
__device__ __forceinline__ unsigned peak_of(const uint4& w) {
  const unsigned m = __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu), __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
  return max(m & 0xFFFFu, m >> 16);
}

// Whether the functions below can take a peak.  Others (zero, next to underflow, infinite, NaN) are the caller's.
__device__ __forceinline__ bool plain_peak(float peak) { return peak >= 0x1p-100f && peak <= 0x1p100f; }

// To the nearest, ties to even, of a quotient evaluated in 64 bits: that of 127 v and peak as FP32 numbers, or as products
// of two 16-bit ones, is a midpoint or more than 2^-40 of its value away from it.
__device__ __forceinline__ int code_of_64(double v, double peak) { return (int)rint(127.0 * v / peak); }

constexpr float kCodeMagic = 12582912.0f;  // 1.5 2^23: adding it rounds to an integer, whose low byte is the sum's

template <int N>
__device__ __forceinline__ void pack_codes(const float (&m)[N], uint32_t (&out)[N / 4]) {  // of sums with kCodeMagic
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const uint32_t a = __byte_perm(__float_as_uint(m[4 * i]), __float_as_uint(m[4 * i + 1]), 0x0040);
    const uint32_t b = __byte_perm(__float_as_uint(m[4 * i + 2]), __float_as_uint(m[4 * i + 3]), 0x0040);
    out[i] = __byte_perm(a, b, 0x5410);
  }
}

// The codes of N elements (11 significant bits and fewer), four to a word, exactly, in three instructions each.
// The quotient 127 v / peak is a midpoint n + 1/2, of at most 9 bits, or 2^-19 of its value and more away from one (127 v
// and peak are integers below 254 2^11 times powers of two).  inv is 127 / peak times 1 + 2^-22, so that v inv is above the
// quotient's magnitude by 1 to 7.1 times 2^-24 of it, whatever the roundings, that is by less than 8 of its last places:
// without its three last bits a midpoint is itself again, to be rounded to even, and nothing else has passed one.
template <int N>
__device__ __forceinline__ void codes_of_elements(const float (&v)[N], float peak, uint32_t (&out)[N / 4]) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(peak));
  const float inv = fmaf(r, fmaf(-peak, r, 1.0f), r) * 127.00003f;  // 127 (1 + 2^-22)
  float m[N];
#pragma unroll
  for (int i = 0; i < N; ++i) m[i] = __uint_as_float(__float_as_uint(v[i] * inv) & ~7u) + kCodeMagic;
  pack_codes(m, out);
}

// The codes of N products of two elements, exactly.  In FP32 the quotient is off by less than 1e-5; where that leaves two
// codes possible, 127 v less the code times the peak decides.  kBits, the values' significant bits: up to 16 that
// remainder is exact in FP32 (127 v and code times peak have at most 23 bits, and a value whose code is not zero lies at
// most 8 binary places below the peak); beyond, the quotient is evaluated in 64 bits.
template <int kBits, int N>
__device__ __forceinline__ void codes_of_products(const float (&v)[N], float peak, uint32_t (&out)[N / 4]) {
  constexpr float kMagic = kCodeMagic;
  const float inv = 127.0f / peak;
  float m[N], near = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    m[i] = fmaf(v[i], inv, kMagic);
    near = fmaxf(near, fabsf(fmaf(v[i], inv, kMagic - m[i])));
  }
  if (near > 0.49998f) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float r = m[i] - kMagic;
      if (fabsf(fmaf(v[i], inv, -r)) > 0.49998f) {
        if (kBits <= 16) {
          const float rem = fmaf(-r, peak, 127.0f * v[i]), a = 2.0f * fabsf(rem);
          if (a > peak || (a == peak && (__float_as_uint(m[i]) & 1u))) m[i] += copysignf(1.0f, rem);
        } else {
          m[i] = kMagic + (float)code_of_64(v[i], peak);
        }
      }
    }
  }
  pack_codes(m, out);
}

// peak / 127, correctly rounded for a peak that plain_peak takes.
__device__ __forceinline__ float scale_of_peak(float peak) {
  const float s = peak * (1.0f / 127.0f);
  return fmaf(fmaf(-s, 127.0f, peak), 1.0f / 127.0f, s);
}

// Four codes as FP32: each byte, its sign bit turned over, as the low byte of 2^23 + 128 + code.
__device__ __forceinline__ void codes_to_f32(uint32_t w, float (&v)[4]) {
  const uint32_t u = w ^ 0x80808080u;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 + i)) - 8388736.0f;
}

}  // namespace nvfp4moe
