// fp4_dev.cuh - device helpers of the 4-bit formats (fp4.cuh).
#pragma once

#include <cuda_fp16.h>

#include "fp4.cuh"
#include "mx.cuh"
#include "ptx.cuh"

namespace moe {

// eight floats -> eight E2M1 codes, the first in the low bits
__device__ __forceinline__ uint32_t e2m1x8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// eight codes -> eight floats
__device__ __forceinline__ void e2m1_values8(uint32_t w, float* v) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(byte)));
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xffffu)));
}

// A block's scale byte from amax's bits (sign cleared; NaN and infinity are
// 0x7f800000 or more), and what its values are multiplied by to become codes.
// inv is 0 where the scale is: the codes are 0 then.
template <bool NV>
__device__ __forceinline__ uint32_t fp4_scale(uint32_t amax_bits, float t, float& inv) {
  if constexpr (NV) {
    if (amax_bits >= 0x7f800000u) { inv = 0.f; return 0x7fu; }
    const uint32_t s = e4m3x2(__fdiv_rn(__uint_as_float(amax_bits), 6.f * t), 0.f) & 0xffu;
    const float d = e4m3_value(s) * t;
    inv = d > 0.f ? fminf(__frcp_rn(d), 3.402823466e38f) : 0.f;    // (finite: 0 stays 0)
    return s;
  } else {
    if (amax_bits >= 0x7f800000u) { inv = 0.f; return 0xffu; }
    const uint32_t be = amax_bits >> 23;
    const uint32_t code = be > 2u ? be - 2u : 0u;
    inv = __uint_as_float((254u - code) << 23);
    return code;
  }
}

// eight f16 pairs' halves -> eight codes (4 words of pairs)
__device__ __forceinline__ uint32_t e2m1x8_h(const uint32_t* h) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f16x2 b0, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f16x2 b1, %2;\n\t"
      "cvt.rn.satfinite.e2m1x2.f16x2 b2, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f16x2 b3, %4;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]));
  return r;
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A tensor scale as the quantisers of bf16 values use it.  With a power of two
// quotients need no division: the quotient of an 8-bit significand and a 4-bit one
// (or 6, or their product) either is one of the halves between two codes, or at
// least 1/256 away from it, so rounding a float32 product with a reciprocal (2^-22
// off at most) to 11 or 12 bits gives the side, and the ties, of the exact
// quotient.  Scales near the ends of float32's range, whose reciprocals would leave
// it, are used times `shift`, a power of two, and so are their values
// (fp4_shift): t is 2^-117 to 2^96 then, s t and its reciprocal are normal.
struct Fp4Tensor {
  float t, inv6, inv, shift;
  bool exact;
};
__device__ __forceinline__ Fp4Tensor fp4_tensor(float t) {
  Fp4Tensor r;
  r.shift = t < 0x1p-94f ? 0x1p32f : t > 0x1p94f ? 0x1p-32f : 1.f;
  t *= r.shift;
  r.t = t;
  const uint32_t b = __float_as_uint(t);
  r.exact = (b & 0x7fffffu) == 0u && b >= (10u << 23) && b <= (223u << 23);    // 2^-117 .. 2^96
  r.inv = __uint_as_float((254u << 23) - b);      // (of a power of two)
  r.inv6 = r.inv * (1.f / 6.f);
  return r;
}

// bf16 values (words of pairs) times t.shift.  Exact, or past bf16's range, where
// its last value saturates as well, or below it, where a code is 0.
template <int N>
__device__ __forceinline__ void fp4_shift(uint32_t (&p)[N], const Fp4Tensor& t) {
  if (t.shift == 1.f) return;
  auto shifted = [&](float v) {
    const float f = v * t.shift;
    return fabsf(v) < INFINITY && fabsf(f) > 0x1.fep127f ? copysignf(0x1.fep127f, f) : f;
  };
#pragma unroll
  for (int i = 0; i < N; ++i) p[i] = pack_bf16x2(shifted(bf16_lo(p[i])), shifted(bf16_hi(p[i])));
}

// the scale byte and the multiplier of a block of bf16 values (shifted)
template <bool NV>
__device__ __forceinline__ uint32_t fp4_scale_bf16(uint32_t amax_bits, const Fp4Tensor& t,
                                                   float& inv) {
  if (!NV || !t.exact) return fp4_scale<NV>(amax_bits, t.t, inv);
  if (amax_bits >= 0x7f800000u) { inv = 0.f; return 0x7fu; }
  const float u = __uint_as_float((__float_as_uint(__uint_as_float(amax_bits) * t.inv6) + 0x800u) & ~0xfffu);
  const uint32_t s = e4m3x2(u, 0.f) & 0xffu;
  inv = s ? __fdividef(1.f, e4m3_value(s)) * t.inv : 0.f;
  return s;
}

// 8 words of bf16 pairs (16 values) -> the largest magnitude's 16 bits
__device__ __forceinline__ uint32_t bf16_amax16(const uint32_t* p) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __vmaxu2(m, p[i] & 0x7fff7fffu);
  return max(m & 0xffffu, m >> 16);
}

// 16 bf16 values (8 words) -> 16 codes (2 words).  exact: through f16's 11 bits
template <bool NV>
__device__ __forceinline__ uint2 fp4_codes16(const uint32_t* p, float inv, bool exact) {
  if (NV && !exact) {
    float u[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      u[2 * i] = bf16_lo(p[i]) * inv;
      u[2 * i + 1] = bf16_hi(p[i]) * inv;
    }
    return make_uint2(e2m1x8(u), e2m1x8(u + 8));
  }
  uint32_t h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = f16x2(bf16_lo(p[i]) * inv, bf16_hi(p[i]) * inv);
  return make_uint2(e2m1x8_h(h), e2m1x8_h(h + 4));
}

// an expert's rows and the number of its first scale tile
struct Fp4Place {
  long long off;             // the expert's first row
  long long tile0;
  int e;
};
// byte offset of (row r of the expert, block kb of K) in the scale buffer
__device__ __forceinline__ long long fp4_scale_at(long long tile0, long long r, int kb, int chunks) {
  return ((tile0 + (r >> 7)) * chunks + (kb >> 2)) * kFp4ChunkBytes +
         static_cast<long long>((r & 31) * 16 + ((r >> 5) & 3) * 4 + (kb & 3));
}

}  // namespace moe
