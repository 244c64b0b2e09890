// 8-bit codes of a cached vector (one token's key or value of one head), shared
// by the kernels that write, read and attend over them (internal).
//
// A vector x is held as codes c_d and one float32 scale s, x_d ~ s c_d:
//   e4m3  s = 2^n, the smallest power of two with max |x| <= 448 s; c_d is x_d / s
//         to nearest even.  A power of two costs a floating code nothing (its steps
//         are relative) and makes s c_d exact in bfloat16: no second rounding.
//   int8  s = max |x| / 127, c_d = round(x_d (127 / max |x|)).
// max |x| below 2^-100: s = 0 and codes 0.  A vector that is not finite has
// s = NaN and codes 0, so that whoever reads it gets NaN.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sv {
namespace codes {

enum { kNone = 0, kE4m3 = 1, kInt8 = 2 };

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// the scale of a vector whose largest magnitude has these bits, and what its elements are multiplied by
template <int C>
__device__ __forceinline__ void scale_of(uint32_t top_bits, float* scale, float* inv) {
  if (top_bits >= 0x7F800000u) {
    *scale = __uint_as_float(0x7FC00000u);
    *inv = 0.f;
  } else if (top_bits < (uint32_t)(127 - 100) << 23) {
    *scale = 0.f;
    *inv = 0.f;
  } else if (C == kE4m3) {
    // top = m 2^e: 448 = 1.75 2^8
    const uint32_t e = (top_bits >> 23) - 8u + ((top_bits & 0x7FFFFFu) > 0x600000u ? 1u : 0u);
    *scale = __uint_as_float(e << 23);
    *inv = __uint_as_float((254u - e) << 23);
  } else {
    const float top = __uint_as_float(top_bits);
    *scale = top / 127.f;
    *inv = 127.f / top;
  }
}

// four codes, the first in the low byte
template <int C>
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d, float inv) {
  if (inv == 0.f) return 0u;                     // also where the elements are not finite
  if constexpr (C == kE4m3) {
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, lo, true);
  } else {
    const uint32_t x = (uint32_t)(int)rintf(a * inv) & 0xFFu, y = (uint32_t)(int)rintf(b * inv) & 0xFFu;
    const uint32_t z = (uint32_t)(int)rintf(c * inv) & 0xFFu, w = (uint32_t)(int)rintf(d * inv);
    return x | y << 8 | z << 16 | w << 24;
  }
}

// what four codes stand for, without the scale
template <int C>
__device__ __forceinline__ void unpack4(uint32_t w, float* x) {
  if constexpr (C == kE4m3) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    const f2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    x[0] = a[0];
    x[1] = a[1];
    x[2] = b[0];
    x[3] = b[1];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = (float)(int8_t)(w >> (8 * i));
  }
}

}  // namespace codes
}  // namespace sv
