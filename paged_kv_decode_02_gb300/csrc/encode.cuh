// encode.cuh -- the one-byte codes of cached rows (append.cu, rotate.cu).
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace pkv {

// Code of x / s for each one-byte format. INT8: clamp(rint(x / s), -127, 127). FP8:
// the conversion instruction's round-to-nearest-even with saturation to the largest
// finite code (448 for E4M3, 57344 for E5M2). Both divisions are IEEE.
template <int CODE>
struct Encode8;
template <>
struct Encode8<CODE_I8> {
  static constexpr float kMax = 127.f;
  __device__ static __forceinline__ uint8_t code(float x, float s) {
    return uint8_t(int8_t(max(-127, min(127, __float2int_rn(__fdiv_rn(x, s))))));
  }
};
template <>
struct Encode8<CODE_E4M3> {
  static constexpr float kMax = 448.f;
  __device__ static __forceinline__ uint8_t code(float x, float s) {
    return uint8_t(__nv_cvt_float_to_fp8(__fdiv_rn(x, s), __NV_SATFINITE, __NV_E4M3));
  }
};
template <>
struct Encode8<CODE_E5M2> {
  static constexpr float kMax = 57344.f;
  __device__ static __forceinline__ uint8_t code(float x, float s) {
    return uint8_t(__nv_cvt_float_to_fp8(__fdiv_rn(x, s), __NV_SATFINITE, __NV_E5M2));
  }
};

// Codes of a row's elements over one scale, as Encode8 gives them, with one reciprocal per
// row in place of a division per element. By Markstein's theorem (IBM J. Res. Dev. 34(1),
// 1990) the correctly rounded quotient is q + (x - q s) r, fused, for r the correctly
// rounded reciprocal of s and q = x r, as long as x - q s is exact: with s from 2^-80 to
// 2^100 it is for |x| >= 2^-102, and below that x / s is under half of every format's
// smallest code. Other scales divide.
template <int CODE>
struct RowEncoder {
  float s, r;
  bool fast;
  __device__ __forceinline__ explicit RowEncoder(float s_)
      : s(s_), r(1.f / s_), fast(s_ >= 0x1p-80f && s_ <= 0x1p100f) {}
  // codes of x[0].x, x[0].y, x[1].x, x[1].y, the first in the low byte
  __device__ __forceinline__ uint32_t four(const float2* x) const {
    if (!fast) {
      return uint32_t(Encode8<CODE>::code(x[0].x, s)) |
             uint32_t(Encode8<CODE>::code(x[0].y, s)) << 8 |
             uint32_t(Encode8<CODE>::code(x[1].x, s)) << 16 |
             uint32_t(Encode8<CODE>::code(x[1].y, s)) << 24;
    }
    float q[4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float2 r2 = make_float2(r, r), t = __fmul2_rn(x[e], r2);
      const float2 y = __ffma2_rn(__ffma2_rn(t, make_float2(-s, -s), x[e]), r2, t);
      q[2 * e] = y.x;
      q[2 * e + 1] = y.y;
    }
    if constexpr (CODE == CODE_I8) {  // |q| rounds to 127 at most: |x| <= 127 s (1 + 2^-24)
      const int i0 = __float2int_rn(q[0]), i1 = __float2int_rn(q[1]);
      const int i2 = __float2int_rn(q[2]), i3 = __float2int_rn(q[3]);
      return prmt(prmt(i0, i1, 0x0040u), prmt(i2, i3, 0x0040u), 0x5410u);
    } else {
      constexpr auto kind = CODE == CODE_E4M3 ? __NV_E4M3 : __NV_E5M2;
      const float2 lo = make_float2(q[0], q[1]), hi = make_float2(q[2], q[3]);
      return uint32_t(__nv_cvt_float2_to_fp8x2(lo, __NV_SATFINITE, kind)) |
             uint32_t(__nv_cvt_float2_to_fp8x2(hi, __NV_SATFINITE, kind)) << 16;
    }
  }
};

}  // namespace pkv
