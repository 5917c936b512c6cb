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

}  // namespace pkv
