// Device helpers of the 8-bit activation checkpoints (sm_103a): element
// types, the group step and the codes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gc_common.cuh"

namespace gc {

constexpr int ACT_GROUP = 32;  // columns that share one step

inline __host__ __device__ int64_t act_ldc(int64_t cols) { return (cols + 31) / 32 * 32; }

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Element i of a vector of run-time type.
__device__ __forceinline__ float load_as_f32(const void* p, int dtype, int64_t i) {
  if (dtype == GC_F32) return static_cast<const float*>(p)[i];
  if (dtype == GC_BF16) return to_f32(static_cast<const __nv_bfloat16*>(p)[i]);
  return to_f32(static_cast<const __half*>(p)[i]);
}

// The step byte b of a group whose largest magnitude has the bits `top`
// (sign clear; a NaN's bits are above infinity's).  top / 2^(E - 6) is in
// [64, 128), E the magnitude's unbiased exponent, and rounds to 128 from
// 127.5 on, that is from the significand 0x7f0000 on: adding 0x10000 to the
// bits carries exactly those into the next exponent.  2^(b - 127) is kept
// normal (b >= 1) and below 2^122 (else 64 * step would overflow fp32).
__device__ __forceinline__ uint32_t act_step(uint32_t top) {
  if (top >= 0x7f800000u) return 255u;
  const int e = min((int)((top + 0x10000u) >> 23), 254);
  return (uint32_t)max(e - 6, 1);
}
// 1 / step, 0 for a group that is not finite.
__device__ __forceinline__ float act_inverse(uint32_t b) { return b == 255u ? 0.0f : __uint_as_float((254u - b) << 23); }
__device__ __forceinline__ float act_scale(uint32_t b) { return __uint_as_float(b << 23); }

// rne(x / step) in [-127, 127], as the low byte of an integer; 0 for a group
// that is not finite (inverse 0; NaN * 0 would not be).
__device__ __forceinline__ int act_code(float x, float inverse) {
  const float v = fminf(fmaxf(__fmul_rn(x, inverse), -127.0f), 127.0f);
  return inverse == 0.0f ? 0 : __float2int_rn(v);
}

}  // namespace gc

// Runs a statement with T the element type of a valid dtype.
#define GC_BY_DTYPE(dtype, T, ...)                                \
  do {                                                            \
    if ((dtype) == GC_F32) { using T = float; __VA_ARGS__; }      \
    else if ((dtype) == GC_BF16) { using T = __nv_bfloat16; __VA_ARGS__; } \
    else { using T = __half; __VA_ARGS__; }                       \
  } while (0)
