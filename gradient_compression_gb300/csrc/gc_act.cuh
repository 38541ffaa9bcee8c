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

// ---------------------------------------------------------------- chunks
// The streaming kernels give a lane 8 consecutive columns (16 bytes of a
// 16-bit type, 8 bytes of codes), four lanes a group of 32; a group's lanes
// are always four of one warp, from a multiple of four on.
constexpr int CHUNK = 8;

// 8 elements as they are in memory.
template <typename T>
struct alignas(16) Raw8 {
  T e[CHUNK];
};

// `n` of the 8 elements from p on, zeros after them.  VEC: p is 16-byte
// aligned.  Read past L1, which keeps what is used again.
template <typename T, bool VEC>
__device__ __forceinline__ Raw8<T> load_chunk(const T* p, int n) {
  Raw8<T> r;
  if (VEC && n == CHUNK) {
    uint4* w = reinterpret_cast<uint4*>(&r);
#pragma unroll
    for (int i = 0; i < (int)sizeof(r) / 16; ++i)
      asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                   : "l"(reinterpret_cast<const uint4*>(p) + i)
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < CHUNK; ++i) r.e[i] = i < n ? p[i] : from_f32<T>(0.0f);
  }
  return r;
}

template <typename T>
__device__ __forceinline__ void unpack(const Raw8<T>& r, float (&v)[CHUNK]) {
#pragma unroll
  for (int i = 0; i < CHUNK; ++i) v[i] = to_f32(r.e[i]);
}

// Writes n of the 8 values.  Without VEC a warp's chunks go through `buf`
// (256 floats of its own): stores of one element per lane at 8 elements'
// distance would be eight times the sectors.  All lanes of the warp take part.
template <typename T, bool VEC>
__device__ __forceinline__ void store_chunk(T* p, int n, const float (&v)[CHUNK], float* buf) {
  if (VEC) {
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < CHUNK; ++i) r.e[i] = from_f32<T>(v[i]);
    if (n == CHUNK) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(r) / 16; ++i)
        reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(&r)[i];
    } else {
#pragma unroll
      for (int i = 0; i < CHUNK; ++i)
        if (i < n) p[i] = r.e[i];
    }
  } else {
    const int lane = threadIdx.x & 31;
    __syncwarp();
    reinterpret_cast<float4*>(buf)[2 * lane] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(buf)[2 * lane + 1] = make_float4(v[4], v[5], v[6], v[7]);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < CHUNK; ++j) {
      const int from = 4 * j + (lane >> 3);
      T* q = reinterpret_cast<T*>(__shfl_sync(FULL, reinterpret_cast<unsigned long long>(p), from));
      if ((lane & 7) < __shfl_sync(FULL, n, from)) q[lane & 7] = from_f32<T>(buf[32 * j + lane]);
    }
  }
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// The step byte of the group that this lane's 8 values belong to.
__device__ __forceinline__ uint32_t chunk_step(const float (&v)[CHUNK]) {
  float top = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < CHUNK; ++i) top = max_nan(top, fabsf(v[i]));
  top = max_nan(top, __shfl_xor_sync(FULL, top, 1));
  top = max_nan(top, __shfl_xor_sync(FULL, top, 2));
  return act_step(__float_as_uint(top));
}
// The 8 codes under step b.  Adding 1.5 * 2^23 rounds to an integer in the low
// bits.  Only the largest finite step (b = 248) can meet magnitudes that round
// past 127.
__device__ __forceinline__ uint2 chunk_codes(const float (&v)[CHUNK], uint32_t b) {
  const float inverse = act_inverse(b);
  uint32_t w[CHUNK];
#pragma unroll
  for (int i = 0; i < CHUNK; ++i) w[i] = __float_as_uint(__fmaf_rn(v[i], inverse, 12582912.0f));
  if (__builtin_expect(b >= 248u, 0)) {
#pragma unroll
    for (int i = 0; i < CHUNK; ++i)
      w[i] = __float_as_uint(__fadd_rn(fminf(fmaxf(__fmul_rn(v[i], inverse), -127.0f), 127.0f), 12582912.0f));
  }
  uint2 c;
  c.x = __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
  c.y = __byte_perm(__byte_perm(w[4], w[5], 0x0040), __byte_perm(w[6], w[7], 0x0040), 0x5410);
  return b == 255u ? make_uint2(0u, 0u) : c;
}
// The values of 8 codes: code + 128 in the low byte of 2^23's significand.
__device__ __forceinline__ void chunk_values(uint2 c, uint32_t b, float (&v)[CHUNK]) {
  const float scale = act_scale(b);
  const uint32_t x = c.x ^ 0x80808080u, y = c.y ^ 0x80808080u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = __fmul_rn(__fsub_rn(__uint_as_float(__byte_perm(x, 0x4B000000u, 0x7440 + i)), 8388736.0f), scale);
    v[4 + i] = __fmul_rn(__fsub_rn(__uint_as_float(__byte_perm(y, 0x4B000000u, 0x7440 + i)), 8388736.0f), scale);
  }
}

__device__ __forceinline__ uint2 load_codes(const int8_t* p) {
  uint2 c;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(c.x), "=r"(c.y) : "l"(p) : "memory");
  return c;
}

// ---------------------------------------------------------------- rings
// Loads in flight without registers for them: each thread copies its own
// chunks of the rows ahead into slots of shared memory that only it reads, so
// that no barrier is needed.  Each copy_group() closes what was copied since
// the last; wait_groups<N>() leaves the newest N groups in flight.
__device__ __forceinline__ void copy_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_groups() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// A thread's slots of 8 elements: the threads' 16-byte words side by side.
template <typename T>
struct Ring {
  static constexpr int WORDS = (int)sizeof(Raw8<T>) / 16;
  uint32_t at;      // shared address of this thread's word of slot 0
  uint32_t stride;  // bytes from word to word: 16 per thread
  __device__ __forceinline__ Ring(void* shared, int threads)
      : at((uint32_t)__cvta_generic_to_shared(shared) + threadIdx.x * 16u), stride((uint32_t)threads * 16u) {}
  static constexpr size_t bytes(int slots, int threads) { return (size_t)slots * WORDS * threads * 16; }
  // n elements from p on (16-byte aligned, and valid even for n = 0), zeros after them.
  __device__ __forceinline__ void copy(int slot, const T* p, int n) const {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
      const int b = min(max(n * (int)sizeof(T) - 16 * i, 0), 16);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at + (uint32_t)(slot * WORDS + i) * stride),
                   "l"(reinterpret_cast<const char*>(p) + (b > 0 ? 16 * i : 0)), "r"(b)
                   : "memory");
    }
  }
  __device__ __forceinline__ void copy(int slot, const T* p) const {  // all 8
#pragma unroll
    for (int i = 0; i < WORDS; ++i)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at + (uint32_t)(slot * WORDS + i) * stride),
                   "l"(reinterpret_cast<const char*>(p) + 16 * i)
                   : "memory");
  }
  __device__ __forceinline__ Raw8<T> take(int slot) const {
    Raw8<T> r;
    uint4* w = reinterpret_cast<uint4*>(&r);
#pragma unroll
    for (int i = 0; i < WORDS; ++i)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                   : "r"(at + (uint32_t)(slot * WORDS + i) * stride)
                   : "memory");
    return r;
  }
};
// The same for 8 codes.
struct CodeRing {
  uint32_t at, stride;
  __device__ __forceinline__ CodeRing(void* shared, int threads)
      : at((uint32_t)__cvta_generic_to_shared(shared) + threadIdx.x * 8u), stride((uint32_t)threads * 8u) {}
  static constexpr size_t bytes(int slots, int threads) { return (size_t)slots * threads * 8; }
  __device__ __forceinline__ void copy(int slot, const int8_t* p, bool in) const {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(at + (uint32_t)slot * stride), "l"(p), "r"(in ? 8 : 0)
                 : "memory");
  }
  __device__ __forceinline__ uint2 take(int slot) const {
    uint2 c;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(c.x), "=r"(c.y) : "r"(at + (uint32_t)slot * stride) : "memory");
    return c;
  }
};

// How the streaming kernels of gc_act.cu cut a matrix: a CTA of 256 threads
// takes 2^wide chunks of 256 / 2^wide rows at a time, from row blockIdx.y *
// slab on to the end of its slab.  A thread's columns never change, so the
// loop over the rows only adds the strides.
struct Tiling {
  int64_t rows, slab;
  int32_t wide, c8s, cols;  // c8s: chunks per row, pad included
};
struct Place {
  int64_t r, end;   // this thread's row, the slab's end
  int32_t step;     // rows to the next
  int32_t c8, n;    // its chunk, elements of it inside the row
  bool in;          // the chunk exists (its row may still be past the end)
};
__device__ __forceinline__ Place place(const Tiling& t) {
  Place p;
  const int rb = threadIdx.x >> t.wide;
  p.step = 256 >> t.wide;
  p.c8 = (int)(blockIdx.x << t.wide) + (int)(threadIdx.x & ((1u << t.wide) - 1u));
  p.r = (int64_t)blockIdx.y * t.slab + rb;
  p.end = min((int64_t)(blockIdx.y + 1) * t.slab, t.rows);
  p.in = p.c8 < t.c8s;
  const int64_t left = (int64_t)t.cols - (int64_t)p.c8 * CHUNK;
  p.n = left < 0 ? 0 : (left < CHUNK ? (int)left : CHUNK);
  return p;
}

}  // namespace gc

// Runs a statement with T the element type of a valid dtype.
#define GC_BY_DTYPE(dtype, T, ...)                                \
  do {                                                            \
    if ((dtype) == GC_F32) { using T = float; __VA_ARGS__; }      \
    else if ((dtype) == GC_BF16) { using T = __nv_bfloat16; __VA_ARGS__; } \
    else { using T = __half; __VA_ARGS__; }                       \
  } while (0)
