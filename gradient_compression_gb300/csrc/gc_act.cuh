// Device helpers of the 8-bit activation checkpoints (sm_103a): element
// types, the group step and the codes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gc_common.cuh"
#include "gc_host.h"

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

template <typename T>
__device__ __forceinline__ void unpack(const Raw8<T>& r, float (&v)[CHUNK]) {
#pragma unroll
  for (int i = 0; i < CHUNK; ++i) v[i] = to_f32(r.e[i]);
}

// Two fp32 operations in one instruction (each lane rounds as its scalar form
// does).  The streaming kernels are bound by the issue of instructions next to
// memory: with scalar arithmetic GELU's backward issued in 82% of the cycles at
// 0.66 of a copy's rate, now 0.89.  A product that is only added to something
// is written as fma2: the assembler fuses mul2 and add2 in some kernels and not
// in others, and the bits are to be the same in all.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ F2 get2(const float* v) { return f2(v[0], v[1]); }
__device__ __forceinline__ void put2(float* v, F2 x) { asm("mov.b64 {%0, %1}, %2;" : "=f"(v[0]), "=f"(v[1]) : "l"(x.v)); }
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// The step byte of the group that this lane's 8 values belong to.
__device__ __forceinline__ uint32_t chunk_step(const float (&v)[CHUNK]) {
  float top = max_nan(fabsf(v[0]), fabsf(v[1]));
#pragma unroll
  for (int i = 2; i < CHUNK; i += 2) top = max_nan(top, fabsf(v[i]), fabsf(v[i + 1]));
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
  for (int i = 0; i < CHUNK; i += 2) {
    float x[2];
    put2(x, fma2(get2(v + i), f2(inverse), f2(12582912.0f)));
    w[i] = __float_as_uint(x[0]), w[i + 1] = __float_as_uint(x[1]);
  }
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
  const F2 scale = f2(act_scale(b)), bias = f2(-8388736.0f);
  const uint32_t x = c.x ^ 0x80808080u, y = c.y ^ 0x80808080u;
#pragma unroll
  for (int i = 0; i < CHUNK; i += 2) {
    const uint32_t w = i < 4 ? x : y;
    const F2 raw = f2(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440 + (i & 3))),
                      __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7441 + (i & 3))));
    put2(v + i, mul2(add2(raw, bias), scale));
  }
}

__device__ __forceinline__ uint2 load_codes(const int8_t* p) {
  uint2 c;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(c.x), "=r"(c.y) : "l"(p) : "memory");
  return c;
}

// ---------------------------------------------------------------- rings
// Loads in flight without registers for them: asynchronous copies of the rows
// ahead into slots of shared memory.  Each copy_group() closes what was copied
// since the last; wait_groups<N>() leaves the newest N groups in flight.
__device__ __forceinline__ void copy_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_groups() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t to, const void* from, int bytes) {  // zeros after `bytes`
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint4 shared16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

// OUT words from byte `off` (0 to 15) on of OUT + 4 words.
template <int OUT>
__device__ __forceinline__ void shift_words(uint32_t (&w)[OUT + 4], int off) {
  if (off & 8) {
#pragma unroll
    for (int i = 0; i < OUT + 2; ++i) w[i] = w[i + 2];
  }
  if (off & 4) {
#pragma unroll
    for (int i = 0; i < OUT + 1; ++i) w[i] = w[i + 1];
  }
  if (off & 3) {
#pragma unroll
    for (int i = 0; i < OUT; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 8 * (off & 3));
  }
}

// A matrix's rows as the streaming kernels read them, a thread's chunk of
// each row to come in a slot of its own.
//  SPAN = false (16-bit types, rows on 16-byte boundaries): each thread copies
//    and reads its own 16 bytes, no barrier is needed.
//  SPAN = true (any rows): a warp's 32 chunks of a row are one span of 256
//    elements; its 16-byte granules are copied as they lie in memory, whole
//    lines at a time, and a lane shifts its elements out of the granules
//    around them.  Every granule read holds an element of the span (only
//    bytes before the first may be a neighbour's, and are not used).
template <typename T, bool SPAN>
struct Rows {
  static constexpr int WORDS = SPAN ? 16 * (int)sizeof(T) + 1 : 1;  // granules of a warp's span, or of a lane
  static constexpr size_t bytes(int slots, int threads) {
    return SPAN ? (size_t)slots * (threads / 32) * WORDS * 16 : (size_t)slots * threads * 16;
  }
  uint32_t at, slot_bytes;
  const T* next;     // the next row's chunk or span
  int64_t step;      // elements from row to row
  int len;           // elements of the chunk or span inside the row
  uint32_t off, doff;  // SPAN: the current row's misalignment in bytes, its change from row to row
  // c8: this thread's chunk; n: its elements inside the row
  __device__ __forceinline__ Rows(void* shared, int threads, const T* row, int64_t stride, int c8, int n, int cols) {
    const int lane = threadIdx.x & 31;
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(shared);
    step = stride;
    if (SPAN) {
      at = base + (threadIdx.x >> 5) * (WORDS * 16u);
      slot_bytes = (uint32_t)(threads / 32) * (WORDS * 16u);
      next = row + (int64_t)(c8 - lane) * CHUNK;
      len = (int)min(max((int64_t)cols - (int64_t)(c8 - lane) * CHUNK, (int64_t)0), (int64_t)(32 * CHUNK));
      off = (uint32_t)((uintptr_t)next & 15u), doff = (uint32_t)((uint64_t)stride * sizeof(T) & 15u);
    } else {
      at = base + threadIdx.x * 16u, slot_bytes = (uint32_t)threads * 16u;
      next = row + (int64_t)c8 * CHUNK, len = n;
    }
  }
  // Starts the next row's copy (nothing for a row that is not there).
  __device__ __forceinline__ void copy(int slot, bool in) {
    if (in && len > 0) {
      const uint32_t to = at + (uint32_t)slot * slot_bytes;
      if (SPAN) {
        const int lane = threadIdx.x & 31, skip = (int)((uintptr_t)next & 15u), total = skip + len * (int)sizeof(T);
        const char* from = reinterpret_cast<const char*>(next) - skip;
#pragma unroll
        for (int g = 0; g < WORDS; g += 32) {
          const int i = g + lane, b = min(total - 16 * i, 16);
          if (i < WORDS && b > 0) copy16(to + 16u * i, from + 16 * i, b);
        }
      } else {
        copy16(to, next, len * (int)sizeof(T));
      }
    }
    next += step;
  }
  // All 8 elements of a chunk inside a row that is there (SPAN = false).
  __device__ __forceinline__ void copy_whole(int slot) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at + (uint32_t)slot * slot_bytes), "l"(next) : "memory");
    next += step;
  }
  // Before the first take of a row, after the wait: the other lanes' copies.
  __device__ __forceinline__ void landed() const {
    if (SPAN) __syncwarp();
  }
  // The current row's chunk as fp32; zeros from element n on.
  __device__ __forceinline__ void take(int slot, int n, float (&v)[CHUNK]) const {
    const uint32_t from = at + (uint32_t)slot * slot_bytes;
    constexpr int W = CHUNK * (int)sizeof(T) / 4;
    uint32_t w[W + 4];
    if (SPAN) {
#pragma unroll
      for (int i = 0; i <= W / 4; ++i) {
        const uint4 x = shared16(from + ((threadIdx.x & 31) * (W / 4) + i) * 16u);
        w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
      }
      shift_words<W>(w, (int)off);
    } else {
      const uint4 x = shared16(from);
      w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    }
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < W; ++i) reinterpret_cast<uint32_t*>(&r)[i] = w[i];
    unpack(r, v);
    if (n < CHUNK) {
#pragma unroll
      for (int e = 0; e < CHUNK; ++e)
        if (e >= n) v[e] = 0.0f;
    }
  }
  // After the last take of a row: on to the next, whose slot's predecessor may
  // be copied over.
  __device__ __forceinline__ void done() {
    if (SPAN) off = (off + doff) & 15u, __syncwarp();
  }
};

// A matrix's rows as they are written.  SPAN: through `stage` (the warp's own),
// shifted to whole granules; the ends element by element.
template <typename T, bool SPAN>
struct RowsOut {
  static constexpr int STAGE = 16 * (int)sizeof(T) + 2;  // 16-byte words of a warp's stage
  T* next;
  int64_t step;
  int len;
  __device__ __forceinline__ RowsOut(T* row, int64_t stride, int c8, int cols) : step(stride) {
    const int lane = threadIdx.x & 31;
    next = row + (int64_t)(SPAN ? c8 - lane : c8) * CHUNK;
    len = SPAN ? (int)min(max((int64_t)cols - (int64_t)(c8 - lane) * CHUNK, (int64_t)0), (int64_t)(32 * CHUNK)) : 0;
  }
  // n elements of the chunk; in: the row is there.  All lanes of the warp.
  __device__ __forceinline__ void put(const float (&v)[CHUNK], int n, bool in, float4* stage) {
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < CHUNK; ++i) r.e[i] = from_f32<T>(v[i]);
    if (SPAN) {
      constexpr int W = CHUNK * (int)sizeof(T) / 16, E = 16 / (int)sizeof(T);  // granules per lane, elements per granule
      const int lane = threadIdx.x & 31;
      const uint32_t at = (uint32_t)__cvta_generic_to_shared(stage);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const uint4 x = reinterpret_cast<const uint4*>(&r)[i];
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at + (1 + lane * W + i) * 16u), "r"(x.x), "r"(x.y),
                     "r"(x.z), "r"(x.w)
                     : "memory");
      }
      __syncwarp();
      const int skip = (int)((uintptr_t)next & 15u), total = in && len > 0 ? skip + len * (int)sizeof(T) : 0;
      char* const to = reinterpret_cast<char*>(next) - skip;
#pragma unroll
      for (int i = 0; i < W; ++i) {  // whole granules
        const int g = lane + 32 * i;
        uint32_t w[8];
        const uint4 a = shared16(at + (uint32_t)(g + (skip ? 0 : 1)) * 16u), b = shared16(at + (uint32_t)(g + 1) * 16u);
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
        shift_words<4>(w, (16 - skip) & 15);
        if (16 * g >= skip && 16 * g + 16 <= total) *reinterpret_cast<uint4*>(to + 16 * g) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      // the first granule's elements and the last one's where they are not
      // whole, a lane for each
      if (skip != 0 || (total & 15) != 0) {
        const int last = total >> 4, g = lane < E ? 0 : last;
        const int byte = 16 * g + (lane & (E - 1)) * (int)sizeof(T);
        const bool whole = 16 * g >= skip && 16 * g + 16 <= total;
        if (lane < 2 * E && (lane < E || last > 0) && !whole && byte >= skip && byte < total) {
          const uint32_t from = at + 16u + (uint32_t)(byte - skip);
          if (sizeof(T) == 4) {
            uint32_t x;
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(from) : "memory");
            *reinterpret_cast<uint32_t*>(to + byte) = x;
          } else {
            uint16_t x;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(from) : "memory");
            *reinterpret_cast<uint16_t*>(to + byte) = x;
          }
        }
      }
    } else if (in) {
      if (n == CHUNK) {
        *reinterpret_cast<uint4*>(next) = *reinterpret_cast<const uint4*>(&r);
      } else {
#pragma unroll
        for (int i = 0; i < CHUNK; ++i)
          if (i < n) next[i] = r.e[i];
      }
    }
    next += step;
  }
};

// A thread's 8 codes of the rows ahead, in slots of its own.
struct CodeRing {
  uint32_t at, stride;
  __device__ __forceinline__ CodeRing(void* shared, int threads)
      : at((uint32_t)__cvta_generic_to_shared(shared) + threadIdx.x * 8u), stride((uint32_t)threads * 8u) {}
  static constexpr size_t bytes(int slots, int threads) { return (size_t)slots * threads * 8; }
  __device__ __forceinline__ void copy(int slot, const int8_t* p) const {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(at + (uint32_t)slot * stride), "l"(p) : "memory");
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

// The GPU that launches go to, -1 without one.
static int current_device() {
  int device = -1;
  if (cudaGetDevice(&device) != cudaSuccess) (void)cudaGetLastError(), device = -1;
  return device;
}

// The CTAs of 256 threads that an SM holds of a kernel; 1 where that cannot be had.
template <auto KERN>
static int resident() {
  static PerDevice ctas;
  const int n = ctas.get(current_device(), [] {
    int held = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&held, KERN, 256, 0) == cudaSuccess) return held;
    (void)cudaGetLastError();
    return 0;
  });
  return n > 0 ? n : 1;
}

// Grants a kernel `bytes` of dynamic shared memory.
template <typename K>
static bool grant_shared(K kern, int bytes) {
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess) return true;
  (void)cudaGetLastError();
  return false;
}

// The widest tile (256 chunks to 4, or to 32 where a warp takes a span of one
// row) that leaves at most a sixteenth of its lanes past the rows' end.
// Large matrices: about ACT_CTAS CTAs (with six for every SM the gates' gradient of
// 8192 x 14336 takes 154 us instead of 145).  Small ones, whose CTAs would have
// a few rows each: one wave of the CTAs that fit (2048 x 4096: 11.4 us instead
// of 12.2; 128 x 14336: 3.8 instead of 4.7; 777 x 4097: 8.5 instead of 9.8).
constexpr int64_t ACT_SMS = 152, ACT_CTAS = ACT_SMS * 8, ACT_FEW = 8;
inline Tiling make_tiling(int64_t rows, int64_t cols, bool span, int ctas, dim3* grid) {
  Tiling t;
  t.rows = rows, t.cols = (int32_t)cols, t.c8s = (int32_t)(act_ldc(cols) / CHUNK);
  t.wide = 8;
  while (t.wide > (span ? 5 : 2) && ((((int64_t)t.c8s + (1 << t.wide) - 1) >> t.wide) << t.wide) > t.c8s + t.c8s / 16) --t.wide;
  const int64_t across = ((int64_t)t.c8s + (1 << t.wide) - 1) >> t.wide, at_once = 256 >> t.wide;
  const int64_t most = (rows + at_once - 1) / at_once;
  int64_t slabs = most * across < ACT_FEW * ACT_CTAS ? ACT_SMS * ctas / across : (ACT_CTAS + across - 1) / across;
  if (slabs < 1) slabs = 1;
  if (slabs > most) slabs = most;
  if (slabs > 65535) slabs = 65535;
  t.slab = ((rows + slabs - 1) / slabs + at_once - 1) / at_once * at_once;
  *grid = dim3((unsigned)across, (unsigned)((rows + t.slab - 1) / t.slab));
  return t;
}
}  // namespace gc

// Runs a statement with T the element type of a valid dtype.
#define GC_BY_DTYPE(dtype, T, ...)                                \
  do {                                                            \
    if ((dtype) == GC_F32) { using T = float; __VA_ARGS__; }      \
    else if ((dtype) == GC_BF16) { using T = __nv_bfloat16; __VA_ARGS__; } \
    else { using T = __half; __VA_ARGS__; }                       \
  } while (0)
