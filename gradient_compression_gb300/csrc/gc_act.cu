// Checkpoints of activations in 8 bits and the gated activation around them.
#include "gc_act.cuh"
#include "gc_host.h"

namespace gc {

constexpr int UNROLL = 4;  // chunks of a thread: their loads are issued before any is used

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) k_act_compress(const T* x, int64_t ld, int64_t cols, Walk w, int8_t* codes,
                                                      uint8_t* steps) {
  chain_wait();
  const int64_t groups = w.c8s / 4;
  Chunk at[UNROLL];
  Raw8<T> raw[UNROLL];
  at[0] = first_chunk(w, (int64_t)blockIdx.x * (256 * UNROLL) + threadIdx.x);
#pragma unroll
  for (int i = 0; i < UNROLL; ++i) {
    if (i) at[i] = at[i - 1], next_chunk(w, at[i]);
    raw[i] = load_chunk<T, VEC>(x + at[i].r * ld + (int64_t)at[i].c8 * CHUNK, chunk_len(w, at[i], cols));
  }
#pragma unroll
  for (int i = 0; i < UNROLL; ++i) {
    float v[CHUNK];
    unpack(raw[i], v);
    const uint32_t b = chunk_step(v);
    const uint2 c = chunk_codes(v, b);
    if (at[i].r < w.rows) store_codes(codes, steps, groups, at[i].r, at[i].c8, c, b);
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) k_act_decompress(const int8_t* codes, const uint8_t* steps, int64_t cols, Walk w,
                                                        T* out, int64_t ld) {
  __shared__ float4 stage[VEC ? 1 : 512];
  chain_wait();
  const int64_t groups = w.c8s / 4;
  Chunk at[UNROLL];
  uint2 c[UNROLL];
  uint32_t b[UNROLL];
  at[0] = first_chunk(w, (int64_t)blockIdx.x * (256 * UNROLL) + threadIdx.x);
#pragma unroll
  for (int i = 0; i < UNROLL; ++i) {
    if (i) at[i] = at[i - 1], next_chunk(w, at[i]);
    c[i] = make_uint2(0u, 0u), b[i] = 1u;
    if (at[i].r < w.rows) c[i] = load_codes(codes, groups, at[i].r, at[i].c8), b[i] = steps[at[i].r * groups + (at[i].c8 >> 2)];
  }
#pragma unroll
  for (int i = 0; i < UNROLL; ++i) {
    float v[CHUNK];
    chunk_values(c[i], b[i], v);
    store_chunk<T, VEC>(out + at[i].r * ld + (int64_t)at[i].c8 * CHUNK, chunk_len(w, at[i], cols), v,
                        reinterpret_cast<float*>(stage) + (threadIdx.x >> 5) * 256);
  }
}

// sigmoid(p(g)) and p'(g): the activation is g * sigmoid(p(g)), its
// derivative s + g s (1 - s) p'(g).  The tanh form of GELU is of this kind
// since (1 + tanh z) / 2 = sigmoid(2 z).  The exponential turns an error of
// u |p| in p into a relative error of the result, |p| up to 87: the rounding
// errors of g^2 and of the last product are carried along in `low` and
// applied as exp(-(p + low)) = exp(-p) (1 - low).
// Below -80, where 1 + exp(-p) is exp(-p) and soon overflows, the sigmoid is
// exp(p).
// PRECISE (fp32 results): correctly rounded division and CUDA's expf.  For
// 16-bit results the hardware's exponential and reciprocal, a few 2^-23 off
// (and |p| 2^-24 from the argument), are 2^-10 of the result's own rounding
// and a third of the instructions, which bound these kernels next to memory.
template <int KIND, bool PRECISE>
__device__ __forceinline__ float gate_sigmoid(float g, float* dp) {
  float p = g, low = 0.0f;
  *dp = 1.0f;
  if (KIND == GC_GATE_GELU_TANH) {
    constexpr float C = 1.5957691216057308f, CA = 0.0713548162726009f;  // 2 sqrt(2/pi), times 0.044715
    // beyond +-30 the sigmoid is 0 or 1 in fp32; the clamp keeps g^3 and p'
    // finite there, so that 0 * p' stays 0 (and lets a NaN through)
    const float t = fabsf(g) > 30.0f ? copysignf(30.0f, g) : g;
    const float t2 = __fmul_rn(t, t), w = __fmaf_rn(CA, t2, C);
    p = __fmul_rn(w, t);
    low = __fmaf_rn(CA * __fmaf_rn(t, t, -t2), t, __fmaf_rn(w, t, -p));
    *dp = __fmaf_rn(2.0f * CA, t2, w);
  }
  const bool far = p < -80.0f;
  const float z = far ? p : -p;
  float e;
  if (PRECISE) {
    e = expf(z);
  } else {
    asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(__fmul_rn(z, 1.4426950408889634f)));
  }
  if (KIND == GC_GATE_GELU_TANH) e = __fmaf_rn(e, far ? low : -low, e);
  const float one = __fadd_rn(1.0f, e);
  float s;
  if (PRECISE) {
    s = __fdiv_rn(1.0f, one);
  } else {
    asm("rcp.approx.f32 %0, %1;" : "=f"(s) : "f"(one));
  }
  return far ? e : s;
}

// The loads of one chunk are issued together; two chunks per thread leave 32
// warps per SM and put 128 bytes per thread in flight.
constexpr int GATED_UNROLL = 2;

template <typename T, int KIND, bool VEC>
__global__ void __launch_bounds__(256)
    k_gated(const T* gate, int64_t ldg, const T* up, int64_t ldu, int64_t cols, Walk w, T* out, int64_t ldo, int8_t* gcodes,
            uint8_t* gsteps, int8_t* ucodes, uint8_t* usteps) {
  __shared__ float4 stage[VEC ? 1 : 512];
  chain_wait();
  const int64_t groups = w.c8s / 4;
  Chunk at[GATED_UNROLL];
  Raw8<T> rg[GATED_UNROLL], ru[GATED_UNROLL];
  at[0] = first_chunk(w, (int64_t)blockIdx.x * (256 * GATED_UNROLL) + threadIdx.x);
#pragma unroll
  for (int i = 0; i < GATED_UNROLL; ++i) {
    if (i) at[i] = at[i - 1], next_chunk(w, at[i]);
    const int n = chunk_len(w, at[i], cols);
    const int64_t c = (int64_t)at[i].c8 * CHUNK;
    rg[i] = load_chunk<T, VEC>(gate + at[i].r * ldg + c, n);
    ru[i] = load_chunk<T, VEC>(up + at[i].r * ldu + c, n);
  }
#pragma unroll
  for (int i = 0; i < GATED_UNROLL; ++i) {
    float g[CHUNK], u[CHUNK], v[CHUNK];
    unpack(rg[i], g);
    unpack(ru[i], u);
    if (gcodes) {
      const uint32_t bg = chunk_step(g), bu = chunk_step(u);
      const uint2 cg = chunk_codes(g, bg), cu = chunk_codes(u, bu);
      if (at[i].r < w.rows) {
        store_codes(gcodes, gsteps, groups, at[i].r, at[i].c8, cg, bg);
        store_codes(ucodes, usteps, groups, at[i].r, at[i].c8, cu, bu);
      }
    }
#pragma unroll
    for (int e = 0; e < CHUNK; ++e) {
      float dp;
      v[e] = __fmul_rn(__fmul_rn(g[e], gate_sigmoid<KIND, sizeof(T) == 4>(g[e], &dp)), u[e]);
    }
    store_chunk<T, VEC>(out + at[i].r * ldo + (int64_t)at[i].c8 * CHUNK, chunk_len(w, at[i], cols), v,
                        reinterpret_cast<float*>(stage) + (threadIdx.x >> 5) * 256);
  }
}

template <typename T, int KIND, bool VEC>
__global__ void __launch_bounds__(256)
    k_gated_backward(const T* dout, int64_t lddo, const int8_t* gcodes, const uint8_t* gsteps, const int8_t* ucodes,
                     const uint8_t* usteps, int64_t cols, Walk w, T* dgate, int64_t lddg, T* dup, int64_t lddu,
                     int8_t* ocodes, uint8_t* osteps) {
  __shared__ float4 stage[VEC ? 1 : 512];
  float* const buf = reinterpret_cast<float*>(stage) + (threadIdx.x >> 5) * 256;
  chain_wait();
  const int64_t groups = w.c8s / 4;
  Chunk at[GATED_UNROLL];
  Raw8<T> rd[GATED_UNROLL];
  uint2 cg[GATED_UNROLL], cu[GATED_UNROLL];
  uint32_t bg[GATED_UNROLL], bu[GATED_UNROLL];
  at[0] = first_chunk(w, (int64_t)blockIdx.x * (256 * GATED_UNROLL) + threadIdx.x);
#pragma unroll
  for (int i = 0; i < GATED_UNROLL; ++i) {
    if (i) at[i] = at[i - 1], next_chunk(w, at[i]);
    rd[i] = load_chunk<T, VEC>(dout + at[i].r * lddo + (int64_t)at[i].c8 * CHUNK, chunk_len(w, at[i], cols));
    cg[i] = cu[i] = make_uint2(0u, 0u), bg[i] = bu[i] = 1u;
    if (at[i].r < w.rows) {
      const int64_t s = at[i].r * groups + (at[i].c8 >> 2);
      cg[i] = load_codes(gcodes, groups, at[i].r, at[i].c8), bg[i] = gsteps[s];
      cu[i] = load_codes(ucodes, groups, at[i].r, at[i].c8), bu[i] = usteps[s];
    }
  }
#pragma unroll
  for (int i = 0; i < GATED_UNROLL; ++i) {
    float g[CHUNK], u[CHUNK], d[CHUNK], a[CHUNK];
    chunk_values(cg[i], bg[i], g);
    chunk_values(cu[i], bu[i], u);
    unpack(rd[i], d);
#pragma unroll
    for (int e = 0; e < CHUNK; ++e) {
      float dp;
      const float s = gate_sigmoid<KIND, sizeof(T) == 4>(g[e], &dp), act = __fmul_rn(g[e], s);
      const float slope = __fmaf_rn(__fmul_rn(act, __fsub_rn(1.0f, s)), dp, s);
      g[e] = __fmul_rn(__fmul_rn(d[e], u[e]), slope);  // dgate
      a[e] = __fmul_rn(act, u[e]);
      u[e] = __fmul_rn(d[e], act);  // dup
    }
    const int n = chunk_len(w, at[i], cols);
    const int64_t c = (int64_t)at[i].c8 * CHUNK;
    store_chunk<T, VEC>(dgate + at[i].r * lddg + c, n, g, buf);
    store_chunk<T, VEC>(dup + at[i].r * lddu + c, n, u, buf);
    if (ocodes) {
      const uint32_t b = chunk_step(a);
      const uint2 q = chunk_codes(a, b);
      if (at[i].r < w.rows) store_codes(ocodes, osteps, groups, at[i].r, at[i].c8, q, b);
    }
  }
}

static Walk make_walk(int64_t rows, int64_t cols) {
  Walk w;
  w.rows = rows, w.c8s = (int32_t)(act_ldc(cols) / CHUNK);
  w.dr = 256 / w.c8s, w.dc = 256 % w.c8s;
  return w;
}
// CTAs for `unroll` chunks per thread; 0 if a grid cannot hold them.
static unsigned walk_grid(const Walk& w, int unroll) {
  const int64_t blocks = (w.rows * w.c8s + 256 * unroll - 1) / (256 * unroll);
  return blocks <= INT64_C(2147483647) ? (unsigned)blocks : 0u;
}

}  // namespace gc

using namespace gc;

extern "C" gc_status gc_act_compress(const void* x, int64_t ld, int32_t dtype, int64_t rows, int64_t cols,
                                     int8_t* codes, uint8_t* steps, void* stream) {
  NvtxRange nvtx_range("gc_act_compress");
  gc_status st = validate_matrix(rows, cols, dtype);
  if (st != GC_OK) return st;
  if (rows == 0) return GC_OK;
  if ((st = check_matrix(x, ld, cols, dtype)) != GC_OK || (st = check_codes(codes, steps)) != GC_OK) return st;
  const Walk w = make_walk(rows, cols);
  const unsigned grid = walk_grid(w, UNROLL);
  if (!grid) return GC_ERR_LAYOUT;
  const bool vec = chunk_aligned(x, ld, dtype);
  GC_BY_DTYPE(dtype, T, launch_chained(vec ? k_act_compress<T, true> : k_act_compress<T, false>, grid, 256, 0,
                                       static_cast<cudaStream_t>(stream), static_cast<const T*>(x), ld, cols, w, codes,
                                       steps));
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}

extern "C" gc_status gc_act_decompress(const int8_t* codes, const uint8_t* steps, int64_t rows, int64_t cols,
                                       void* out, int64_t ldo, int32_t dtype, void* stream) {
  NvtxRange nvtx_range("gc_act_decompress");
  gc_status st = validate_matrix(rows, cols, dtype);
  if (st != GC_OK) return st;
  if (rows == 0) return GC_OK;
  if ((st = check_codes(codes, steps)) != GC_OK || (st = check_matrix(out, ldo, cols, dtype)) != GC_OK) return st;
  const Walk w = make_walk(rows, cols);
  const unsigned grid = walk_grid(w, UNROLL);
  if (!grid) return GC_ERR_LAYOUT;
  const bool vec = chunk_aligned(out, ldo, dtype);
  GC_BY_DTYPE(dtype, T, launch_chained(vec ? k_act_decompress<T, true> : k_act_decompress<T, false>, grid, 256, 0,
                                       static_cast<cudaStream_t>(stream), codes, steps, cols, w, static_cast<T*>(out),
                                       ldo));
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}

extern "C" gc_status gc_gated_act(int32_t kind, const void* gate, int64_t ldg, const void* up, int64_t ldu,
                                  int32_t dtype, int64_t rows, int64_t cols, void* out, int64_t ldo,
                                  int8_t* gate_codes, uint8_t* gate_steps, int8_t* up_codes, uint8_t* up_steps,
                                  void* stream) {
  NvtxRange nvtx_range("gc_gated_act");
  gc_status st = validate_matrix(rows, cols, dtype);
  if (st != GC_OK) return st;
  if (kind != GC_GATE_SILU && kind != GC_GATE_GELU_TANH) return GC_ERR_INVALID_ARG;
  if (rows == 0) return GC_OK;
  if ((st = check_matrix(gate, ldg, cols, dtype)) != GC_OK || (st = check_matrix(up, ldu, cols, dtype)) != GC_OK ||
      (st = check_matrix(out, ldo, cols, dtype)) != GC_OK)
    return st;
  if (gate_codes || gate_steps || up_codes || up_steps)
    if ((st = check_codes(gate_codes, gate_steps)) != GC_OK || (st = check_codes(up_codes, up_steps)) != GC_OK)
      return st;
  const Walk w = make_walk(rows, cols);
  const unsigned grid = walk_grid(w, GATED_UNROLL);
  if (!grid) return GC_ERR_LAYOUT;
  const bool vec = chunk_aligned(gate, ldg, dtype) && chunk_aligned(up, ldu, dtype) && chunk_aligned(out, ldo, dtype);
  GC_BY_DTYPE(dtype, T, {
    auto kern = kind == GC_GATE_SILU ? (vec ? k_gated<T, GC_GATE_SILU, true> : k_gated<T, GC_GATE_SILU, false>)
                                     : (vec ? k_gated<T, GC_GATE_GELU_TANH, true> : k_gated<T, GC_GATE_GELU_TANH, false>);
    launch_chained(kern, grid, 256, 0, static_cast<cudaStream_t>(stream), static_cast<const T*>(gate), ldg,
                   static_cast<const T*>(up), ldu, cols, w, static_cast<T*>(out), ldo, gate_codes, gate_steps, up_codes,
                   up_steps);
  });
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}

extern "C" gc_status gc_gated_act_backward(int32_t kind, const void* dout, int64_t lddo, int32_t dtype,
                                           const int8_t* gate_codes, const uint8_t* gate_steps,
                                           const int8_t* up_codes, const uint8_t* up_steps, int64_t rows,
                                           int64_t cols, void* dgate, int64_t lddg, void* dup, int64_t lddu,
                                           int8_t* out_codes, uint8_t* out_steps, void* stream) {
  NvtxRange nvtx_range("gc_gated_act_backward");
  gc_status st = validate_matrix(rows, cols, dtype);
  if (st != GC_OK) return st;
  if (kind != GC_GATE_SILU && kind != GC_GATE_GELU_TANH) return GC_ERR_INVALID_ARG;
  if (rows == 0) return GC_OK;
  if ((st = check_matrix(dout, lddo, cols, dtype)) != GC_OK || (st = check_matrix(dgate, lddg, cols, dtype)) != GC_OK ||
      (st = check_matrix(dup, lddu, cols, dtype)) != GC_OK || (st = check_codes(gate_codes, gate_steps)) != GC_OK ||
      (st = check_codes(up_codes, up_steps)) != GC_OK)
    return st;
  if (out_codes || out_steps)
    if ((st = check_codes(out_codes, out_steps)) != GC_OK) return st;
  const Walk w = make_walk(rows, cols);
  const unsigned grid = walk_grid(w, GATED_UNROLL);
  if (!grid) return GC_ERR_LAYOUT;
  const bool vec = chunk_aligned(dout, lddo, dtype) && chunk_aligned(dgate, lddg, dtype) && chunk_aligned(dup, lddu, dtype);
  GC_BY_DTYPE(dtype, T, {
    auto kern = kind == GC_GATE_SILU
                    ? (vec ? k_gated_backward<T, GC_GATE_SILU, true> : k_gated_backward<T, GC_GATE_SILU, false>)
                    : (vec ? k_gated_backward<T, GC_GATE_GELU_TANH, true> : k_gated_backward<T, GC_GATE_GELU_TANH, false>);
    launch_chained(kern, grid, 256, 0, static_cast<cudaStream_t>(stream), static_cast<const T*>(dout), lddo, gate_codes,
                   gate_steps, up_codes, up_steps, cols, w, static_cast<T*>(dgate), lddg, static_cast<T*>(dup), lddu,
                   out_codes, out_steps);
  });
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}
