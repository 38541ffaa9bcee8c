// Checkpoints of activations in 8 bits and the gated activation around them.
#include "gc_act.cuh"
#include "gc_host.h"

namespace gc {

// Every kernel here is one pass over its matrices, bound by memory; the times
// below are for 32768 x 4096 (checkpoints) and 8192 x 14336 (gates), and the
// share of the rate of a plain copy (6.67 TB/s) that their bytes reach.
//
// The loops keep AHEAD - 1 rows' loads in flight while they work on one, in
// rings of shared memory.  Four CTAs per SM with 112 bytes per thread in
// flight are 114 KB; the two dies' memories are about 1.5 us away under load,
// and 6.7 TB/s is 44 KB per SM and us.  Rows that are not on 16-byte
// boundaries cost the shifting of their spans on top, and are bound by the
// issue of instructions.

// The step from the group's largest magnitude, over four lanes, then the
// codes.  bf16 64 us (0.96), fp32 108 us (0.94), bf16 rows of 4095 86 us (0.71).
template <typename T, bool SPAN>
__global__ void __launch_bounds__(256, 4) k_act_compress(const T* x, int64_t ld, Tiling t, int8_t* codes, uint8_t* steps) {
  constexpr int AHEAD = 8 / (int)(sizeof(T) / 2);
  __shared__ float4 shared[Rows<T, SPAN>::bytes(AHEAD, 256) / 16];
  chain_wait();
  const Place p = place(t);
  const int64_t ldc = (int64_t)t.c8s * CHUNK, groups = t.c8s / 4;
  Rows<T, SPAN> in(shared, 256, x + p.r * ld, p.step * ld, p.c8, p.n, t.cols);
  int8_t* pc = codes + p.r * ldc + (int64_t)p.c8 * CHUNK;
  uint8_t* ps = steps + p.r * groups + (p.c8 >> 2);
  const int64_t dc = p.step * ldc, ds = p.step * groups;
  int64_t r = p.r, next = p.r;
  auto copy = [&](int slot) {
    in.copy(slot, next < p.end);
    copy_group();
    next += p.step;
  };
#pragma unroll
  for (int i = 0; i < AHEAD - 1; ++i) copy(i);
  int slot = 0;
  for (int64_t lead = (int64_t)blockIdx.y * t.slab; lead < p.end; lead += p.step, r += p.step, pc += dc, ps += ds) {
    float v[CHUNK];
    wait_groups<AHEAD - 2>();
    in.landed();
    in.take(slot, r < p.end ? p.n : 0, v);
    in.done();
    copy((slot + AHEAD - 1) % AHEAD);
    slot = (slot + 1) % AHEAD;
    const uint32_t b = chunk_step(v);
    const uint2 c = chunk_codes(v, b);
    if (p.in && r < p.end) {
      *reinterpret_cast<uint2*>(pc) = c;
      if ((p.c8 & 3) == 0) *ps = (uint8_t)b;
    }
  }
}

// Codes and steps take three registers a row, so the rows ahead stay there:
// eight of a 16-bit type, four of fp32 (four and eight: 66 and 112 us, and 92
// for rows of 4095).  bf16 64 us (0.96), fp32 107 us (0.95), bf16 rows of 4095
// 71 us (0.86).
template <typename T, bool SPAN>
__global__ void __launch_bounds__(256, SPAN && sizeof(T) == 2 ? 2 : 3)
    k_act_decompress(const int8_t* codes, const uint8_t* steps, Tiling t, T* out, int64_t ld) {
  constexpr int ROWS = 16 / (int)sizeof(T);
  __shared__ float4 stage[SPAN ? 8 * RowsOut<T, SPAN>::STAGE : 1];
  chain_wait();
  const Place p = place(t);
  const int64_t ldc = (int64_t)t.c8s * CHUNK, groups = t.c8s / 4;
  const int8_t* pc = codes + p.r * ldc + (int64_t)p.c8 * CHUNK;
  const uint8_t* ps = steps + p.r * groups + (p.c8 >> 2);
  RowsOut<T, SPAN> to(out + p.r * ld, p.step * ld, p.c8, t.cols);
  float4* const own = stage + (SPAN ? (threadIdx.x >> 5) * RowsOut<T, SPAN>::STAGE : 0);
  const int64_t dc = p.step * ldc, ds = p.step * groups;
  uint2 c[ROWS];
  uint32_t b[ROWS];
  auto fetch = [&](int64_t r) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i, r += p.step, pc += dc, ps += ds) {
      c[i] = make_uint2(0u, 0u), b[i] = 1u;
      if (p.in && r < p.end) c[i] = load_codes(pc), b[i] = __ldg(ps);
    }
  };
  int64_t r = p.r, lead = (int64_t)blockIdx.y * t.slab;
  fetch(r);
  for (; lead < p.end; lead += ROWS * p.step) {
    uint2 cn[ROWS];
    uint32_t bn[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) cn[i] = c[i], bn[i] = b[i];
    if (lead + ROWS * p.step < p.end) fetch(r + ROWS * p.step);
#pragma unroll
    for (int i = 0; i < ROWS; ++i, r += p.step) {
      if (lead + i * p.step >= p.end) break;
      float v[CHUNK];
      chunk_values(cn[i], bn[i], v);
      to.put(v, p.n, r < p.end, own);
    }
  }
}

// sigmoid(p(g)) and p'(g): the activation is g * sigmoid(p(g)), its
// derivative s + g s (1 - s) p'(g).  The tanh form of GELU is of this kind
// since (1 + tanh z) / 2 = sigmoid(2 z).  The exponential turns an error of
// u |p| in p into a relative error of the result, |p| up to 87: the rounding
// errors of g^2 and of the last product are carried along in `low` and
// applied as exp(-(p + low)) = exp(-p) (1 - low).
constexpr float GELU_C = 1.5957691216057308f, GELU_CA = 0.0713548162726009f;  // 2 sqrt(2/pi), times 0.044715
// Beyond +-30 GELU's sigmoid is 0 or 1 in fp32; the clamp keeps g^3 and p'
// finite there, so that 0 * p' stays 0 (and lets a NaN through).
constexpr float GELU_FAR = 30.0f;

// For fp32 results: correctly rounded division and CUDA's expf.  Below -80,
// where 1 + exp(-p) is exp(-p) and soon overflows, the sigmoid is exp(p).
template <int KIND>
__device__ __forceinline__ float gate_sigmoid(float g, float* dp) {
  float p = g, low = 0.0f;
  *dp = 1.0f;
  if (KIND == GC_GATE_GELU_TANH) {
    const float t = fabsf(g) > GELU_FAR ? copysignf(GELU_FAR, g) : g;
    const float t2 = __fmul_rn(t, t), w = __fmaf_rn(GELU_CA, t2, GELU_C);
    p = __fmul_rn(w, t);
    low = __fmaf_rn(GELU_CA * __fmaf_rn(t, t, -t2), t, __fmaf_rn(w, t, -p));
    *dp = __fmaf_rn(2.0f * GELU_CA, t2, w);
  }
  const bool far = p < -80.0f;
  float e = expf(far ? p : -p);
  if (KIND == GC_GATE_GELU_TANH) e = __fmaf_rn(e, far ? low : -low, e);
  return far ? e : __fdiv_rn(1.0f, __fadd_rn(1.0f, e));
}

__device__ __forceinline__ float ex2_ftz(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_ftz(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// For 16-bit results, two at a time: the hardware's exponential and
// reciprocal, a few 2^-23 off (and |p| 2^-23 from SiLU's argument), are at most 2^-8
// of the result's own rounding and a third of the instructions.
// SiLU: with h = 2^(-g log2(e) / 2) the sigmoid is 1 / (1 + h^2), taken as
// 2^-64 / (2^-64 + (2^-32 h)^2): neither the sum overflows nor the reciprocal
// vanishes before the sigmoid is below all of fp32 (1 + e^-g itself is past
// the reciprocal's 2^126 from g = -87.3 on, where the product is still 1e-36).
// GELU: with h = 2^(-z/2), z = |p| log2(e), and f = h^2 the sigmoid is
// 1 / (1 + f) on the right and f / (1 + f) on the left, where nothing
// overflows and f reaches below 2^-126 (the exponential itself does not).
template <int KIND>
__device__ __forceinline__ F2 gate_sigmoid2(const float* g, F2* dp) {
  constexpr float LOG2E = 1.4426950408889634f;
  float x[2], r[2];
  if (KIND == GC_GATE_SILU) {
    constexpr float SMALL = 5.421010862427522e-20f, ROOT = 2.3283064365386963e-10f;  // 2^-64, 2^-32
    put2(x, mul2(get2(g), f2(-0.5f * LOG2E)));
    const F2 h = mul2(f2(ex2_ftz(x[0]), ex2_ftz(x[1])), f2(ROOT));
    put2(r, fma2(h, h, f2(SMALL)));
    *dp = f2(1.0f);
    return mul2(f2(rcp_ftz(r[0]), rcp_ftz(r[1])), f2(SMALL));
  }
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(x[0]) : "f"(fabsf(g[0])), "f"(GELU_FAR));
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(x[1]) : "f"(fabsf(g[1])), "f"(GELU_FAR));
  const F2 t = get2(x), minus_t = mul2(t, f2(-1.0f)), minus_t2 = mul2(t, minus_t);
  const F2 w = fma2(minus_t2, f2(-0.5f * LOG2E * GELU_CA), f2(0.5f * LOG2E * GELU_C)), minus_z = mul2(w, minus_t);
  const F2 low = fma2(mul2(t, f2(0.5f * LOG2E * GELU_CA)), fma2(t, t, minus_t2), fma2(w, t, minus_z));
  *dp = fma2(minus_t2, f2(-3.0f * GELU_CA), f2(GELU_C));
  put2(x, minus_z);
  F2 h = f2(ex2_ftz(x[0]), ex2_ftz(x[1]));
  h = fma2(h, mul2(low, f2(-0.693147180559945f)), h);
  const F2 f = mul2(h, h);
  put2(x, fma2(h, h, f2(1.0f)));
  const F2 right = f2(rcp_ftz(x[0]), rcp_ftz(x[1]));
  put2(r, right), put2(x, mul2(f, right));
  return f2(g[0] < 0.0f ? x[0] : r[0], g[1] < 0.0f ? x[1] : r[1]);
}

// Registers for the packed arithmetic matter more than a fourth CTA per SM
// (two for spans).  With both checkpoints: bf16 148 us for either kind (0.96;
// GELU with scalar arithmetic 172), fp32 276 us (0.90) and 320 with GELU, bf16
// rows of 14335 181 us (0.78) and 225.
template <typename T, int KIND, bool SPAN>
__global__ void __launch_bounds__(256, SPAN && sizeof(T) == 2 ? 2 : 3)
    k_gated(const T* gate, int64_t ldg, const T* up, int64_t ldu, Tiling t, T* out, int64_t ldo, int8_t* gcodes,
            uint8_t* gsteps, int8_t* ucodes, uint8_t* usteps) {
  constexpr int AHEAD = 4 / (int)(sizeof(T) / 2);
  constexpr size_t RING = Rows<T, SPAN>::bytes(AHEAD, 256) / 16;
  __shared__ float4 shared[2 * RING + (SPAN ? 8 * RowsOut<T, SPAN>::STAGE : 0)];
  chain_wait();
  const Place p = place(t);
  const int64_t ldc = (int64_t)t.c8s * CHUNK, groups = t.c8s / 4;
  Rows<T, SPAN> gin(shared, 256, gate + p.r * ldg, p.step * ldg, p.c8, p.n, t.cols);
  Rows<T, SPAN> uin(shared + RING, 256, up + p.r * ldu, p.step * ldu, p.c8, p.n, t.cols);
  RowsOut<T, SPAN> to(out + p.r * ldo, p.step * ldo, p.c8, t.cols);
  float4* const own = shared + 2 * RING + (SPAN ? (threadIdx.x >> 5) * RowsOut<T, SPAN>::STAGE : 0);
  int64_t ac = p.r * ldc + (int64_t)p.c8 * CHUNK, as = p.r * groups + (p.c8 >> 2);  // offsets of codes and steps
  const int64_t dc = p.step * ldc, ds = p.step * groups;
  int64_t r = p.r, next = p.r;
  auto copy = [&](int slot) {
    gin.copy(slot, next < p.end), uin.copy(slot, next < p.end);
    copy_group();
    next += p.step;
  };
#pragma unroll
  for (int i = 0; i < AHEAD - 1; ++i) copy(i);
  int slot = 0;
  for (int64_t lead = (int64_t)blockIdx.y * t.slab; lead < p.end; lead += p.step, r += p.step) {
    const int n = r < p.end ? p.n : 0;
    float g[CHUNK], u[CHUNK];
    wait_groups<AHEAD - 2>();
    gin.landed();
    gin.take(slot, n, g), uin.take(slot, n, u);
    gin.done(), uin.done();
    copy((slot + AHEAD - 1) % AHEAD);
    slot = (slot + 1) % AHEAD;
    if (gcodes) {
      const uint32_t bg = chunk_step(g), bu = chunk_step(u);
      const uint2 cg = chunk_codes(g, bg), cu = chunk_codes(u, bu);
      if (p.in && r < p.end) {
        *reinterpret_cast<uint2*>(gcodes + ac) = cg;
        *reinterpret_cast<uint2*>(ucodes + ac) = cu;
        if ((p.c8 & 3) == 0) gsteps[as] = (uint8_t)bg, usteps[as] = (uint8_t)bu;
      }
      ac += dc, as += ds;
    }
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < CHUNK; ++e) {
        float dp;
        g[e] = __fmul_rn(__fmul_rn(g[e], gate_sigmoid<KIND>(g[e], &dp)), u[e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < CHUNK; e += 2) {
        F2 dp;
        put2(g + e, mul2(mul2(get2(g + e), gate_sigmoid2<KIND>(g + e, &dp)), get2(u + e)));
      }
    }
    to.put(g, n, r < p.end, own);
  }
}

// dout and both codes come through rings, the step bytes through registers.
// Three CTAs per SM (two for spans): the fourth would leave 64 registers and
// spill (152 and 184 us).  bf16 145 us (0.98), GELU 160 us (0.89; 214 with
// scalar arithmetic); with the activation's checkpoint 168 and 182 us; fp32
// 308 us (0.80); bf16 rows of 14335 193 us (0.74).
template <typename T, int KIND, bool SPAN>
__global__ void __launch_bounds__(256, SPAN ? 2 : 3)
    k_gated_backward(const T* dout, int64_t lddo, const int8_t* gcodes, const uint8_t* gsteps, const int8_t* ucodes,
                     const uint8_t* usteps, Tiling t, T* dgate, int64_t lddg, T* dup, int64_t lddu, int8_t* ocodes,
                     uint8_t* osteps) {
  constexpr int AHEAD = sizeof(T) == 2 ? 4 : 2;
  constexpr size_t RING = Rows<T, SPAN>::bytes(AHEAD, 256) / 16;
  __shared__ float4 shared[RING + (SPAN ? 8 * RowsOut<T, SPAN>::STAGE : 0)];
  __shared__ uint2 code_slots[2 * AHEAD * 256];
  chain_wait();
  const Place p = place(t);
  const int64_t ldc = (int64_t)t.c8s * CHUNK, groups = t.c8s / 4;
  Rows<T, SPAN> din(shared, 256, dout + p.r * lddo, p.step * lddo, p.c8, p.n, t.cols);
  RowsOut<T, SPAN> gto(dgate + p.r * lddg, p.step * lddg, p.c8, t.cols), uto(dup + p.r * lddu, p.step * lddu, p.c8, t.cols);
  float4* const own = shared + RING + (SPAN ? (threadIdx.x >> 5) * RowsOut<T, SPAN>::STAGE : 0);
  const CodeRing code(code_slots, 256);
  int64_t ac = p.r * ldc + (int64_t)p.c8 * CHUNK, as = p.r * groups + (p.c8 >> 2), r = p.r;
  const int64_t dc = p.step * ldc, ds = p.step * groups;
  int64_t next = p.r, nc = ac;
  auto copy = [&](int slot) {
    din.copy(slot, next < p.end);
    if (next < p.end && p.in) code.copy(2 * slot, gcodes + nc), code.copy(2 * slot + 1, ucodes + nc);
    copy_group();
    next += p.step, nc += dc;
  };
  // step bytes of AHEAD rows, loaded as many rows earlier
  uint32_t bg[AHEAD], bu[AHEAD];
  auto fetch_steps = [&](int64_t row, int64_t at) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i, row += p.step, at += ds) {
      bg[i] = bu[i] = 1u;
      if (p.in && row < p.end) bg[i] = __ldg(gsteps + at), bu[i] = __ldg(usteps + at);
    }
  };
  fetch_steps(r, as);
#pragma unroll
  for (int i = 0; i < AHEAD - 1; ++i) copy(i);
  for (int64_t lead = (int64_t)blockIdx.y * t.slab; lead < p.end;) {
    uint32_t ng[AHEAD], nu[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) ng[i] = bg[i], nu[i] = bu[i];
    if (lead + AHEAD * p.step < p.end) fetch_steps(r + AHEAD * p.step, as + AHEAD * ds);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (lead >= p.end) break;
      const int n = r < p.end ? p.n : 0;
      float g[CHUNK], u[CHUNK], d[CHUNK], a[CHUNK];
      wait_groups<AHEAD - 2>();
      din.landed();
      din.take(i, n, d);
      din.done();
      chunk_values(code.take(2 * i), ng[i], g);
      chunk_values(code.take(2 * i + 1), nu[i], u);
      copy((i + AHEAD - 1) % AHEAD);
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int e = 0; e < CHUNK; ++e) {
          float dp;
          const float s = gate_sigmoid<KIND>(g[e], &dp), act = __fmul_rn(g[e], s);
          const float slope = __fmaf_rn(__fmul_rn(act, __fsub_rn(1.0f, s)), dp, s);
          g[e] = __fmul_rn(__fmul_rn(d[e], u[e]), slope);  // dgate
          a[e] = __fmul_rn(act, u[e]);
          u[e] = __fmul_rn(d[e], act);  // dup
        }
      } else {
#pragma unroll
        for (int e = 0; e < CHUNK; e += 2) {
          F2 dp;
          const F2 s = gate_sigmoid2<KIND>(g + e, &dp), act = mul2(get2(g + e), s), de = get2(d + e), ue = get2(u + e);
          const F2 slope = fma2(mul2(act, fma2(s, f2(-1.0f), f2(1.0f))), dp, s);
          put2(g + e, mul2(mul2(de, ue), slope));
          put2(a + e, mul2(act, ue));
          put2(u + e, mul2(de, act));
        }
      }
      gto.put(g, n, r < p.end, own);
      uto.put(u, n, r < p.end, own);
      if (ocodes) {
        const uint32_t b = chunk_step(a);
        const uint2 q = chunk_codes(a, b);
        if (p.in && r < p.end) {
          *reinterpret_cast<uint2*>(ocodes + ac) = q;
          if ((p.c8 & 3) == 0) osteps[as] = (uint8_t)b;
        }
      }
      ac += dc, as += ds, r += p.step, lead += p.step;
    }
  }
}

// The kernel for rows on 16-byte boundaries, or for any.  (fp32 takes spans
// always: 8 fp32 per lane are 32 bytes, and copies of every other 16 bytes
// reached 0.6 of the copy's rate.)
template <typename K>
struct RowKernel {
  K kern;
  int ctas;  // that an SM holds
};
template <auto ALIGNED, auto ANY>
static RowKernel<decltype(ANY)> row_kernel(bool span) {
  return span ? RowKernel<decltype(ANY)>{ANY, resident<ANY>()} : RowKernel<decltype(ANY)>{ALIGNED, resident<ALIGNED>()};
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
  const bool span = !chunk_aligned(x, ld, dtype);
  GC_BY_DTYPE(dtype, T, {
    const auto k = row_kernel<&k_act_compress<T, sizeof(T) == 4>, &k_act_compress<T, true>>(span);
    dim3 grid;
    // of the six that fit three, longer ones: 777 x 4096 takes 3.1 us instead of
    // 3.7 (but spans of 4000 x 3333, bound by instructions, 17.2 instead of 11.9)
    const Tiling t = make_tiling(rows, cols, span, span || k.ctas < 3 ? k.ctas : 3, &grid);
    launch_chained(k.kern, grid, 256, 0, static_cast<cudaStream_t>(stream), static_cast<const T*>(x), ld, t, codes, steps);
  });
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}

extern "C" gc_status gc_act_decompress(const int8_t* codes, const uint8_t* steps, int64_t rows, int64_t cols,
                                       void* out, int64_t ldo, int32_t dtype, void* stream) {
  NvtxRange nvtx_range("gc_act_decompress");
  gc_status st = validate_matrix(rows, cols, dtype);
  if (st != GC_OK) return st;
  if (rows == 0) return GC_OK;
  if ((st = check_codes(codes, steps)) != GC_OK || (st = check_matrix(out, ldo, cols, dtype)) != GC_OK) return st;
  const bool span = !chunk_aligned(out, ldo, dtype);
  GC_BY_DTYPE(dtype, T, {
    const auto k = row_kernel<&k_act_decompress<T, sizeof(T) == 4>, &k_act_decompress<T, true>>(span);
    dim3 grid;
    const Tiling t = make_tiling(rows, cols, span, k.ctas, &grid);
    launch_chained(k.kern, grid, 256, 0, static_cast<cudaStream_t>(stream), codes, steps, t, static_cast<T*>(out), ldo);
  });
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
  const bool span = !(chunk_aligned(gate, ldg, dtype) && chunk_aligned(up, ldu, dtype) && chunk_aligned(out, ldo, dtype));
  GC_BY_DTYPE(dtype, T, {
    constexpr bool S = sizeof(T) == 4;
    const auto k = kind == GC_GATE_SILU ? row_kernel<&k_gated<T, GC_GATE_SILU, S>, &k_gated<T, GC_GATE_SILU, true>>(span)
                                        : row_kernel<&k_gated<T, GC_GATE_GELU_TANH, S>, &k_gated<T, GC_GATE_GELU_TANH, true>>(span);
    dim3 grid;
    const Tiling t = make_tiling(rows, cols, span, k.ctas, &grid);
    launch_chained(k.kern, grid, 256, 0, static_cast<cudaStream_t>(stream), static_cast<const T*>(gate), ldg,
                   static_cast<const T*>(up), ldu, t, static_cast<T*>(out), ldo, gate_codes, gate_steps, up_codes,
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
  const bool span = !(chunk_aligned(dout, lddo, dtype) && chunk_aligned(dgate, lddg, dtype) && chunk_aligned(dup, lddu, dtype));
  GC_BY_DTYPE(dtype, T, {
    constexpr bool S = sizeof(T) == 4;
    const auto k = kind == GC_GATE_SILU
                       ? row_kernel<&k_gated_backward<T, GC_GATE_SILU, S>, &k_gated_backward<T, GC_GATE_SILU, true>>(span)
                       : row_kernel<&k_gated_backward<T, GC_GATE_GELU_TANH, S>, &k_gated_backward<T, GC_GATE_GELU_TANH, true>>(span);
    dim3 grid;
    const Tiling t = make_tiling(rows, cols, span, k.ctas, &grid);
    launch_chained(k.kern, grid, 256, 0, static_cast<cudaStream_t>(stream), static_cast<const T*>(dout), lddo, gate_codes,
                   gate_steps, up_codes, up_steps, t, static_cast<T*>(dgate), lddg, static_cast<T*>(dup), lddu,
                   out_codes, out_steps);
  });
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}
