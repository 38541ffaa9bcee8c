// Checkpoints of activations in 8 bits and the gated activation around them.
#include "gc_act.cuh"
#include "gc_host.h"

namespace gc {

// One warp per group of 32 columns, a lane per column.
template <typename T>
__global__ void __launch_bounds__(256) k_act_compress(const T* x, int64_t ld, int64_t rows, int64_t cols,
                                                      int64_t groups, int8_t* codes, uint8_t* steps) {
  chain_wait();
  const int lane = threadIdx.x & 31;
  const int64_t total = rows * groups, stride = (int64_t)gridDim.x * 8;
  for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < total; i += stride) {
    const int64_t r = i / groups, c = (i - r * groups) * 32 + lane;
    const float v = c < cols ? to_f32(x[r * ld + c]) : 0.0f;
    const uint32_t b = act_step(__reduce_max_sync(FULL, __float_as_uint(fabsf(v))));
    codes[i * 32 + lane] = (int8_t)act_code(v, act_inverse(b));
    if (lane == 0) steps[i] = (uint8_t)b;
  }
}

template <typename T>
__global__ void __launch_bounds__(256) k_act_decompress(const int8_t* codes, const uint8_t* steps, int64_t rows,
                                                        int64_t cols, int64_t groups, T* out, int64_t ld) {
  chain_wait();
  const int lane = threadIdx.x & 31;
  const int64_t total = rows * groups, stride = (int64_t)gridDim.x * 8;
  for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < total; i += stride) {
    const int64_t r = i / groups, c = (i - r * groups) * 32 + lane;
    if (c < cols) out[r * ld + c] = from_f32<T>(__fmul_rn((float)codes[i * 32 + lane], act_scale(steps[i])));
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
template <int KIND>
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
  float e = expf(far ? p : -p);
  if (KIND == GC_GATE_GELU_TANH) e = __fmaf_rn(e, far ? low : -low, e);
  return far ? e : __fdiv_rn(1.0f, __fadd_rn(1.0f, e));
}

template <typename T, int KIND>
__global__ void __launch_bounds__(256)
    k_gated(const T* gate, int64_t ldg, const T* up, int64_t ldu, int64_t rows, int64_t cols, int64_t groups,
            T* out, int64_t ldo, int8_t* gcodes, uint8_t* gsteps, int8_t* ucodes, uint8_t* usteps) {
  chain_wait();
  const int lane = threadIdx.x & 31;
  const int64_t total = rows * groups, stride = (int64_t)gridDim.x * 8;
  for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < total; i += stride) {
    const int64_t r = i / groups, c = (i - r * groups) * 32 + lane;
    const float g = c < cols ? to_f32(gate[r * ldg + c]) : 0.0f, u = c < cols ? to_f32(up[r * ldu + c]) : 0.0f;
    float dp;
    if (c < cols) out[r * ldo + c] = from_f32<T>(__fmul_rn(__fmul_rn(g, gate_sigmoid<KIND>(g, &dp)), u));
    if (gcodes) {
      const uint32_t bg = act_step(__reduce_max_sync(FULL, __float_as_uint(fabsf(g))));
      const uint32_t bu = act_step(__reduce_max_sync(FULL, __float_as_uint(fabsf(u))));
      gcodes[i * 32 + lane] = (int8_t)act_code(g, act_inverse(bg));
      ucodes[i * 32 + lane] = (int8_t)act_code(u, act_inverse(bu));
      if (lane == 0) gsteps[i] = (uint8_t)bg, usteps[i] = (uint8_t)bu;
    }
  }
}

template <typename T, int KIND>
__global__ void __launch_bounds__(256)
    k_gated_backward(const T* dout, int64_t lddo, const int8_t* gcodes, const uint8_t* gsteps,
                     const int8_t* ucodes, const uint8_t* usteps, int64_t rows, int64_t cols, int64_t groups, T* dgate,
                     int64_t lddg, T* dup, int64_t lddu, int8_t* ocodes, uint8_t* osteps) {
  chain_wait();
  const int lane = threadIdx.x & 31;
  const int64_t total = rows * groups, stride = (int64_t)gridDim.x * 8;
  for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < total; i += stride) {
    const int64_t r = i / groups, c = (i - r * groups) * 32 + lane;
    const float g = __fmul_rn((float)gcodes[i * 32 + lane], act_scale(gsteps[i]));
    const float u = __fmul_rn((float)ucodes[i * 32 + lane], act_scale(usteps[i]));
    float dp;
    const float s = gate_sigmoid<KIND>(g, &dp), a = __fmul_rn(g, s);
    if (c < cols) {
      const float d = to_f32(dout[r * lddo + c]);
      dgate[r * lddg + c] = from_f32<T>(d * u * __fmaf_rn(a * (1.0f - s), dp, s));
      dup[r * lddu + c] = from_f32<T>(d * a);
    }
    if (ocodes) {
      const float v = __fmul_rn(a, u);
      const uint32_t b = act_step(__reduce_max_sync(FULL, __float_as_uint(fabsf(v))));
      ocodes[i * 32 + lane] = (int8_t)act_code(v, act_inverse(b));
      if (lane == 0) osteps[i] = (uint8_t)b;
    }
  }
}

static unsigned groups_grid(int64_t total) {
  const int64_t blocks = (total + 7) / 8;
  return (unsigned)(blocks < 152 * 64 ? blocks : 152 * 64);
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
  const int64_t groups = act_ldc(cols) / 32;
  GC_BY_DTYPE(dtype, T, launch_chained(k_act_compress<T>, groups_grid(rows * groups), 256, 0,
                                       static_cast<cudaStream_t>(stream), static_cast<const T*>(x), ld, rows, cols,
                                       groups, codes, steps));
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}

extern "C" gc_status gc_act_decompress(const int8_t* codes, const uint8_t* steps, int64_t rows, int64_t cols,
                                       void* out, int64_t ldo, int32_t dtype, void* stream) {
  NvtxRange nvtx_range("gc_act_decompress");
  gc_status st = validate_matrix(rows, cols, dtype);
  if (st != GC_OK) return st;
  if (rows == 0) return GC_OK;
  if ((st = check_codes(codes, steps)) != GC_OK || (st = check_matrix(out, ldo, cols, dtype)) != GC_OK) return st;
  const int64_t groups = act_ldc(cols) / 32;
  GC_BY_DTYPE(dtype, T, launch_chained(k_act_decompress<T>, groups_grid(rows * groups), 256, 0,
                                       static_cast<cudaStream_t>(stream), codes, steps, rows, cols, groups,
                                       static_cast<T*>(out), ldo));
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
  const int64_t groups = act_ldc(cols) / 32;
  GC_BY_DTYPE(dtype, T, launch_chained(kind == GC_GATE_SILU ? k_gated<T, GC_GATE_SILU> : k_gated<T, GC_GATE_GELU_TANH>,
                                       groups_grid(rows * groups), 256, 0, static_cast<cudaStream_t>(stream), static_cast<const T*>(gate), ldg,
                                       static_cast<const T*>(up), ldu, rows, cols, groups, static_cast<T*>(out), ldo,
                                       gate_codes, gate_steps, up_codes, up_steps));
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
  const int64_t groups = act_ldc(cols) / 32;
  GC_BY_DTYPE(dtype, T, launch_chained(kind == GC_GATE_SILU ? k_gated_backward<T, GC_GATE_SILU>
                                                            : k_gated_backward<T, GC_GATE_GELU_TANH>,
                                       groups_grid(rows * groups), 256, 0, static_cast<cudaStream_t>(stream), static_cast<const T*>(dout), lddo,
                                       gate_codes, gate_steps, up_codes, up_steps, rows, cols, groups,
                                       static_cast<T*>(dgate), lddg, static_cast<T*>(dup), lddu, out_codes,
                                       out_steps));
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}
