// RMS norm with the residual's addition, its checkpoint and its gradient.
#include "gc_act.cuh"
#include "gc_host.h"

namespace gc {

constexpr int NTHREADS = 256;

// The sum over the CTA, the same bits in every thread.
__device__ __forceinline__ float cta_sum(float v, float* red) {
  for (int o = 16; o; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(FULL, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = red[0];
  for (int w = 1; w < NTHREADS / 32; ++w) s = __fadd_rn(s, red[w]);
  return s;
}

// One CTA per row: the sum of squares, then the outputs, a warp per group.
template <typename T>
__global__ void __launch_bounds__(NTHREADS)
    k_rmsnorm(const T* x, int64_t ldx, const T* res, int64_t ldr, const void* weight, int wtype, float eps,
              int64_t rows, int64_t cols, int64_t groups, T* y, int64_t ldy, T* h, int64_t ldh, float* rstd,
              int8_t* codes, uint8_t* steps) {
  __shared__ float red[NTHREADS / 32];
  chain_wait();
  const int lane = threadIdx.x & 31;
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    auto sum_at = [&](int64_t c) {
      const float v = to_f32(x[r * ldx + c]);
      return res ? __fadd_rn(v, to_f32(res[r * ldr + c])) : v;
    };
    float ss = 0.0f;
    for (int64_t c = threadIdx.x; c < cols; c += NTHREADS) {
      const float v = sum_at(c);
      ss = __fmaf_rn(v, v, ss);
    }
    ss = cta_sum(ss, red);
    const float rs = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)cols), eps)));
    if (rstd && threadIdx.x == 0) rstd[r] = rs;
    for (int64_t g = threadIdx.x >> 5; g < groups; g += NTHREADS / 32) {
      const int64_t c = g * 32 + lane;
      const float v = c < cols ? sum_at(c) : 0.0f;
      const float q = c < cols ? __fmul_rn(v, rs) : 0.0f;
      if (c < cols) {
        if (h) h[r * ldh + c] = from_f32<T>(v);
        if (y) y[r * ldy + c] = from_f32<T>(weight ? __fmul_rn(q, load_as_f32(weight, wtype, c)) : q);
      }
      if (codes) {
        const uint32_t b = act_step(__reduce_max_sync(FULL, __float_as_uint(fabsf(q))));
        codes[(r * groups + g) * 32 + lane] = (int8_t)act_code(q, act_inverse(b));
        if (lane == 0) steps[r * groups + g] = (uint8_t)b;
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(NTHREADS)
    k_rmsnorm_backward(const T* dy, int64_t lddy, const T* dh, int64_t lddh, const int8_t* codes, const uint8_t* steps,
                       const float* rstd, const void* weight, int wtype, int64_t rows, int64_t cols, int64_t groups,
                       T* dx, int64_t lddx) {
  __shared__ float red[NTHREADS / 32];
  chain_wait();
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    auto terms = [&](int64_t c, float* q) {
      *q = __fmul_rn((float)codes[r * groups * 32 + c], act_scale(steps[r * groups + c / 32]));
      const float d = to_f32(dy[r * lddy + c]);
      return weight ? __fmul_rn(d, load_as_f32(weight, wtype, c)) : d;
    };
    float s = 0.0f;
    for (int64_t c = threadIdx.x; c < cols; c += NTHREADS) {
      float q;
      const float gw = terms(c, &q);
      s = __fmaf_rn(gw, q, s);
    }
    s = __fdiv_rn(cta_sum(s, red), (float)cols);
    const float rs = rstd[r];
    for (int64_t c = threadIdx.x; c < cols; c += NTHREADS) {
      float q;
      const float gw = terms(c, &q);
      float v = __fmul_rn(rs, __fmaf_rn(-q, s, gw));
      if (dh) v = __fadd_rn(v, to_f32(dh[r * lddh + c]));
      dx[r * lddx + c] = from_f32<T>(v);
    }
  }
}

// dw[c] over rows [p * span, (p + 1) * span) of part p: a thread per column.
template <typename T>
__global__ void __launch_bounds__(NTHREADS)
    k_rmsnorm_dw(const T* dy, int64_t lddy, const int8_t* codes, const uint8_t* steps, int64_t rows, int64_t cols,
                 int64_t groups, int64_t span, float* part) {
  chain_wait();
  const int64_t c = (int64_t)blockIdx.x * NTHREADS + threadIdx.x;
  if (c >= cols) return;
  const int64_t r0 = blockIdx.y * span, r1 = min(r0 + span, rows);
  float s = 0.0f;
  for (int64_t r = r0; r < r1; ++r)
    s = __fmaf_rn(to_f32(dy[r * lddy + c]),
                  __fmul_rn((float)codes[r * groups * 32 + c], act_scale(steps[r * groups + c / 32])), s);
  part[blockIdx.y * cols + c] = s;
}

__global__ void __launch_bounds__(NTHREADS) k_rmsnorm_dw_join(const float* part, int parts, int64_t cols, float* dw,
                                                              int accumulate) {
  chain_wait();
  const int64_t c = (int64_t)blockIdx.x * NTHREADS + threadIdx.x;
  if (c >= cols) return;
  float s = 0.0f;
  for (int p = 0; p < parts; ++p) s = __fadd_rn(s, part[p * cols + c]);
  dw[c] = accumulate ? __fadd_rn(dw[c], s) : s;
}

static int dw_parts(int64_t rows) { return (int)(rows < 64 ? (rows < 1 ? 1 : rows) : 64); }

}  // namespace gc

using namespace gc;

extern "C" gc_status gc_rmsnorm(const void* x, int64_t ldx, const void* residual, int64_t ldr, int32_t dtype,
                                const void* weight, int32_t weight_dtype, float eps, int64_t rows, int64_t cols,
                                void* y, int64_t ldy, void* h, int64_t ldh, float* rstd, int8_t* codes,
                                uint8_t* steps, void* stream) {
  NvtxRange nvtx_range("gc_rmsnorm");
  gc_status st = validate_matrix(rows, cols, dtype);
  if (st != GC_OK) return st;
  if (!(eps >= 0.0f) || (weight && !valid_dtype(weight_dtype))) return GC_ERR_INVALID_ARG;
  if (rows == 0) return GC_OK;
  if ((st = check_matrix(x, ldx, cols, dtype)) != GC_OK ||
      (residual && (st = check_matrix(residual, ldr, cols, dtype)) != GC_OK) ||
      (y && (st = check_matrix(y, ldy, cols, dtype)) != GC_OK) ||
      (h && (st = check_matrix(h, ldh, cols, dtype)) != GC_OK) ||
      ((codes || steps) && (st = check_codes(codes, steps)) != GC_OK))
    return st;
  const int64_t groups = act_ldc(cols) / 32;
  const unsigned grid = (unsigned)(rows < 152 * 64 ? rows : 152 * 64);
  GC_BY_DTYPE(dtype, T, launch_chained(k_rmsnorm<T>, grid, NTHREADS, 0, static_cast<cudaStream_t>(stream),
                                       static_cast<const T*>(x), ldx, static_cast<const T*>(residual), ldr, weight,
                                       weight_dtype, eps, rows, cols, groups, static_cast<T*>(y), ldy,
                                       static_cast<T*>(h), ldh, rstd, codes, steps));
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}

extern "C" gc_status gc_rmsnorm_backward_workspace_size(int64_t rows, int64_t cols, size_t* bytes) {
  const gc_status st = validate_matrix(rows, cols, GC_F32);
  if (st != GC_OK) return st;
  if (!bytes) return GC_ERR_INVALID_ARG;
  *bytes = (size_t)dw_parts(rows) * (size_t)cols * sizeof(float);
  return GC_OK;
}

extern "C" gc_status gc_rmsnorm_backward(const void* dy, int64_t lddy, const void* dh, int64_t lddh, int32_t dtype,
                                         const int8_t* codes, const uint8_t* steps, const float* rstd,
                                         const void* weight, int32_t weight_dtype, int64_t rows, int64_t cols,
                                         void* dx, int64_t lddx, float* dw, uint32_t flags, void* workspace,
                                         size_t ws_bytes, void* stream) {
  NvtxRange nvtx_range("gc_rmsnorm_backward");
  gc_status st = validate_matrix(rows, cols, dtype);
  if (st != GC_OK) return st;
  if ((weight && !valid_dtype(weight_dtype)) || (flags & ~GC_ACCUMULATE)) return GC_ERR_INVALID_ARG;
  if (dw) {
    size_t need = 0;
    gc_rmsnorm_backward_workspace_size(rows, cols, &need);
    if ((st = check_workspace(workspace, ws_bytes, need)) != GC_OK) return st;
    if ((uintptr_t)dw & 3u) return GC_ERR_ALIGNMENT;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned cgrid = (unsigned)((cols + NTHREADS - 1) / NTHREADS);
  const int acc = (flags & GC_ACCUMULATE) ? 1 : 0;
  if (rows == 0) {
    if (dw && !acc) launch_chained(k_rmsnorm_dw_join, cgrid, NTHREADS, 0, s, (const float*)nullptr, 0, cols, dw, 0);
    return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
  }
  if ((st = check_matrix(dy, lddy, cols, dtype)) != GC_OK || (dh && (st = check_matrix(dh, lddh, cols, dtype)) != GC_OK) ||
      (st = check_matrix(dx, lddx, cols, dtype)) != GC_OK || (st = check_codes(codes, steps)) != GC_OK)
    return st;
  if (!rstd) return GC_ERR_INVALID_ARG;
  const int64_t groups = act_ldc(cols) / 32;
  const unsigned grid = (unsigned)(rows < 152 * 64 ? rows : 152 * 64);
  if (dw) {  // before dx, which may overwrite dy
    float* part = static_cast<float*>(workspace);
    const int parts = dw_parts(rows);
    GC_BY_DTYPE(dtype, T, launch_chained(k_rmsnorm_dw<T>, dim3(cgrid, parts), NTHREADS, 0, s,
                                         static_cast<const T*>(dy), lddy, codes, steps, rows, cols, groups,
                                         (rows + parts - 1) / parts, part));
    launch_chained(k_rmsnorm_dw_join, cgrid, NTHREADS, 0, s, (const float*)part, parts, cols, dw, acc);
  }
  GC_BY_DTYPE(dtype, T, launch_chained(k_rmsnorm_backward<T>, grid, NTHREADS, 0, s, static_cast<const T*>(dy), lddy,
                                       static_cast<const T*>(dh), lddh, codes, steps, rstd, weight, weight_dtype, rows,
                                       cols, groups, static_cast<T*>(dx), lddx));
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}
