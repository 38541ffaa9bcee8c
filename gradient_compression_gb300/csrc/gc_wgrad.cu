// Weight gradient from an activation checkpoint.
#include "gc_act.cuh"
#include "gc_host.h"

namespace gc {

// 32 x 32 tile of dw per CTA of 32 x 8 threads, 32 rows of dy and q at a
// time in shared memory, fp32 multiply-adds.
template <typename T>
__global__ void __launch_bounds__(256)
    k_weight_grad(const T* dy, int64_t lddy, int64_t rows, int64_t n, const int8_t* codes, const uint8_t* steps,
                  int64_t k, int64_t groups, const void* cscale, int ctype, float* dw, int64_t lddw, int accumulate) {
  __shared__ float sa[32][33], sb[32][33];
  chain_wait();
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int64_t n0 = (int64_t)blockIdx.y * 32, k0 = (int64_t)blockIdx.x * 32, kc = k0 + tx;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t t0 = 0; t0 < rows; t0 += 32) {
    __syncthreads();
    for (int i = ty; i < 32; i += 8) {
      const int64_t t = t0 + i;
      sa[i][tx] = t < rows && n0 + tx < n ? to_f32(dy[t * lddy + n0 + tx]) : 0.0f;
      sb[i][tx] = t < rows && kc < k
                      ? __fmul_rn((float)codes[t * groups * 32 + kc], act_scale(steps[t * groups + kc / 32]))
                      : 0.0f;
    }
    __syncthreads();
    for (int i = 0; i < 32; ++i)
      for (int j = 0; j < 4; ++j) acc[j] = __fmaf_rn(sa[i][ty + 8 * j], sb[i][tx], acc[j]);
  }
  for (int j = 0; j < 4; ++j) {
    const int64_t r = n0 + ty + 8 * j;
    if (r >= n || kc >= k) continue;
    const float v = cscale ? __fmul_rn(acc[j], load_as_f32(cscale, ctype, kc)) : acc[j];
    float* o = dw + r * lddw + kc;
    *o = accumulate ? __fadd_rn(*o, v) : v;
  }
}

}  // namespace gc

using namespace gc;

extern "C" gc_status gc_act_weight_grad_workspace_size(int64_t rows, int64_t n, int64_t k, int32_t dtype,
                                                       size_t* bytes) {
  gc_status st = validate_matrix(rows, n, dtype);
  if (st == GC_OK) st = validate_matrix(rows, k, dtype);
  if (st != GC_OK) return st;
  if (!bytes) return GC_ERR_INVALID_ARG;
  *bytes = 0;
  return GC_OK;
}

extern "C" gc_status gc_act_weight_grad(const void* dy, int64_t lddy, int32_t dtype, int64_t rows, int64_t n,
                                        const int8_t* codes, const uint8_t* steps, int64_t k, const void* col_scale,
                                        int32_t col_scale_dtype, float* dw, int64_t lddw, uint32_t flags,
                                        void* workspace, size_t ws_bytes, void* stream) {
  NvtxRange nvtx_range("gc_act_weight_grad");
  size_t need = 0;
  gc_status st = gc_act_weight_grad_workspace_size(rows, n, k, dtype, &need);
  if (st != GC_OK) return st;
  if ((col_scale && !valid_dtype(col_scale_dtype)) || (flags & ~GC_ACCUMULATE)) return GC_ERR_INVALID_ARG;
  if ((st = check_workspace(workspace, ws_bytes, need)) != GC_OK || (st = check_matrix(dw, lddw, k, GC_F32)) != GC_OK)
    return st;
  if (rows > 0 && ((st = check_matrix(dy, lddy, n, dtype)) != GC_OK || (st = check_codes(codes, steps)) != GC_OK))
    return st;
  const int64_t groups = act_ldc(k) / 32;
  const dim3 grid((unsigned)((k + 31) / 32), (unsigned)((n + 31) / 32));
  if (grid.y > 65535u) return GC_ERR_INVALID_ARG;
  GC_BY_DTYPE(dtype, T, launch_chained(k_weight_grad<T>, grid, 256, 0, static_cast<cudaStream_t>(stream),
                                       static_cast<const T*>(dy), lddy, rows, n, codes, steps, k, groups, col_scale,
                                       col_scale_dtype, dw, lddw, (flags & GC_ACCUMULATE) ? 1 : 0));
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}
