// The global gradient norm over many tensors, and clipping by it.
#include <algorithm>
#include <new>
#include <vector>

#include "gc_act.cuh"
#include "gc_host.h"

namespace gc {

// A launch takes its tensors' addresses by value, as a kernel parameter: no
// table in device memory that would have to be kept, copied or waited for, and
// gradients may lie elsewhere at every call.  The tensors are cut into tiles of
// GN_TILE elements; a CTA takes a contiguous range of all tiles.
constexpr int GN_TILE = 4096, GN_CAP = 1024, GN_CTAS = 152 * 6;
template <int CAP>
struct GnTable {
  const void* in[CAP];
  int64_t n[CAP];
  uint32_t first[CAP + 1];  // tile that the tensor starts with
  uint8_t type[CAP];
  int32_t count;
};
template <int CAP>
struct GcTable {
  GnTable<CAP> t;
  void* out[CAP];
  uint8_t otype[CAP];
};

// The tensor that holds a tile.
template <int CAP>
__device__ __forceinline__ int gn_tensor(const GnTable<CAP>& t, uint32_t tile) {
  int lo = 0, hi = t.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.first[mid] <= tile)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// The sum of squares of each CTA's tiles, in 64 bits, in an order that the sizes
// alone set.
template <int CAP>
__global__ void __launch_bounds__(256) k_grad_norm(const __grid_constant__ GnTable<CAP> t, double* part) {
  __shared__ double warps[8];
  chain_wait();
  const uint32_t tiles = t.first[t.count];
  const uint32_t begin = (uint32_t)((uint64_t)tiles * blockIdx.x / gridDim.x), end = (uint32_t)((uint64_t)tiles * (blockIdx.x + 1) / gridDim.x);
  double sum = 0.0;
  int i = begin < end ? gn_tensor(t, begin) : 0;
  for (uint32_t tile = begin; tile < end; ++tile) {
    while (tile >= t.first[i + 1]) ++i;
    const int64_t from = (int64_t)(tile - t.first[i]) * GN_TILE, to = min(from + GN_TILE, t.n[i]);
    for (int64_t e = from + threadIdx.x; e < to; e += 256) {
      const double x = (double)load_as_f32(t.in[i], t.type[i], e);
      sum += x * x;
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(FULL, sum, d);
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) sum += warps[w];
    part[blockIdx.x] = sum;
  }
}

// The root of the CTAs' sums, added in their order.
__global__ void __launch_bounds__(256) k_grad_norm_join(const double* part, int count, float* norm) {
  __shared__ double warps[8];
  chain_wait();
  double sum = 0.0;
  for (int i = threadIdx.x; i < count; i += 256) sum += part[i];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(FULL, sum, d);
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) sum += warps[w];
    *norm = (float)sqrt(sum);
  }
}

__device__ __forceinline__ void store_f32(void* p, int dtype, int64_t i, float v) {
  if (dtype == GC_F32)
    static_cast<float*>(p)[i] = v;
  else if (dtype == GC_BF16)
    static_cast<__nv_bfloat16*>(p)[i] = from_f32<__nv_bfloat16>(v);
  else
    static_cast<__half*>(p)[i] = from_f32<__half>(v);
}

template <int CAP>
__global__ void __launch_bounds__(256) k_grad_clip(const __grid_constant__ GcTable<CAP> g, const float* norm, float max_norm) {
  chain_wait();
  const GnTable<CAP>& t = g.t;
  const float n = *norm, c = n > max_norm ? __fdiv_rn(max_norm, n) : 1.0f;
  const uint32_t tiles = t.first[t.count];
  const uint32_t begin = (uint32_t)((uint64_t)tiles * blockIdx.x / gridDim.x), end = (uint32_t)((uint64_t)tiles * (blockIdx.x + 1) / gridDim.x);
  int i = begin < end ? gn_tensor(t, begin) : 0;
  for (uint32_t tile = begin; tile < end; ++tile) {
    while (tile >= t.first[i + 1]) ++i;
    if (c == 1.0f && g.out[i] == t.in[i]) continue;  // in place, as it is
    const int64_t from = (int64_t)(tile - t.first[i]) * GN_TILE, to = min(from + GN_TILE, t.n[i]);
    for (int64_t e = from + threadIdx.x; e < to; e += 256)
      store_f32(g.out[i], g.otype[i], e, __fmul_rn(c, load_as_f32(t.in[i], t.type[i], e)));
  }
}

// The checks of a list of tensors.  So many elements are at most 2^30 tiles.
constexpr int64_t GN_MOST = INT64_C(1) << 42;
static gc_status check_tensors(const gc_tensor* t, int32_t count) {
  if (count < 0 || (count > 0 && !t)) return GC_ERR_INVALID_ARG;
  int64_t left = GN_MOST;
  for (int32_t i = 0; i < count; ++i) {
    if (!valid_dtype(t[i].dtype) || (t[i].numel > 0 && !t[i].data)) return GC_ERR_INVALID_ARG;
    if (t[i].numel < 0 || t[i].numel > left) return GC_ERR_LAYOUT;
    left -= t[i].numel;
    const gc_status st = check_vector(t[i].data, t[i].dtype);
    if (st != GC_OK) return st;
  }
  return GC_OK;
}
static int32_t grad_launches(int32_t count) { return (count + GN_CAP - 1) / GN_CAP; }

// Fills a table with tensors from `at` on, as many as there is room for;
// returns the first that is not in it.
template <int CAP>
static int32_t fill_table(GnTable<CAP>* t, const gc_tensor* in, int32_t at, int32_t count, int32_t (&from)[CAP]) {
  t->count = 0;
  uint64_t tiles = 0;
  for (; at < count && t->count < CAP; ++at) {
    if (in[at].numel == 0) continue;
    t->in[t->count] = in[at].data, t->n[t->count] = in[at].numel, t->type[t->count] = (uint8_t)in[at].dtype;
    t->first[t->count] = (uint32_t)tiles, from[t->count] = at;
    tiles += ((uint64_t)in[at].numel + GN_TILE - 1) / GN_TILE, ++t->count;
  }
  t->first[t->count] = (uint32_t)tiles;
  return at;
}
static unsigned grad_grid(uint32_t tiles) { return tiles < (uint32_t)GN_CTAS ? tiles : (unsigned)GN_CTAS; }

template <int CAP>
static int32_t launch_norm(const gc_tensor* in, int32_t at, int32_t count, double* part, int* parts, cudaStream_t s) {
  GnTable<CAP> t;
  int32_t from[CAP];
  at = fill_table(&t, in, at, count, from);
  if (t.count == 0) return at;
  const unsigned grid = grad_grid(t.first[t.count]);
  launch_chained(&k_grad_norm<CAP>, grid, 256, 0, s, t, part + *parts);
  *parts += (int)grid;
  return at;
}
template <int CAP>
static int32_t launch_clip(const gc_tensor* in, const gc_tensor* out, int32_t at, int32_t count, const float* norm, float max_norm,
                           cudaStream_t s) {
  GcTable<CAP> g;
  int32_t from[CAP];
  at = fill_table(&g.t, in, at, count, from);
  if (g.t.count == 0) return at;
  for (int i = 0; i < g.t.count; ++i) g.out[i] = out[from[i]].data, g.otype[i] = (uint8_t)out[from[i]].dtype;
  launch_chained(&k_grad_clip<CAP>, grad_grid(g.t.first[g.t.count]), 256, 0, s, g, norm, max_norm);
  return at;
}

// Whether no two tensors that are written share memory, and none that is
// written holds any of another one that is read, or the norm.
static gc_status check_apart(const gc_tensor* in, const gc_tensor* out, int32_t count, const float* norm) {
  struct Range {
    uintptr_t begin, end;
  };
  try {
    std::vector<Range> w;
    w.reserve((size_t)count);
    for (int32_t i = 0; i < count; ++i)
      if (out[i].numel > 0) {
        const uintptr_t p = (uintptr_t)out[i].data;
        w.push_back({p, p + (uintptr_t)out[i].numel * dtype_bytes(out[i].dtype)});
      }
    const auto before = [](const Range& a, const Range& b) { return a.begin < b.begin; };
    if (!std::is_sorted(w.begin(), w.end(), before)) std::sort(w.begin(), w.end(), before);
    for (size_t i = 1; i < w.size(); ++i)
      if (w[i].begin < w[i - 1].end) return GC_ERR_INVALID_ARG;
    const auto meets = [&w](uintptr_t p, uintptr_t end) {  // the first written range that ends after p
      const auto r = std::upper_bound(w.begin(), w.end(), p, [](uintptr_t x, const Range& a) { return x < a.end; });
      return r != w.end() && r->begin < end;
    };
    if (meets((uintptr_t)norm, (uintptr_t)(norm + 1))) return GC_ERR_INVALID_ARG;
    for (int32_t i = 0; i < count; ++i) {
      if (in[i].numel == 0 || (in[i].data == out[i].data && in[i].dtype == out[i].dtype)) continue;
      const uintptr_t p = (uintptr_t)in[i].data;
      if (meets(p, p + (uintptr_t)in[i].numel * dtype_bytes(in[i].dtype))) return GC_ERR_INVALID_ARG;
    }
  } catch (const std::bad_alloc&) {
    return GC_ERR_CUDA;
  }
  return GC_OK;
}

}  // namespace gc

using namespace gc;

extern "C" gc_status gc_grad_norm_workspace_size(int32_t count, size_t* bytes) {
  if (count < 0 || !bytes) return GC_ERR_INVALID_ARG;
  *bytes = align_up((size_t)(grad_launches(count) > 1 ? grad_launches(count) : 1) * GN_CTAS * sizeof(double), 256);
  return GC_OK;
}

extern "C" gc_status gc_grad_norm(const gc_tensor* tensors, int32_t count, float* norm, void* workspace, size_t ws_bytes,
                                  void* stream) {
  NvtxRange nvtx_range("gc_grad_norm");
  gc_status st = check_tensors(tensors, count);
  if (st != GC_OK) return st;
  if (!norm) return GC_ERR_INVALID_ARG;
  size_t need = 0;
  if ((st = gc_grad_norm_workspace_size(count, &need)) != GC_OK || (st = check_vector(norm, GC_F32)) != GC_OK ||
      (st = check_workspace(workspace, ws_bytes, need)) != GC_OK)
    return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  double* const part = static_cast<double*>(workspace);
  int parts = 0;
  for (int32_t at = 0; at < count;)
    at = count - at <= 16 ? launch_norm<16>(tensors, at, count, part, &parts, s)
         : count - at <= 192 ? launch_norm<192>(tensors, at, count, part, &parts, s)
                             : launch_norm<GN_CAP>(tensors, at, count, part, &parts, s);
  launch_chained(k_grad_norm_join, 1, 256, 0, s, part, parts, norm);
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}

extern "C" gc_status gc_grad_clip(const gc_tensor* in, const gc_tensor* out, int32_t count, const float* norm, float max_norm,
                                  void* stream) {
  NvtxRange nvtx_range("gc_grad_clip");
  gc_status st = check_tensors(in, count);
  if (st != GC_OK || (st = check_tensors(out, count)) != GC_OK) return st;
  if (!norm || !(max_norm >= 0.0f)) return GC_ERR_INVALID_ARG;
  if ((st = check_vector(norm, GC_F32)) != GC_OK) return st;
  bool any = false;
  for (int32_t i = 0; i < count; ++i) {
    if (in[i].numel != out[i].numel) return GC_ERR_LAYOUT;
    any = any || in[i].numel > 0;
  }
  if ((st = check_apart(in, out, count, norm)) != GC_OK || !any) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  for (int32_t at = 0; at < count;)
    at = count - at <= 16 ? launch_clip<16>(in, out, at, count, norm, max_norm, s)
         : count - at <= 192 ? launch_clip<192>(in, out, at, count, norm, max_norm, s)
                             : launch_clip<GN_CAP>(in, out, at, count, norm, max_norm, s);
  return cudaGetLastError() == cudaSuccess ? GC_OK : GC_ERR_CUDA;
}
