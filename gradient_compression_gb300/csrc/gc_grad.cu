// The global gradient norm over many tensors, and clipping by it.
#include <algorithm>
#include <new>
#include <vector>

#include "gc_act.cuh"
#include "gc_host.h"

namespace gc {

// A launch takes its tensors' addresses by value, as a kernel parameter: no
// table in device memory that would have to be kept, copied or waited for, and
// gradients may lie elsewhere at every call.  Memory is read in granules of 16
// bytes as they lie, whatever element a tensor starts at; GN_TILE granules are a
// tile, four for each thread of a CTA, which takes a contiguous range of all
// tiles, so that it looks a tensor up once and then walks on.
//
// Both kernels are one pass bound by memory.  The norm: six CTAs an SM, one wave
// (8.03e9 elements in bf16 2.18 ms, 7.4 TB/s; five or twelve the same, four 2.25,
// eight, whose registers do not suffice, 2.40).  Clipping: as many CTAs as there are
// tiles, up to 256 an SM, three at a time: 3.35e8 elements from bf16 to fp32 287 us,
// 7.0 TB/s, where 6 and 16 an SM take 349 and 316 (a CTA that has done its range
// makes room at once, and the ranges written at a time lie closer together).  In
// place 3.35e8 elements in bf16 take 189 us (7.1 TB/s), and 41 where nothing is to be
// clipped: so many CTAs' starts.
constexpr int GN_TILE = 1024, GN_CAP = 1024, GN_CTAS = 152 * 6, GC_CTAS = 152 * 256;
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

// The granules of a tensor that a thread has of a tile: thread, thread + 256, ...
// Element 0 of granule g is element g * E - skip of the tensor.
template <typename T>
struct Granules {
  static constexpr int E = 16 / (int)sizeof(T);
  int64_t e[4];  // the first element of each
  uint4 w[4];
  __device__ __forceinline__ Granules(const void* p, int64_t n, uint32_t tile) {
    const int skip = (int)((uintptr_t)p & 15u) / (int)sizeof(T);
    const uint4* from = reinterpret_cast<const uint4*>(static_cast<const char*>(p) - skip * sizeof(T));
    const int64_t g = (int64_t)tile * GN_TILE + threadIdx.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      e[i] = (g + 256 * i) * E - skip;
      w[i] = make_uint4(0u, 0u, 0u, 0u);
      if (e[i] < n)
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                     : "l"(from + g + 256 * i));
    }
  }
  __device__ __forceinline__ bool whole(int i, int64_t n) const { return e[i] >= 0 && e[i] + E <= n; }
  __device__ __forceinline__ void values(int i, float (&v)[E]) const {
    if constexpr (sizeof(T) == 4) {
      v[0] = __uint_as_float(w[i].x), v[1] = __uint_as_float(w[i].y), v[2] = __uint_as_float(w[i].z), v[3] = __uint_as_float(w[i].w);
    } else {
      Raw8<T> r;
      *reinterpret_cast<uint4*>(&r) = w[i];
      unpack(r, v);
    }
  }
};

// The squares of a thread's granules in 64 bits, for what fp32 does not hold.
// (Out of line: its registers would be the common path's.)
template <typename T>
__device__ __noinline__ double gn_squares64(const void* p, int64_t n, uint32_t tile) {
  constexpr int E = Granules<T>::E;
  const int skip = (int)((uintptr_t)p & 15u) / (int)sizeof(T);
  const int64_t g = (int64_t)tile * GN_TILE + threadIdx.x;
  double sum = 0.0;
  for (int i = 0; i < 4; ++i)
    for (int64_t e = max((g + 256 * i) * E - skip, (int64_t)0); e < min((g + 256 * i + 1) * E - skip, n); ++e) {
      const double x = (double)to_f32(static_cast<const T*>(p)[e]);
      sum += x * x;
    }
  return sum;
}

// The squares of a thread's granules.  Up to 32 elements are added in fp32,
// four chains of at most eight; where the result says that a square left fp32's
// range, or that all are so small that what was lost may matter, again in 64
// bits: elements below 2^-63, whose squares are rounded to multiples of 2^-149,
// do not matter beside a sum of 2^-80.  Tensors of such small elements (about 1e-12 and
// less) are read at 0.35 TB/s in bf16 and 0.69 in fp32 instead of 7: a few instructions
// in 64 bits for each element.
template <typename T>
__device__ __forceinline__ double gn_squares(const void* p, int64_t n, uint32_t tile) {
  using G = Granules<T>;
  constexpr int E = G::E;
  const G g(p, n, tile);
  F2 a = f2(0.0f), b = f2(0.0f);
  uint32_t any = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v[E];
    g.values(i, v);
    any |= g.w[i].x | g.w[i].y | g.w[i].z | g.w[i].w;
    if (!g.whole(i, n)) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (g.e[i] + e < 0 || g.e[i] + e >= n) v[e] = 0.0f;
    }
#pragma unroll
    for (int e = 0; e < E; e += 4) a = fma2(get2(v + e), get2(v + e), a), b = fma2(get2(v + e + 2), get2(v + e + 2), b);
  }
  float s[2];
  put2(s, add2(a, b));
  const float all = __fadd_rn(s[0], s[1]);
  if (any != 0u && !(all >= 0x1p-80f && all < __int_as_float(0x7f800000))) return gn_squares64<T>(p, n, tile);
  return (double)all;
}

// The sum of squares of each CTA's tiles, in 64 bits, in an order set by the sizes,
// the types and where in a granule each tensor starts (which elements are summed in
// fp32 together).
template <int CAP>
__global__ void __launch_bounds__(256, 6) k_grad_norm(const __grid_constant__ GnTable<CAP> t, double* part) {
  __shared__ double warps[8];
  chain_wait();
  const uint32_t tiles = t.first[t.count];
  const uint32_t begin = (uint32_t)((uint64_t)tiles * blockIdx.x / gridDim.x), end = (uint32_t)((uint64_t)tiles * (blockIdx.x + 1) / gridDim.x);
  double sum = 0.0;
  int i = begin < end ? gn_tensor(t, begin) : 0;
  for (uint32_t tile = begin; tile < end; ++i) {
    const uint32_t first = t.first[i], stop = min(t.first[i + 1], end);
    const void* const p = t.in[i];
    const int64_t n = t.n[i];
    const int type = t.type[i];
    if (type == GC_F32)
      for (; tile < stop; ++tile) sum += gn_squares<float>(p, n, tile - first);
    else if (type == GC_BF16)
      for (; tile < stop; ++tile) sum += gn_squares<__nv_bfloat16>(p, n, tile - first);
    else
      for (; tile < stop; ++tile) sum += gn_squares<__half>(p, n, tile - first);
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
  for (int i = threadIdx.x; i < count; i += 4 * 256) {  // four loads at a time: a wave's sums at once
    double v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = i + 256 * j < count ? part[i + 256 * j] : 0.0;
#pragma unroll
    for (int j = 0; j < 4; ++j) sum += v[j];
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(FULL, sum, d);
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) sum += warps[w];
    *norm = (float)sqrt(sum);
  }
}

// c times a tile.  Where the output's elements lie as the granules do (all of an
// arena's, when the sizes before them are multiples of eight), a granule is
// written as 8, 16 or 32 bytes; else, and at a tensor's ends, element by element,
// neighbours by neighbouring lanes (3.35e8 elements one element off: bf16 to bf16 297 us
// instead of 191, bf16 to fp32 360 instead of 286, fp32 to fp32 435 instead of 382).
template <typename T, typename U>
__device__ __forceinline__ void gc_scale(const void* p, void* out, int64_t n, uint32_t tile, float c) {
  using G = Granules<T>;
  constexpr int E = G::E;
  const int skip = (int)((uintptr_t)p & 15u) / (int)sizeof(T);
  U* const to = static_cast<U*>(out);
  if (((uintptr_t)(to - skip) & (E * sizeof(U) - 1)) == 0u) {
    const G g(p, n, tile);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (g.e[i] >= n) break;
      float v[E];
      g.values(i, v);
      alignas(32) U r[E];
#pragma unroll
      for (int e = 0; e < E; e += 2) put2(v + e, mul2(get2(v + e), f2(c))), r[e] = from_f32<U>(v[e]), r[e + 1] = from_f32<U>(v[e + 1]);
      const uint32_t* const w = reinterpret_cast<const uint32_t*>(r);
      if (!g.whole(i, n)) {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (g.e[i] + e >= 0 && g.e[i] + e < n) to[g.e[i] + e] = r[e];
      } else if constexpr (E * sizeof(U) == 32) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to + g.e[i]), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
      } else if constexpr (E * sizeof(U) == 16) {
        *reinterpret_cast<uint4*>(to + g.e[i]) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        *reinterpret_cast<uint2*>(to + g.e[i]) = make_uint2(w[0], w[1]);
      }
    }
  } else {
    const T* const from = static_cast<const T*>(p);
    const int64_t e0 = max((int64_t)tile * GN_TILE * E - skip, (int64_t)0), e1 = min((int64_t)(tile + 1) * GN_TILE * E - skip, n);
    for (int64_t e = e0 + threadIdx.x; e < e1; e += 256 * 8) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = e + 256 * j < e1 ? to_f32(from[e + 256 * j]) : 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (e + 256 * j < e1) to[e + 256 * j] = from_f32<U>(__fmul_rn(c, v[j]));
    }
  }
}
template <typename T>
__device__ __forceinline__ void gc_scale_to(const void* p, void* out, int otype, int64_t n, uint32_t tile, uint32_t stop, uint32_t first,
                                            float c) {
  if (otype == GC_F32)
    for (; tile < stop; ++tile) gc_scale<T, float>(p, out, n, tile - first, c);
  else if (otype == GC_BF16)
    for (; tile < stop; ++tile) gc_scale<T, __nv_bfloat16>(p, out, n, tile - first, c);
  else
    for (; tile < stop; ++tile) gc_scale<T, __half>(p, out, n, tile - first, c);
}

template <int CAP>
__global__ void __launch_bounds__(256, 3) k_grad_clip(const __grid_constant__ GcTable<CAP> g, const float* norm, float max_norm) {
  chain_wait();
  const GnTable<CAP>& t = g.t;
  const float total = *norm, c = total > max_norm ? __fdiv_rn(max_norm, total) : 1.0f;
  const uint32_t tiles = t.first[t.count];
  const uint32_t begin = (uint32_t)((uint64_t)tiles * blockIdx.x / gridDim.x), end = (uint32_t)((uint64_t)tiles * (blockIdx.x + 1) / gridDim.x);
  int i = begin < end ? gn_tensor(t, begin) : 0;
  for (uint32_t tile = begin; tile < end; ++i) {
    const uint32_t first = t.first[i], stop = min(t.first[i + 1], end);
    const void* const p = t.in[i];
    void* const out = g.out[i];
    const int type = t.type[i];
    if (c == 1.0f && out == p)
      ;  // in place, as it is
    else if (type == GC_F32)
      gc_scale_to<float>(p, out, g.otype[i], t.n[i], tile, stop, first, c);
    else if (type == GC_BF16)
      gc_scale_to<__nv_bfloat16>(p, out, g.otype[i], t.n[i], tile, stop, first, c);
    else
      gc_scale_to<__half>(p, out, g.otype[i], t.n[i], tile, stop, first, c);
    tile = stop;
  }
}

// The checks of a list of tensors.  So many elements are at most 2^30 tiles,
// and one more for each tensor.
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
    const uint64_t granules = (((uintptr_t)in[at].data & 15u) + (uint64_t)in[at].numel * dtype_bytes(in[at].dtype) + 15) / 16;
    tiles += (granules + GN_TILE - 1) / GN_TILE, ++t->count;
  }
  t->first[t->count] = (uint32_t)tiles;
  return at;
}

template <int CAP>
static int32_t launch_norm(const gc_tensor* in, int32_t at, int32_t count, double* part, int* parts, cudaStream_t s) {
  GnTable<CAP> t;
  int32_t from[CAP];
  at = fill_table(&t, in, at, count, from);
  if (t.count == 0) return at;
  const uint32_t tiles = t.first[t.count];
  const unsigned grid = tiles < (uint32_t)GN_CTAS ? tiles : (unsigned)GN_CTAS;
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
  const uint32_t tiles = g.t.first[g.t.count];
  launch_chained(&k_grad_clip<CAP>, tiles < (uint32_t)GC_CTAS ? tiles : (unsigned)GC_CTAS, 256, 0, s, g, norm, max_norm);
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
