// Host-side helpers of libgc: argument validation and workspace sizing.
#pragma once

#include <nvtx3/nvToolsExt.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "../../include/gc.h"

namespace gc {

// Names the enclosing host scope (an entry point, or the enqueueing of one
// phase of it) in profiler timelines: an NVTX range, which costs nothing
// when no profiler is attached.
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

// A positive number that a kernel's launches need of the GPU that they go to,
// found out once on each: that one was asked says nothing about another, and a
// failure (0) is not remembered.  Zero-initialised statics only.
class PerDevice {
 public:
  template <typename F>
  int get(int device, F&& find) {
    if (device < 0 || device >= DEVICES) return find();
    int n = known_[device].load(std::memory_order_acquire);
    if (n == 0 && (n = find()) != 0) known_[device].store(n, std::memory_order_release);
    return n;
  }

 private:
  static constexpr int DEVICES = 64;
  std::atomic<int> known_[DEVICES];
};

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0u; }

// Checks a host layout: T >= 1, off[0] >= 0, 1 <= n_t < 2^31; with
// `sparse`, also 0 <= k_t <= n_t, koff[0] >= 0 and koff[t+1] - koff[t] = k_t.
// off[0] > 0 or koff[0] > 0: the layout is a bucket, a contiguous range of
// tensors of a larger arena, addressed with that arena's element and entry
// offsets.
inline gc_status validate_layout(const gc_layout* h, bool sparse) {
  if (!h || h->num_tensors < 1 || !h->off) return GC_ERR_INVALID_ARG;
  if (sparse && (!h->k || !h->koff)) return GC_ERR_INVALID_ARG;
  if (h->off[0] < 0) return GC_ERR_LAYOUT;
  if (sparse && h->koff[0] < 0) return GC_ERR_LAYOUT;
  for (int t = 0; t < h->num_tensors; ++t) {
    const int64_t n = h->off[t + 1] - h->off[t];
    if (n < 1 || n > INT64_C(2147483647)) return GC_ERR_LAYOUT;
    if (sparse) {
      const int64_t k = h->k[t];
      if (k < 0 || k > n) return GC_ERR_LAYOUT;
      if (h->koff[t + 1] - h->koff[t] != k) return GC_ERR_LAYOUT;
    }
  }
  return GC_OK;
}

// Matrix and checkpoint arguments of the activation entry points.
inline bool valid_dtype(int32_t d) { return d == GC_F32 || d == GC_BF16 || d == GC_F16; }
inline size_t dtype_bytes(int32_t d) { return d == GC_F32 ? 4 : 2; }
inline gc_status validate_matrix(int64_t rows, int64_t cols, int32_t dtype) {
  if (rows < 0 || cols < 1 || rows > INT64_C(2147483647) || cols > INT64_C(2147483647)) return GC_ERR_LAYOUT;
  return valid_dtype(dtype) ? GC_OK : GC_ERR_INVALID_ARG;
}
inline gc_status check_matrix(const void* p, int64_t ld, int64_t cols, int32_t dtype) {
  if (!p) return GC_ERR_INVALID_ARG;
  if (ld < cols) return GC_ERR_LAYOUT;
  return ((uintptr_t)p & (dtype_bytes(dtype) - 1)) ? GC_ERR_ALIGNMENT : GC_OK;
}
// A vector that may be missing.
inline gc_status check_vector(const void* p, int32_t dtype) {
  return ((uintptr_t)p & (dtype_bytes(dtype) - 1)) ? GC_ERR_ALIGNMENT : GC_OK;
}
// 16-bit rows that start on 16-byte boundaries.
inline bool chunk_aligned(const void* p, int64_t ld, int32_t dtype) {
  return dtype != GC_F32 && aligned16(p) && ld % 8 == 0;
}
inline gc_status check_codes(const int8_t* codes, const uint8_t* steps) {
  if (!codes || !steps) return GC_ERR_INVALID_ARG;
  return aligned16(codes) ? GC_OK : GC_ERR_ALIGNMENT;
}
inline gc_status check_workspace(const void* ws, size_t have, size_t need) {
  return need > 0 && (!ws || have < need || ((uintptr_t)ws & 255u)) ? GC_ERR_WORKSPACE : GC_OK;
}

// Defined by the operation files.
size_t topk_workspace_bytes(const gc_layout* h, bool sampled);
size_t dense_workspace_bytes(const gc_layout* h);
size_t sparse_decompress_workspace_bytes(const gc_layout* h);

}  // namespace gc
