// The runtime calls that libgc's activation entry points make, for two GPUs
// that are not there: launches do nothing but check that their kernel was
// granted the shared memory it asks for on the GPU that is current.
#include <cuda_runtime_api.h>

#include <map>
#include <utility>

static int device = 0, failing = 0, pending = 0, regs = 96;
static unsigned grid_y = 0;
static std::map<std::pair<const void*, int>, int> granted;

extern "C" {
void fake_device(int d) { device = d; }
void fake_failing(int f) { failing = f; }
unsigned fake_grid_y() { return grid_y; }

cudaError_t cudaGetDevice(int* d) {
  *d = device;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute a, int v) {
  if (failing) return pending = 1, cudaErrorInvalidValue;
  if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) granted[{f, device}] = v;
  return cudaSuccess;
}
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void*) {
  if (failing) return pending = 1, cudaErrorInvalidValue;
  *a = cudaFuncAttributes();
  a->numRegs = regs;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void*, int, size_t, unsigned) {
  if (failing) return pending = 1, cudaErrorInvalidValue;
  *n = device == 0 ? 2 : 5;
  return cudaSuccess;
}
static int encode(...) { return 0; }
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** f, unsigned, unsigned long long, cudaDriverEntryPointQueryResult* q) {
  if (failing) return pending = 1, cudaErrorInvalidValue;
  *f = reinterpret_cast<void*>(&encode), *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
  const auto it = granted.find({f, device});
  if (c->dynamicSmemBytes > 48 * 1024 && (it == granted.end() || (size_t)it->second < c->dynamicSmemBytes))
    return pending = 2, cudaErrorInvalidValue;  // the plain launch that follows is refused, too
  grid_y = c->gridDim.y;
  return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void**, size_t, cudaStream_t) { return cudaErrorInvalidValue; }
cudaError_t cudaLaunchKernel(const void*, dim3, dim3, void**, size_t, cudaStream_t) { return cudaErrorInvalidValue; }
cudaError_t cudaGetLastError() { return pending > 0 ? --pending, cudaErrorInvalidValue : cudaSuccess; }
}
