// runtime.cpp -- the CUDA runtime calls that the library's host code makes,
// without a GPU, for tests of that code: four devices, each with its own
// shared-memory limits per kernel, launches that are checked against them and
// recorded, and launches that fail when told to.
#include <cuda_runtime_api.h>

#include <map>
#include <utility>

#include "internal.h"

namespace {
int device, failures, bad_launch, launches, attribute_calls;  // bad_launch: 1 is the next one
cudaError_t last_error;
std::map<std::pair<int, const void*>, int> limits;
int last_grid, last_smem, last_stages;

cudaError_t note(cudaError_t e) {
  if (e != cudaSuccess) last_error = e;
  return e;
}

CUresult encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
  return CUDA_SUCCESS;
}
}  // namespace

extern "C" {

// ---- what a test sets and reads
void fake_set_device(int d) { device = d; }
void fake_fail_calls(int n) { failures = n; }  // the next n attribute and launch calls
void fake_fail_launch(int n) { bad_launch = n + 1; }  // the n-th launch from now, 0 the next
int fake_launches() { return launches; }
int fake_attribute_calls() { return attribute_calls; }
int fake_last_grid() { return last_grid; }
int fake_last_stages() { return last_stages; }

// ---- the runtime
cudaError_t cudaGetDevice(int* d) {
  *d = device;
  return cudaSuccess;
}
cudaError_t cudaGetLastError() {
  const cudaError_t e = last_error;
  last_error = cudaSuccess;
  return e;
}
cudaError_t cudaPeekAtLastError() { return last_error; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
  *v = a == cudaDevAttrComputeCapabilityMajor   ? 10
       : a == cudaDevAttrComputeCapabilityMinor ? 3
       : a == cudaDevAttrMultiProcessorCount    ? 152
                                                : 0;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute, int v) {
  ++attribute_calls;
  if (failures > 0) return --failures, note(cudaErrorUnknown);
  limits[{device, f}] = v;
  return cudaSuccess;
}
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void*) {
  *a = cudaFuncAttributes{};
  a->numRegs = 168;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t* c) {
  *n = 152 / c->attrs[0].val.clusterDim.x;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void** args) {
  if (failures > 0) return --failures, note(cudaErrorUnknown);
  if (bad_launch > 0 && --bad_launch == 0) return note(cudaErrorUnknown);
  // 48 KB in all without the attribute; a kernel's static part is not known here: 2 KB
  const auto l = limits.find({device, f});
  const size_t limit = l == limits.end() ? 46 << 10 : l->second;
  if (c->dynamicSmemBytes > limit) return note(cudaErrorInvalidValue);
  ++launches;
  last_grid = c->gridDim.x;
  // (of a product: its second argument)
  if (c->dynamicSmemBytes > (100 << 10))
    last_stages = static_cast<const moe::BlockscaleArgs*>(args[1])->stages;
  return cudaSuccess;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** p, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
  *p = reinterpret_cast<void*>(&encode);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
void** __cudaRegisterFatBinary(void*) {
  static void* handle;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, void*, void*, void*,
                            void*, int*) {}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}

}  // extern "C"
