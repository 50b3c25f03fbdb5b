// fake_cudart.cpp -- a stand-in for the CUDA runtime that libdspark.so is linked with, for tests of its host
// side without a GPU: nothing runs, launches are written down.  Devices differ in their number of SMs, and a
// function's attributes are kept for the device that was current, as the runtime keeps them: a launch that asks
// for more dynamic shared memory than its function may have on the current device is refused.
#include <cuda_runtime_api.h>

#include <cstdio>
#include <cstring>
#include <map>
#include <string>
#include <tuple>

namespace {
int device = 0;
std::map<const void*, std::string> names;
std::map<std::tuple<int, const void*, int>, int> attributes;
std::string launches;  // a line each: device, grid, bytes of dynamic shared memory, function

cudaError_t launch(const void* func, dim3 grid, size_t smem) {
  const auto a = attributes.find({device, func, (int)cudaFuncAttributeMaxDynamicSharedMemorySize});
  if (smem > (a == attributes.end() ? 49152 : (size_t)a->second)) return cudaErrorInvalidValue;
  launches += std::to_string(device) + " " + std::to_string(grid.x) + " " + std::to_string(smem) + " " + names[func] + "\n";
  return cudaSuccess;
}
int encode_map() { return 0; }
alignas(256) char symbol[256];
}  // namespace

extern "C" {
void fake_set_device(int d) { device = d; }
const char* fake_launches() { return launches.c_str(); }
void fake_clear() { launches.clear(); }

cudaError_t cudaGetDevice(int* d) { return *d = device, cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int d) {
  *v = a == cudaDevAttrMultiProcessorCount ? 152 - 20 * d : a == cudaDevAttrL2CacheSize ? 129 << 20 : 0;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* func, cudaFuncAttribute a, int v) {
  return attributes[{device, func, (int)a}] = v, cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* func, void**) {
  return launch(func, c->gridDim, c->dynamicSmemBytes);
}
cudaError_t __cudaGetKernel(cudaKernel_t* k, const void* func) { return *k = (cudaKernel_t)func, cudaSuccess; }
cudaError_t __cudaLaunchKernel(cudaKernel_t k, dim3 grid, dim3, void**, size_t smem, cudaStream_t) {
  return launch((const void*)k, grid, smem);
}
static dim3 pushed_grid, pushed_block;
static size_t pushed_smem;
static void* pushed_stream;
unsigned __cudaPushCallConfiguration(dim3 grid, dim3 block, size_t smem, void* stream) {
  pushed_grid = grid, pushed_block = block, pushed_smem = smem, pushed_stream = stream;
  return 0;
}
cudaError_t __cudaPopCallConfiguration(dim3* grid, dim3* block, size_t* smem, void* stream) {
  *grid = pushed_grid, *block = pushed_block, *smem = pushed_smem, *(void**)stream = pushed_stream;
  return cudaSuccess;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char* name, void** f, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* r) {
  const bool known = !strcmp(name, "cuTensorMapEncodeTiled");
  *f = known ? (void*)encode_map : nullptr;
  if (r) *r = known ? cudaDriverEntryPointSuccess : cudaDriverEntryPointSymbolNotFound;
  return cudaSuccess;
}
cudaError_t cudaGetSymbolAddress(void** p, const void*) { return *p = symbol, cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char* cudaGetErrorString(cudaError_t) { return "refused by the stand-in"; }
cudaError_t cudaMemcpyAsync(void*, const void*, size_t, cudaMemcpyKind, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaEventCreate(cudaEvent_t*) { return cudaSuccess; }
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaEventSynchronize(cudaEvent_t) { return cudaSuccess; }
cudaError_t cudaEventElapsedTime(float*, cudaEvent_t, cudaEvent_t) { return cudaSuccess; }

void** __cudaRegisterFatBinary(void*) {
  static void* handle;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char* func, char*, const char* name, int, uint3*, uint3*, dim3*, dim3*, int*) {
  names[func] = name;
}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
}
