// The CUDA runtime as the library's host side sees it, without a GPU: two devices of different sizes, and a record of
// what was launched on which.  A launch fails as the runtime's would where a kernel asks for more shared memory than it
// was allowed on that device.
#include <cuda.h>
#include <cuda_runtime.h>
#include <unistd.h>

#include <map>
#include <mutex>
#include <string>
#include <utility>
#include <vector>

namespace {
struct Launch {
  int dev, kernel, smem, cluster;
  unsigned gx, gy, gz, block;
};
std::mutex mu;
std::map<const void*, int> kernels;
std::map<std::pair<int, const void*>, int> limits;
std::vector<Launch> launches;
thread_local int current = 0;
const int kSms[2] = {152, 40};

CUresult encode(...) { return CUDA_SUCCESS; }
}  // namespace

extern "C" {
void fake_set_device(int d) { current = d; }
int fake_launches(int* out, int most) {   // eight numbers each; forgets them
  std::lock_guard<std::mutex> lock(mu);
  int n = 0;
  for (const Launch& l : launches)
    if (n < most) {
      const int v[8] = {l.dev, l.kernel, l.smem, l.cluster, (int)l.gx, (int)l.gy, (int)l.gz, (int)l.block};
      for (int i = 0; i < 8; ++i) out[8 * n + i] = v[i];
      ++n;
    }
  launches.clear();
  return n;
}

void** __cudaRegisterFatBinary(void*) {
  static void* handle;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char* stub, char*, const char*, int, uint3*, uint3*, dim3*, dim3*, int*) {
  std::lock_guard<std::mutex> lock(mu);
  const int n = (int)kernels.size();
  kernels.emplace(stub, n);
}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
cudaError_t __cudaPopCallConfiguration(dim3*, dim3*, size_t*, void*) { return cudaErrorNotSupported; }
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void**, size_t, cudaStream_t) { return cudaErrorNotSupported; }
cudaError_t __cudaGetKernel(cudaKernel_t*, const void*) { return cudaErrorNotSupported; }

cudaError_t cudaGetDevice(int* d) {
  *d = current;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int dev) {
  *v = kSms[dev];
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute, int v) {
  std::lock_guard<std::mutex> lock(mu);
  limits[{current, f}] = v;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void*, int threads, size_t, unsigned) {
  usleep(200);                            // long enough for another thread to look meanwhile
  *n = 1024 / threads > 0 ? 1024 / threads : 1;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t* c) {
  usleep(200);
  *n = kSms[current] / (int)c->attrs[0].val.clusterDim.x;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
  std::lock_guard<std::mutex> lock(mu);
  const auto limit = limits.find({current, f});
  if (c->dynamicSmemBytes > (size_t)(limit == limits.end() ? 48 * 1024 : limit->second)) return cudaErrorInvalidValue;
  int cluster = 1;
  for (unsigned i = 0; i < c->numAttrs; ++i)
    if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) cluster = (int)c->attrs[i].val.clusterDim.x;
  launches.push_back({current, kernels[f], (int)c->dynamicSmemBytes, cluster, c->gridDim.x, c->gridDim.y, c->gridDim.z,
                      c->blockDim.x * c->blockDim.y});
  return cudaSuccess;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char* name, void** fn, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
  const bool known = std::string(name) == "cuTensorMapEncodeTiled";
  *fn = known ? reinterpret_cast<void*>(&encode) : nullptr;
  if (q) *q = known ? cudaDriverEntryPointSuccess : cudaDriverEntryPointSymbolNotFound;
  return known ? cudaSuccess : cudaErrorInvalidValue;
}
cudaError_t cudaMemcpyToSymbol(const void*, const void*, size_t, size_t, cudaMemcpyKind) { return cudaSuccess; }
cudaError_t cudaMemcpyFromSymbol(void*, const void*, size_t, size_t, cudaMemcpyKind) { return cudaSuccess; }
cudaError_t cudaGetSymbolAddress(void** p, const void*) {
  *p = reinterpret_cast<void*>(0x100000);
  return cudaSuccess;
}
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaDeviceSynchronize() { return cudaSuccess; }
const char* cudaGetErrorString(cudaError_t) { return "refused by the stand-in runtime"; }
}
