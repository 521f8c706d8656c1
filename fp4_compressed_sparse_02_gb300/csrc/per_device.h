// What belongs to one GPU and is set or looked up once: a kernel's shared-memory limit, how many of its CTAs run at
// once.  A process may use several GPUs, and calls come from any thread.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <mutex>

namespace csa2 {

constexpr int kMaxDevices = 64;

// One T for each device.
template <typename T>
class PerDevice {
 public:
  // *value: the current device's T, which make(T&) -> cudaError_t fills on the device's first call.
  template <typename F>
  cudaError_t get(const T** value, F&& make) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!ready_[dev].load(std::memory_order_acquire)) {
      std::lock_guard<std::mutex> lock(mu_);
      if (!ready_[dev].load(std::memory_order_relaxed)) {
        e = make(value_[dev]);
        if (e != cudaSuccess) return e;
        ready_[dev].store(true, std::memory_order_release);
      }
    }
    *value = &value_[dev];
    return cudaSuccess;
  }

 private:
  std::mutex mu_;
  std::atomic<bool> ready_[kMaxDevices] = {};
  T value_[kMaxDevices] = {};
};

// The dynamic shared memory that one kernel may use on each device (48 KB until it is raised).
class SmemLimit {
 public:
  template <typename K>
  cudaError_t raise(K* kernel, size_t bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (bytes <= bytes_[dev].load(std::memory_order_acquire)) return cudaSuccess;
    std::lock_guard<std::mutex> lock(mu_);
    if (bytes <= bytes_[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) bytes_[dev].store(bytes, std::memory_order_release);
    return e;
  }

 private:
  std::mutex mu_;
  std::atomic<size_t> bytes_[kMaxDevices] = {};
};

// Streaming multiprocessors of the current device.
inline cudaError_t sm_count(int* sms) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  return e != cudaSuccess ? e : cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}

}  // namespace csa2
