// Host-side helpers shared by the files that define the C ABI: alignment,
// device information, launches, supported page sizes.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <utility>

#include "wmtp.h"

namespace wmtp {
namespace {

constexpr int kMaxDevices = 64;
constexpr size_t kWsAlign = 256;
constexpr int kMaxGridYZ = 65535;       // gridDim.y / gridDim.z limit

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// ---------------------------------------------------------------- device info
struct DeviceInfo {
  int sms = 0;
};

DeviceInfo g_dev[kMaxDevices];
std::once_flag g_dev_once[kMaxDevices];

wmtp_status current_device(int* dev, DeviceInfo* info) {
  if (cudaGetDevice(dev) != cudaSuccess || *dev < 0 || *dev >= kMaxDevices) return WMTP_ERR_CUDA;
  const int d = *dev;
  std::call_once(g_dev_once[d], [d]() {
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, d) == cudaSuccess) g_dev[d].sms = sms;
  });
  if (g_dev[d].sms <= 0) return WMTP_ERR_CUDA;
  *info = g_dev[d];
  return WMTP_OK;
}

// One attribute of one kernel, set once per device.  Only a success is
// remembered: a failed attempt (its error cleared from this library's runtime
// state) is retried by the next call.  Concurrent first calls from several host
// threads serialise on the mutex.
struct FuncAttrOnce {
  std::atomic<bool> done[kMaxDevices];
  std::mutex mu;
};

template <typename Kern>
wmtp_status ensure_func_attr(FuncAttrOnce& once, Kern kern, cudaFuncAttribute attr, int value) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return WMTP_ERR_CUDA;
  if (once.done[dev].load(std::memory_order_acquire)) return WMTP_OK;
  std::lock_guard<std::mutex> lock(once.mu);
  if (once.done[dev].load(std::memory_order_relaxed)) return WMTP_OK;
  if (cudaFuncSetAttribute(kern, attr, value) != cudaSuccess) {
    (void)cudaGetLastError();
    return WMTP_ERR_CUDA;
  }
  once.done[dev].store(true, std::memory_order_release);
  return WMTP_OK;
}

// The widest cluster of one kernel on one device.  More than 8 CTAs are not
// portable: a part of a GPU may have no place for them.  fits(): how many clusters
// of `wide` CTAs the runtime says fit at once, negative if it failed, which is not
// remembered.
constexpr int kPortableCluster = 8;
struct WidestOnce {
  std::atomic<int> most[kMaxDevices];  // 0: not asked yet
};

template <typename Fits>
int widest_cluster(WidestOnce& once, int dev, int wide, Fits fits) {
  int most = once.most[dev].load(std::memory_order_acquire);
  if (most != 0) return most;
  const int n = fits();
  most = n > 0 ? wide : kPortableCluster;
  if (n >= 0) once.most[dev].store(most, std::memory_order_release);
  return most;
}

// ---------------------------------------------------------------- launches
// A launch whose success is read from the launch call itself, never from
// cudaGetLastError (which would also report an unrelated earlier error left
// on this thread, after the kernel had been queued).  `programmatic`: launch
// as a programmatic dependent of the previous work on the stream (the kernel
// must execute griddepcontrol.wait before its first memory access).  `cluster`:
// CTAs per thread-block cluster, along x; it divides gridDim.x.
template <typename... Exp, typename... Act>
wmtp_status launch_clusters(bool programmatic, void (*kern)(Exp...), dim3 grid, dim3 block, int cluster,
                            cudaStream_t st, Act&&... args) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = 0;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (programmatic) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = n > 0 ? attr : nullptr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Act>(args)...) == cudaSuccess ? WMTP_OK : WMTP_ERR_CUDA;
}

template <typename... Exp, typename... Act>
wmtp_status launch_plain(bool programmatic, void (*kern)(Exp...), dim3 grid, dim3 block, cudaStream_t st,
                         Act&&... args) {
  return launch_clusters(programmatic, kern, grid, block, 1, st, std::forward<Act>(args)...);
}

// ---------------------------------------------------------------- shapes
bool supported_page(int p) { return p == 16 || p == 32 || p == 64 || p == 128 || p == 256; }

}  // namespace
}  // namespace wmtp
