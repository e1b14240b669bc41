// The device error word of one translation unit (kernels set bits in it
// instead of trapping), with its address and a read-and-clear, and the SM
// count of the current device.  TILE_DEVICE_STATUS(name) defines g_status,
// status_address() and the function status_<name>().
#pragma once

#include <cuda_runtime.h>

#include <atomic>

#include "launch.h"

namespace tile {

inline int sm_count_of_device() {
    static std::atomic<int> cache[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
    int v = cache[dev].load(std::memory_order_relaxed);
    if (v == 0) {
        if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        cache[dev].store(v, std::memory_order_relaxed);
    }
    return v;
}

}  // namespace tile

#define TILE_DEVICE_STATUS(name)                                                              \
    namespace tile {                                                                          \
    namespace {                                                                               \
    __device__ unsigned int g_status;                                                         \
    unsigned int *status_address(cudaError_t *err) {                                          \
        static std::atomic<unsigned int *> cache[kMaxDevices];                                \
        int dev = 0;                                                                          \
        *err = cudaGetDevice(&dev);                                                           \
        if (*err != cudaSuccess) return nullptr;                                              \
        if (dev < 0 || dev >= kMaxDevices) {                                                  \
            *err = cudaErrorInvalidDevice;                                                    \
            return nullptr;                                                                   \
        }                                                                                     \
        unsigned int *p = cache[dev].load(std::memory_order_acquire);                         \
        if (p == nullptr) {                                                                   \
            *err = cudaGetSymbolAddress(reinterpret_cast<void **>(&p), g_status);             \
            if (*err != cudaSuccess) return nullptr;                                          \
            cache[dev].store(p, std::memory_order_release);                                   \
        }                                                                                     \
        return p;                                                                             \
    }                                                                                         \
    }                                                                                         \
    cudaError_t status_##name(unsigned int *value, cudaStream_t stream) {                     \
        cudaError_t err = cudaMemcpyFromSymbolAsync(value, g_status, sizeof(unsigned int), 0, \
                                                    cudaMemcpyDeviceToHost, stream);          \
        if (err == cudaSuccess) err = cudaStreamSynchronize(stream);                          \
        if (err != cudaSuccess || *value == 0) return err;                                    \
        const unsigned int zero = 0;                                                          \
        err = cudaMemcpyToSymbolAsync(g_status, &zero, sizeof(unsigned int), 0,               \
                                      cudaMemcpyHostToDevice, stream);                        \
        return err == cudaSuccess ? cudaStreamSynchronize(stream) : err;                      \
    }                                                                                         \
    }
