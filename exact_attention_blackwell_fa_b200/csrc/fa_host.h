// fa_host.h -- host-side pieces shared by the library's translation units: the device
// check and pointer alignment.
#pragma once

#include <cstdint>
#include <mutex>

#include <cuda_runtime.h>

#include "../../include/fa.h"

namespace fa {

struct DeviceInfo {
    int sm_count = 0;
    bool ok = false;  // compute capability 10.0 (B200 class, sm_100a code runs)
};

constexpr int kMaxDevices = 64;

inline fa_status device_info(DeviceInfo* out)
{
    static DeviceInfo cache[kMaxDevices];
    static std::mutex mu;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FA_ERR_CUDA;
    std::lock_guard<std::mutex> lk(mu);
    if (cache[dev].sm_count == 0) {
        int major = 0, minor = 0, sms = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return FA_ERR_CUDA;
        cache[dev].sm_count = sms;
        cache[dev].ok = (major == 10 && minor == 0);
    }
    *out = cache[dev];
    return out->ok ? FA_OK : FA_ERR_UNSUPPORTED;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The status word of the paged-cache kernels (fa_paged.cu); fa_last_device_status and
// fa_clear_device_status cover it together with the attention kernels' own.
cudaError_t paged_status_read(uint32_t (&h)[4], cudaStream_t s);
cudaError_t paged_status_clear(cudaStream_t s);

}  // namespace fa
