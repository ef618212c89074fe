// host.h -- host-side checks shared by the C entry points.
#pragma once

#include <hip/hip_runtime.h>

#include <cstring>

namespace lstm_amd {

// ptr is device (or managed) memory of device dev.
inline bool is_device_ptr(const void *ptr, int dev) {
    hipPointerAttribute_t attr;
    std::memset(&attr, 0, sizeof(attr));
    if (hipPointerGetAttributes(&attr, ptr) != hipSuccess) {
        (void)hipGetLastError();
        return false;
    }
    const bool dev_mem = attr.type == hipMemoryTypeDevice || attr.type == hipMemoryTypeManaged;
    return dev_mem && attr.device == dev;
}

}  // namespace lstm_amd
