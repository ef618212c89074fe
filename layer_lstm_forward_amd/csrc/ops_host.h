// ops_host.h -- host-side checks and workspace sums of the operators' C entry points.
#pragma once

#include <cstddef>
#include <cstdint>

#include "../../include/lstm_ops.h"
#include "host.h"

namespace lstm_amd {

inline size_t elem(int dtype) { return dtype == LSTM_BF16 ? 2 : 4; }

constexpr size_t kAlign = 256;  // of a part of a workspace

// acc += a * b * c * d bytes, 256-byte aligned; false on overflow.
inline bool add_bytes(size_t *acc, size_t a, size_t b, size_t c, size_t d) {
    size_t n;
    if (__builtin_mul_overflow(a, b, &n) || __builtin_mul_overflow(n, c, &n) || __builtin_mul_overflow(n, d, &n))
        return false;
    if (n > SIZE_MAX / 4 - *acc) return false;
    *acc += (n + kAlign - 1) / kAlign * kAlign;
    return true;
}

inline lstm_status current_device(int *dev) {
    if (hipGetDevice(dev) == hipSuccess) return LSTM_OK;
    (void)hipGetLastError();
    return LSTM_ERR_DEVICE;
}

inline lstm_status launched(hipError_t e) {
    if (e == hipSuccess) return LSTM_OK;
    (void)hipGetLastError();
    return LSTM_ERR_LAUNCH;
}

inline bool view_ok(const lstm_view *v) { return v && v->data; }

// Every pointer of the list that is given lies on the device.
inline bool all_on_device(const void *const *p, int n, int dev) {
    for (int i = 0; i < n; ++i)
        if (p[i] && !is_device_ptr(p[i], dev)) return false;
    return true;
}

}  // namespace lstm_amd
