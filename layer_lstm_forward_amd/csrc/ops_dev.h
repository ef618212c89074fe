// ops_dev.h -- device helpers of the operators of include/lstm_ops.h.
#pragma once

#include "device.h"

namespace lstm_amd {

// v in the storage type, to nearest even; infinities and NaN stay what they are.
template <class DT>
__device__ inline typename DT::S round_to(float v) {
    if constexpr (sizeof(typename DT::S) == 2)
        return __builtin_bit_cast(uint16_t, (__bf16)v);
    else
        return v;
}

}  // namespace lstm_amd
