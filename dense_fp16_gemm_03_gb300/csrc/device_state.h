// Per-device state that the translation units of the library share: the
// capability gate, the SM count and the device error word (gemm_api.cu).
#pragma once

#include <stdint.h>

#include "gemm_f16.h"

namespace gemm_f16 {

struct DeviceState {
    int num_sms;
    unsigned long long ctx_id;  // the context the addresses belong to
    uint32_t *error_word;       // device address of the error word gemm_f16_take_device_error reads
};

// State of the current device; GEMM_ERR_ARCH if it is not compute capability 10.3.
__attribute__((visibility("hidden"))) gemm_status_t current_device_state(DeviceState *out);

// A stamp unique to one launch, for flags that are set to it (never zero).
__attribute__((visibility("hidden"))) uint64_t next_launch_stamp();

}  // namespace gemm_f16
