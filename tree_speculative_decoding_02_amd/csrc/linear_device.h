// linear_device.h - linear attention with a decay: shapes and arguments of its kernels.
#pragma once

#include "delta_device.h"

namespace bole {

struct LinearArgs {
    float *H0;
    const void *q, *k, *v;
    const float *gate;
    const int32_t *offsets;  // of prompts
    void *out;
    int32_t *status;
    DeltaShape s;
};

// Every token in turn, any shape and gate (linear_walk.hip).
hipError_t launch_linear_walk(const LinearArgs &a, const bole_linear_dims_t &d, bool prompts,
                              hipStream_t stream);

}  // namespace bole
