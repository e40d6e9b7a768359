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

// Sequences cut into segments of `seg` tokens, `slots` of them (spare ones among them): sequence b owns
// slots from floor(first row / seg) + b on.
// Workspace: of each sequence of more than one segment, from slot 2 floor(first row / seg) on (a
// sequence of n > seg rows has at most 2 floor(n / seg) segments, so they do not meet).
__device__ __forceinline__ size_t space_slot(int lo, int seg, int i) { return 2 * (size_t)(lo / seg) + i; }
inline size_t space_slots(int64_t tokens, int64_t seg) { return tokens > seg ? 2 * (size_t)(tokens / seg) : 0; }

// Every token in turn, any shape and gate (linear_walk.hip).
hipError_t launch_linear_step_walk(const LinearArgs &a, const bole_linear_dims_t &d, hipStream_t stream);
size_t linear_walk_workspace(const bole_linear_dims_t &d);
hipError_t launch_linear_walk(const LinearArgs &a, const bole_linear_dims_t &d, void *workspace,
                              hipStream_t stream);

}  // namespace bole
