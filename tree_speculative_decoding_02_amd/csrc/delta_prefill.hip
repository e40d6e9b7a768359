// delta_prefill.hip - prompts through the gated delta rule: kernel selection.
#include "delta_device.h"
#include "launch.h"

namespace bole {

size_t delta_prefill_workspace(const bole_delta_dims_t &d) {
    (void)d;
    return 0;
}

hipError_t launch_delta_prefill(float *H0, const void *q, const void *k, const void *v,
                                const float *gate, const float *beta, const int32_t *seq_offsets,
                                void *out, void *workspace, const bole_delta_dims_t &d,
                                int32_t *seq_status, hipStream_t stream) {
    (void)workspace;
    return launch_delta_prefill_walk(H0, q, k, v, gate, beta, seq_offsets, out, d, seq_status,
                                     stream);
}

}  // namespace bole
