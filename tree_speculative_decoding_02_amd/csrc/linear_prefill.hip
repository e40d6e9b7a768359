// linear_prefill.hip - prompts through linear attention with a decay.
#include "linear_device.h"
#include "launch.h"

namespace bole {

static DeltaShape shape(const bole_linear_dims_t &d) {
    return {d.batch, d.heads, d.key_heads, d.d_k, d.d_v, d.total_tokens};
}

size_t linear_prefill_workspace(const bole_linear_dims_t &d) {
    (void)d;
    return 0;
}

hipError_t launch_linear_prefill(float *H0, const void *q, const void *k, const void *v,
                                 const float *gate, const int32_t *seq_offsets, void *out,
                                 void *workspace, const bole_linear_dims_t &d, int32_t *seq_status,
                                 hipStream_t stream) {
    (void)workspace;
    const LinearArgs a = {H0, q, k, v, gate, seq_offsets, out, seq_status, shape(d)};
    return launch_linear_walk(a, d, true, stream);
}

hipError_t launch_linear_step(float *H0, const void *q, const void *k, const void *v,
                              const float *gate, void *out, const bole_linear_dims_t &d,
                              hipStream_t stream) {
    const LinearArgs a = {H0, q, k, v, gate, nullptr, out, nullptr, shape(d)};
    return launch_linear_walk(a, d, false, stream);
}

}  // namespace bole
