// linear_api.hip - linear attention's part of the C ABI (include/bole.h): host-side argument
// checks and kernel selection. No allocation, no synchronisation.
#include <hip/hip_runtime.h>

#include "bole.h"
#include "launch.h"

namespace {

enum { kOpPrefill = 0, kOpStep = 1 };

bole_status_t from_hip(hipError_t e) { return e == hipSuccess ? BOLE_OK : BOLE_ERR_HIP; }

}  // namespace

extern "C" {

bole_status_t bole_linear_check_dims(const bole_linear_dims_t *d, int32_t op) {
    if (d == nullptr || op < kOpPrefill || op > kOpStep) return BOLE_ERR_INVALID_VALUE;
    if (d->batch < 0 || d->heads < 1 || d->key_heads < 1 || d->d_k < 1 || d->d_v < 1 ||
        d->total_tokens < 0 || d->heads % d->key_heads != 0)
        return BOLE_ERR_INVALID_VALUE;
    if (d->factor_dtype != BOLE_DTYPE_BF16 && d->factor_dtype != BOLE_DTYPE_F32)
        return BOLE_ERR_INVALID_VALUE;
    if (d->gate_kind != BOLE_GATE_SCALAR && d->gate_kind != BOLE_GATE_VECTOR)
        return BOLE_ERR_INVALID_VALUE;
    if (d->flags & ~BOLE_FLAG_FORCE_GENERIC) return BOLE_ERR_INVALID_VALUE;
    if (op == kOpStep && d->total_tokens != d->batch) return BOLE_ERR_INVALID_VALUE;
    if (d->d_k > 256 || d->d_v > 256) return BOLE_ERR_UNSUPPORTED;
    // A launch has fewer than 2^32 threads: of a state, 64 for each 8 of its columns and 256 or
    // more; of a prompt's 64 tokens and value head, 256 for each 64 columns.
    const int64_t units = (int64_t)d->batch * d->heads, most = 1LL << 32;
    const int64_t each = d->d_v <= 32 ? 256 : (d->d_v + 7) / 8 * 64;
    const int64_t chunks = op == kOpPrefill ? ((int64_t)d->total_tokens / 64 + d->batch) * d->heads : 0;
    if (units + 8 > most / each || chunks >= most / (256 * ((d->d_v + 63) / 64))) return BOLE_ERR_UNSUPPORTED;
    return BOLE_OK;
}

size_t bole_linear_prefill_workspace_size(const bole_linear_dims_t *dims) {
    if (bole_linear_check_dims(dims, kOpPrefill) != BOLE_OK) return 0;
    return bole::linear_prefill_workspace(*dims);
}

bole_status_t bole_linear_prefill(float *H0, const void *q, const void *k, const void *v,
                                  const float *gate, const int32_t *seq_offsets, void *out,
                                  void *workspace, size_t workspace_bytes,
                                  const bole_linear_dims_t *dims, int32_t *seq_status,
                                  bole_stream_t stream) {
    const bole_status_t st = bole_linear_check_dims(dims, kOpPrefill);
    if (st != BOLE_OK) return st;
    const bole_linear_dims_t &d = *dims;
    if (d.batch == 0) return BOLE_OK;
    if (H0 == nullptr || seq_offsets == nullptr) return BOLE_ERR_INVALID_VALUE;
    if (d.total_tokens > 0 &&
        (q == nullptr || k == nullptr || v == nullptr || gate == nullptr || out == nullptr))
        return BOLE_ERR_INVALID_VALUE;
    const size_t need = bole::linear_prefill_workspace(d);
    if (need > 0 && (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 16 != 0 ||
                     workspace_bytes < need))
        return BOLE_ERR_INVALID_VALUE;
    return from_hip(bole::launch_linear_prefill(H0, q, k, v, gate, seq_offsets, out, workspace, d,
                                                seq_status, reinterpret_cast<hipStream_t>(stream)));
}

bole_status_t bole_linear_step(float *H0, const void *q, const void *k, const void *v,
                               const float *gate, void *out, const bole_linear_dims_t *dims,
                               bole_stream_t stream) {
    const bole_status_t st = bole_linear_check_dims(dims, kOpStep);
    if (st != BOLE_OK) return st;
    const bole_linear_dims_t &d = *dims;
    if (d.batch == 0) return BOLE_OK;
    if (H0 == nullptr || q == nullptr || k == nullptr || v == nullptr || gate == nullptr ||
        out == nullptr)
        return BOLE_ERR_INVALID_VALUE;
    return from_hip(bole::launch_linear_step(H0, q, k, v, gate, out, d,
                                             reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
