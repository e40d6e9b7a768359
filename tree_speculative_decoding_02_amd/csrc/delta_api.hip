// delta_api.hip - the gated delta rule's part of the C ABI (include/bole.h): host-side
// argument checks and kernel selection. No allocation, no synchronisation.
#include <hip/hip_runtime.h>

#include "bole.h"
#include "launch.h"

namespace {

enum { kOpPrefill = 0, kOpStep = 1, kOpVerify = 2, kOpCommit = 3 };

bole_status_t from_hip(hipError_t e) { return e == hipSuccess ? BOLE_OK : BOLE_ERR_HIP; }

hipStream_t stream_of(bole_stream_t s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace

extern "C" {

bole_status_t bole_delta_check_dims(const bole_delta_dims_t *d, int32_t op) {
    if (d == nullptr || op < kOpPrefill || op > kOpCommit) return BOLE_ERR_INVALID_VALUE;
    if (d->batch < 0 || d->heads < 1 || d->key_heads < 1 || d->d_k < 1 || d->d_v < 1 ||
        d->total_tokens < 0 || d->heads % d->key_heads != 0)
        return BOLE_ERR_INVALID_VALUE;
    if (d->factor_dtype != BOLE_DTYPE_BF16 && d->factor_dtype != BOLE_DTYPE_F32)
        return BOLE_ERR_INVALID_VALUE;
    if (d->flags & ~BOLE_FLAG_FORCE_GENERIC) return BOLE_ERR_INVALID_VALUE;
    if (op == kOpCommit && d->max_path < 0) return BOLE_ERR_INVALID_VALUE;
    if (op == kOpStep && d->total_tokens != d->batch) return BOLE_ERR_INVALID_VALUE;
    if (d->d_k > 256 || d->d_v > 256) return BOLE_ERR_UNSUPPORTED;
    if (op == kOpCommit && d->max_path > bole::kMaxTreeNodesHost) return BOLE_ERR_UNSUPPORTED;
    // A launch has fewer than 2^32 threads: of a state, 64 for each 8 of its columns and 256 or
    // more (prompts: 512 for each 16); of a prompt's 64 tokens and value head, 256.
    const int64_t units = (int64_t)d->batch * d->heads, most = 1LL << 32;
    const int64_t chunks = op == kOpPrefill ? ((int64_t)d->total_tokens / 64 + d->batch) * d->heads : 0;
    const int64_t each = op == kOpPrefill ? (d->d_v + 15) / 16 * 512 : d->d_v <= 32 ? 256 : (d->d_v + 7) / 8 * 64;
    if (units + 8 > most / each || chunks >= most / 256) return BOLE_ERR_UNSUPPORTED;
    return BOLE_OK;
}

size_t bole_delta_prefill_workspace_size(const bole_delta_dims_t *dims) {
    if (bole_delta_check_dims(dims, kOpPrefill) != BOLE_OK) return 0;
    return bole::delta_prefill_workspace(*dims);
}

bole_status_t bole_delta_prefill(float *H0, const void *q, const void *k, const void *v,
                                 const float *gate, const float *beta,
                                 const int32_t *seq_offsets, void *out, void *workspace,
                                 size_t workspace_bytes, const bole_delta_dims_t *dims,
                                 int32_t *seq_status, bole_stream_t stream) {
    const bole_status_t st = bole_delta_check_dims(dims, kOpPrefill);
    if (st != BOLE_OK) return st;
    const bole_delta_dims_t &d = *dims;
    if (d.batch == 0) return BOLE_OK;
    if (H0 == nullptr || seq_offsets == nullptr) return BOLE_ERR_INVALID_VALUE;
    if (d.total_tokens > 0 && (q == nullptr || k == nullptr || v == nullptr || gate == nullptr ||
                               beta == nullptr || out == nullptr))
        return BOLE_ERR_INVALID_VALUE;
    const size_t need = bole::delta_prefill_workspace(d);
    if (need > 0 && (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 16 != 0 ||
                     workspace_bytes < need))
        return BOLE_ERR_INVALID_VALUE;
    return from_hip(bole::launch_delta_prefill(H0, q, k, v, gate, beta, seq_offsets, out, workspace,
                                               d, seq_status, stream_of(stream)));
}

bole_status_t bole_delta_step(float *H0, const void *q, const void *k, const void *v,
                              const float *gate, const float *beta, void *out,
                              const bole_delta_dims_t *dims, bole_stream_t stream) {
    const bole_status_t st = bole_delta_check_dims(dims, kOpStep);
    if (st != BOLE_OK) return st;
    if (dims->batch == 0) return BOLE_OK;
    if (H0 == nullptr || q == nullptr || k == nullptr || v == nullptr || gate == nullptr ||
        beta == nullptr || out == nullptr)
        return BOLE_ERR_INVALID_VALUE;
    return from_hip(bole::launch_delta_step(H0, q, k, v, gate, beta, out, *dims, stream_of(stream)));
}

bole_status_t bole_delta_tree_verify(const float *H0, const void *q, const void *k, const void *v,
                                     const float *gate, const float *beta, const int32_t *parent,
                                     const int32_t *node_offsets, void *out,
                                     const bole_delta_dims_t *dims, int32_t *tree_status,
                                     bole_stream_t stream) {
    const bole_status_t st = bole_delta_check_dims(dims, kOpVerify);
    if (st != BOLE_OK) return st;
    const bole_delta_dims_t &d = *dims;
    if (d.batch == 0) return BOLE_OK;
    if (H0 == nullptr || node_offsets == nullptr) return BOLE_ERR_INVALID_VALUE;
    if (d.total_tokens > 0 && (q == nullptr || k == nullptr || v == nullptr || gate == nullptr ||
                               beta == nullptr || parent == nullptr || out == nullptr))
        return BOLE_ERR_INVALID_VALUE;
    return from_hip(bole::launch_delta_verify(H0, q, k, v, gate, beta, parent, node_offsets, out, d,
                                              tree_status, stream_of(stream)));
}

bole_status_t bole_delta_commit_path(float *H0, const void *k, const void *v, const float *gate,
                                     const float *beta, const int32_t *parent,
                                     const int32_t *node_offsets, const int32_t *accepted_idx,
                                     const int32_t *accepted_len, const bole_delta_dims_t *dims,
                                     int32_t *path_nodes, int32_t *tree_status,
                                     bole_stream_t stream) {
    const bole_status_t st = bole_delta_check_dims(dims, kOpCommit);
    if (st != BOLE_OK) return st;
    const bole_delta_dims_t &d = *dims;
    if (d.batch == 0) return BOLE_OK;
    if (H0 == nullptr || node_offsets == nullptr || accepted_len == nullptr)
        return BOLE_ERR_INVALID_VALUE;
    if (d.max_path > 0 && accepted_idx == nullptr) return BOLE_ERR_INVALID_VALUE;
    if (d.total_tokens > 0 && (k == nullptr || v == nullptr || gate == nullptr ||
                               beta == nullptr || parent == nullptr))
        return BOLE_ERR_INVALID_VALUE;
    return from_hip(bole::launch_delta_commit(H0, k, v, gate, beta, parent, node_offsets,
                                              accepted_idx, accepted_len, d, path_nodes,
                                              tree_status, stream_of(stream)));
}

}  // extern "C"
