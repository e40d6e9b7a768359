// window_api.hip - the windowed attention's part of the C ABI (include/bole.h): host-side
// argument checks. No allocation, no synchronisation.
#include <hip/hip_runtime.h>

#include <cmath>

#include "bole.h"
#include "launch.h"

extern "C" {

bole_status_t bole_window_check_dims(const bole_window_dims_t *d) {
    if (d == nullptr) return BOLE_ERR_INVALID_VALUE;
    if (d->batch < 0 || d->heads < 1 || d->kv_heads < 1 || d->heads % d->kv_heads != 0 ||
        d->head_dim < 1 || d->total_rows < 0 || d->num_pages < 0 || d->max_pages < 0 ||
        d->window < 1 || d->sinks < 0 || !std::isfinite(2.f * d->scale))  // (so is its product with log2 e)
        return BOLE_ERR_INVALID_VALUE;
    if (d->page_size < 1 || (d->page_size & (d->page_size - 1)) != 0) return BOLE_ERR_INVALID_VALUE;
    if (d->dtype != BOLE_DTYPE_BF16 && d->dtype != BOLE_DTYPE_F32) return BOLE_ERR_INVALID_VALUE;
    if (d->flags & ~BOLE_FLAG_FORCE_GENERIC) return BOLE_ERR_INVALID_VALUE;
    if (d->head_dim > 256 || d->page_size > 1024 || d->heads > 65535) return BOLE_ERR_UNSUPPORTED;
    // Positions, those of the next few key tiles behind the last among them, and (sequences +
    // rows) x heads fit 31 bits, and a launch has fewer than 2^32 threads: 64 a row, or 256 for
    // each 64 rows a key head packs and up to three times a sequence (of few rows).
    const int64_t rows = d->total_rows, batch = d->batch;
    if ((int64_t)d->max_pages * d->page_size + rows > (1LL << 31) - 1024 ||
        (rows + batch) * d->heads > 0x7fffffffLL || rows >= 1LL << 26 ||
        rows * d->heads / 64 + 3 * batch * d->kv_heads >= 1LL << 24)
        return BOLE_ERR_UNSUPPORTED;
    return BOLE_OK;
}

size_t bole_window_workspace_size(const bole_window_dims_t *dims) {
    if (bole_window_check_dims(dims) != BOLE_OK) return 0;
    return bole::window_workspace(*dims);
}

bole_status_t bole_window_attention(const void *q, const void *k, const void *v,
                                    const void *k_cache, const void *v_cache,
                                    const int32_t *page_table, const int32_t *cache_len,
                                    const int32_t *parent, const int32_t *node_offsets, void *out,
                                    void *workspace, size_t workspace_bytes,
                                    const bole_window_dims_t *dims, int32_t *seq_status,
                                    bole_stream_t stream) {
    const bole_status_t st = bole_window_check_dims(dims);
    if (st != BOLE_OK) return st;
    const bole_window_dims_t &d = *dims;
    if (d.batch == 0) return BOLE_OK;
    if (cache_len == nullptr || node_offsets == nullptr) return BOLE_ERR_INVALID_VALUE;
    if (d.total_rows > 0 && (q == nullptr || k == nullptr || v == nullptr || out == nullptr))
        return BOLE_ERR_INVALID_VALUE;
    if (d.max_pages > 0 && page_table == nullptr) return BOLE_ERR_INVALID_VALUE;
    if (d.num_pages > 0 && (k_cache == nullptr || v_cache == nullptr)) return BOLE_ERR_INVALID_VALUE;
    const size_t need = bole::window_workspace(d);
    if (need > 0 && (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 16 != 0 ||
                     workspace_bytes < need))
        return BOLE_ERR_INVALID_VALUE;
    const hipError_t e = bole::launch_window(q, k, v, k_cache, v_cache, page_table, cache_len, parent,
                                             node_offsets, out, workspace, d, seq_status,
                                             reinterpret_cast<hipStream_t>(stream));
    return e == hipSuccess ? BOLE_OK : BOLE_ERR_HIP;
}

}  // extern "C"
