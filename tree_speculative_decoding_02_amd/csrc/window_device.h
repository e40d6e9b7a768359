// window_device.h - what the windowed attention kernels share: shapes, sequence lookup, the
// visible part of the cache and its validation.
#pragma once

#include "delta_device.h"

namespace bole {

struct WindowShape {
    int B, H, HK, D, T;                        // sequences, query heads, key heads, width, rows
    int pages, page_shift, max_pages;          // cache
    int window, sinks;
    float scale;
};

struct WindowArgs {
    const void *q, *k, *v, *k_cache, *v_cache;
    const int32_t *page_table, *cache_len, *parent, *offsets;
    void *out;
    int32_t *status;
    WindowShape s;
};

// The matrix-core kernels (window_mfma.hip).
bool window_mfma_applies(const bole_window_dims_t &d, const WindowArgs &a);
hipError_t launch_window_mfma(const WindowArgs &a, const bole_window_dims_t &d, void *workspace,
                              hipStream_t stream);

// The last sequence whose first row is at or before `row` (ordered offsets): the one that
// owns the row, if any does. B >= 1.
__device__ __forceinline__ int sequence_of(const int32_t *__restrict__ off, int B, int row) {
    int lo = 0, hi = B;  // off[lo] <= row or lo == 0; off[hi] > row or hi == B
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= row) lo = mid; else hi = mid;
    }
    return lo;
}

// Whether the sequence's cache can hold len tokens.
__device__ __forceinline__ int length_status(const WindowShape &s, int len) {
    return len < 0 || len > ((int64_t)s.max_pages << s.page_shift) ? BOLE_TREE_BAD_CACHE : BOLE_TREE_OK;
}

// Whether the pages that the sequence's rows see exist: those of the first min(sinks, len)
// positions and of the ones behind the first row's window. One wavefront; a valid length.
__device__ __forceinline__ int pages_status(const WindowArgs &a, int b, int len) {
    const WindowShape &s = a.s;
    const int32_t *table = a.page_table + (size_t)b * s.max_pages;
    const int from = max(0, len - s.window + 1), round = (1 << s.page_shift) - 1;
    const int sink_end = (int)(((int64_t)min(s.sinks, len) + round) >> s.page_shift);
    const int first = from >> s.page_shift;
    const int end = len == from ? first : (int)(((int64_t)len + round) >> s.page_shift);
    bool bad = false;
    for (int i = lane_id(); i < sink_end; i += 64) bad |= (unsigned)table[i] >= (unsigned)s.pages;
    for (int i = first + lane_id(); i < end; i += 64) bad |= (unsigned)table[i] >= (unsigned)s.pages;
    return __any(bad) ? BOLE_TREE_BAD_CACHE : BOLE_TREE_OK;
}

}  // namespace bole
