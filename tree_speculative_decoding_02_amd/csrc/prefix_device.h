// prefix_device.h - arguments of attention behind shared prefixes.
#pragma once

#include "window_device.h"

namespace bole {

struct PrefixArgs {
    WindowArgs w;                    // own tokens: a window of everything, no first tokens
    const int32_t *prefix_table, *prefix_len, *group_offsets;
    int groups, max_prefix_pages;
};

// The prefix of a sequence: group g's, of len tokens; found: it has one.
struct Group {
    bool found;
    int g, len;
};

// The group of sequence b (ordered group offsets).
__device__ __forceinline__ Group group_of(const PrefixArgs &a, int b) {
    Group x = {false, 0, 0};
    if (a.groups == 0) return x;
    x.g = sequence_of(a.group_offsets, a.groups, b);
    x.found = a.group_offsets[x.g] <= b && b < a.group_offsets[x.g + 1];
    if (x.found) x.len = a.prefix_len[x.g];
    return x;
}

// Whether the pages of positions x0 .. x1 - 1 of prefix g exist. One wavefront.
__device__ __forceinline__ int prefix_pages_status(const PrefixArgs &a, int g, int x0, int x1) {
    const int shift = a.w.s.page_shift;
    const int32_t *table = a.prefix_table + (size_t)g * a.max_prefix_pages;
    bool bad = false;
    if (x0 < x1)
        for (int i = (x0 >> shift) + lane_id(); i <= (x1 - 1) >> shift; i += 64)
            bad |= (unsigned)table[i] >= (unsigned)a.w.s.pages;
    return __any(bad) ? BOLE_TREE_BAD_CACHE : BOLE_TREE_OK;
}

// Whether prefix g of len tokens lies in pages that exist. One wavefront.
__device__ __forceinline__ int prefix_status(const PrefixArgs &a, int g, int len) {
    if (len < 0 || len > ((int64_t)a.max_prefix_pages << a.w.s.page_shift)) return BOLE_TREE_BAD_CACHE;
    return prefix_pages_status(a, g, 0, len);
}

// The matrix-core kernels (prefix_mfma.hip).
bool prefix_mfma_applies(const bole_prefix_dims_t &d, const PrefixArgs &a);
hipError_t launch_prefix_mfma(const PrefixArgs &a, const bole_prefix_dims_t &d, void *workspace,
                              hipStream_t stream);

}  // namespace bole
