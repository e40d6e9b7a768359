// prefix_attention.hip - attention of sequences that share long prefixes over a paged cache: a row
// sees its group's prefix, its sequence's cached tokens and the rows on its path;
// out = sum_s w_s v_s,  w = softmax(scale q . k_s).
#include <cmath>

#include "prefix_device.h"
#include "launch.h"

namespace bole {

// Any width up to 256 and either type: one wavefront per (row, query head). Keys come 64 at a
// time, a key a lane, with a running maximum and sum; a lane then owns output dimensions
// lane, lane + 64, .. and adds the keys' values. Only seen keys and values are loaded.
template <typename T>
__global__ __launch_bounds__(64) void prefix_generic_kernel(const PrefixArgs p) {
    const WindowArgs &a = p.w;
    const WindowShape &s = a.s;
    const int row = blockIdx.x, h = blockIdx.y, hk = h / (s.H / s.HK), lane = lane_id();
    const bool ordered = offsets_ordered(a.offsets, s.B, s.T) &&
                         (p.groups == 0 || offsets_ordered(p.group_offsets, p.groups, s.B));
    if (row == 0 && h == 0 && a.status)
        for (int b = lane; b < s.B; b += 64)
            if (!ordered || a.offsets[b + 1] == a.offsets[b])
                a.status[b] = ordered ? BOLE_TREE_OK : BOLE_TREE_BAD_SIZE;
    if (!ordered) return;
    const int b = sequence_of(a.offsets, s.B, row);
    const int lo = a.offsets[b], n = a.offsets[b + 1] - lo, i = row - lo;
    if (i < 0 || i >= n) return;
    const int len = a.cache_len[b];
    const Group group = group_of(p, b);
    int st = a.parent && n > kMaxTree ? BOLE_TREE_BAD_SIZE : BOLE_TREE_OK;
    uint64_t mask = 0;
    if (a.parent && st == BOLE_TREE_OK) {
        const WaveTopo t = wave_topology(a.parent + lo, n);
        st = t.bad;
        mask = shfl_u64(t.mask, i);
    }
    if (st == BOLE_TREE_OK) st = length_status(s, len);
    if (st == BOLE_TREE_OK) st = pages_status(a, b, len);
    if (st == BOLE_TREE_OK && group.found) st = prefix_status(p, group.g, group.len);
    if (i == 0 && h == 0 && lane == 0 && a.status) a.status[b] = st;
    T *o = static_cast<T *>(a.out) + ((size_t)row * s.H + h) * s.D;
    if (st != BOLE_TREE_OK) {
        if (st != BOLE_TREE_BAD_SIZE)
            for (int e = lane; e < s.D; e += 64) o[e] = (T)__builtin_nanf("");
        return;
    }
    const T *q = static_cast<const T *>(a.q) + ((size_t)row * s.H + h) * s.D;
    const int ps = 1 << s.page_shift;
    float m = -INFINITY, sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    // keys x0 + lane that are seen: of the pages of `table`, or (none) own rows
    auto block = [&](const int32_t *table, int x0, bool seen) {
        const T *kp = static_cast<const T *>(table ? a.k_cache : a.k);
        const T *vp = static_cast<const T *>(table ? a.v_cache : a.v);
        const int x = x0 + lane;
        size_t mine = 0;
        float z = -INFINITY;
        if (seen) {
            mine = table ? (((size_t)table[x >> s.page_shift] * s.HK + hk) * ps + (x & (ps - 1))) * s.D
                         : ((size_t)(lo + x) * s.HK + hk) * s.D;
            z = 0.f;
            for (int e = 0; e < s.D; ++e) z = fmaf(to_f32(q[e]), to_f32(kp[mine + e]), z);
            z *= s.scale;
        }
        float top = z;
        for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
        const uint64_t live = __ballot(seen);
        if (live == 0) return;
        const float next = fmaxf(m, top), keep = m == -INFINITY ? 0.f : expf(m - next);
        const float w = seen ? expf(z - next) : 0.f;
        float add = w;
        for (int d = 1; d < 64; d <<= 1) add += __shfl_xor(add, d, 64);
        sum = sum * keep + add;
        m = next;
        for (int j = 0; j < 4; ++j) acc[j] *= keep;
        for (uint64_t l = live; l; l &= l - 1) {
            const int y = __ffsll((unsigned long long)l) - 1;
            const float wy = __shfl(w, y, 64);
            const size_t off = (size_t)shfl_u64(mine, y);
            for (int j = 0; j < 4; ++j)
                if (lane + 64 * j < s.D) acc[j] = fmaf(wy, to_f32(vp[off + lane + 64 * j]), acc[j]);
        }
    };
    const int32_t *prefix = p.prefix_table + (size_t)group.g * p.max_prefix_pages;
    for (int x = 0; x < group.len; x += 64) block(prefix, x, x + lane < group.len);
    const int32_t *table = a.page_table + (size_t)b * s.max_pages;
    for (int x = 0; x < len; x += 64) block(table, x, x + lane < len);
    if (a.parent) {
        block(nullptr, 0, (mask >> lane) & 1ull);
    } else {
        for (int x = 0; x <= i; x += 64) block(nullptr, x, x + lane <= i);
    }
    for (int j = 0; j < 4; ++j)
        if (lane + 64 * j < s.D) o[lane + 64 * j] = (T)(acc[j] / sum);
}

hipError_t launch_prefix(const void *q, const void *k, const void *v, const void *k_cache,
                         const void *v_cache, const int32_t *prefix_table, const int32_t *prefix_len,
                         const int32_t *group_offsets, const int32_t *page_table,
                         const int32_t *cache_len, const int32_t *parent, const int32_t *node_offsets,
                         void *out, void *workspace, const bole_prefix_dims_t &d, int32_t *seq_status,
                         hipStream_t stream) {
    const PrefixArgs a = {{q, k, v, k_cache, v_cache, page_table, cache_len, parent, node_offsets, out,
                           seq_status,
                           {d.batch, d.heads, d.kv_heads, d.head_dim, d.total_rows, d.num_pages,
                            __builtin_ctz((unsigned)d.page_size), d.max_pages, 0x7fffffff, 0, d.scale}},
                          prefix_table, prefix_len, group_offsets, d.groups, d.max_prefix_pages};
    if (prefix_mfma_applies(d, a)) return launch_prefix_mfma(a, d, workspace, stream);
    const dim3 grid((unsigned)(d.total_rows > 0 ? d.total_rows : 1), (unsigned)d.heads);
    if (d.dtype == BOLE_DTYPE_F32)
        prefix_generic_kernel<float><<<grid, dim3(64), 0, stream>>>(a);
    else
        prefix_generic_kernel<__bf16><<<grid, dim3(64), 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace bole

extern "C" {

bole_status_t bole_prefix_check_dims(const bole_prefix_dims_t *d) {
    if (d == nullptr) return BOLE_ERR_INVALID_VALUE;
    if (d->batch < 0 || d->heads < 1 || d->kv_heads < 1 || d->heads % d->kv_heads != 0 ||
        d->head_dim < 1 || d->total_rows < 0 || d->num_pages < 0 || d->max_pages < 0 || d->groups < 0 ||
        d->max_prefix_pages < 0 || !std::isfinite(2.f * d->scale))
        return BOLE_ERR_INVALID_VALUE;
    if (d->page_size < 1 || (d->page_size & (d->page_size - 1)) != 0) return BOLE_ERR_INVALID_VALUE;
    if (d->dtype != BOLE_DTYPE_BF16 && d->dtype != BOLE_DTYPE_F32) return BOLE_ERR_INVALID_VALUE;
    if (d->flags & ~BOLE_FLAG_FORCE_GENERIC) return BOLE_ERR_INVALID_VALUE;
    if (d->head_dim > 256 || d->page_size > 1024 || d->heads > 65535) return BOLE_ERR_UNSUPPORTED;
    // Positions, those of the next few key tiles behind the last among them, and (sequences +
    // groups) x heads fit 31 bits, and a launch has fewer than 2^32 threads: 64 a row and head (in
    // fours), or 256 for each 16 rows a key head packs and up to three times a sequence or group (of few rows).
    const int64_t rows = d->total_rows, lists = (int64_t)d->batch + d->groups;
    if ((int64_t)d->max_pages * d->page_size + rows > (1LL << 31) - 1024 ||
        (int64_t)d->max_prefix_pages * d->page_size + rows > (1LL << 31) - 1024 ||
        lists * d->heads > 0x7fffffffLL || rows * d->heads + 3 >= 1LL << 26 ||
        rows * d->heads / 16 + 3 * lists * d->kv_heads >= 1LL << 24)
        return BOLE_ERR_UNSUPPORTED;
    return BOLE_OK;
}

size_t bole_prefix_workspace_size(const bole_prefix_dims_t *dims) {
    if (bole_prefix_check_dims(dims) != BOLE_OK) return 0;
    return bole::prefix_workspace(*dims);
}

bole_status_t bole_prefix_attention(const void *q, const void *k, const void *v,
                                    const void *k_cache, const void *v_cache,
                                    const int32_t *prefix_table, const int32_t *prefix_len,
                                    const int32_t *group_offsets, const int32_t *page_table,
                                    const int32_t *cache_len, const int32_t *parent,
                                    const int32_t *node_offsets, void *out, void *workspace,
                                    size_t workspace_bytes, const bole_prefix_dims_t *dims,
                                    int32_t *seq_status, bole_stream_t stream) {
    const bole_status_t st = bole_prefix_check_dims(dims);
    if (st != BOLE_OK) return st;
    const bole_prefix_dims_t &d = *dims;
    if (d.batch == 0) return BOLE_OK;
    if (cache_len == nullptr || node_offsets == nullptr) return BOLE_ERR_INVALID_VALUE;
    if (d.total_rows > 0 && (q == nullptr || k == nullptr || v == nullptr || out == nullptr))
        return BOLE_ERR_INVALID_VALUE;
    if (d.max_pages > 0 && page_table == nullptr) return BOLE_ERR_INVALID_VALUE;
    if (d.groups > 0 && (prefix_len == nullptr || group_offsets == nullptr ||
                         (d.max_prefix_pages > 0 && prefix_table == nullptr)))
        return BOLE_ERR_INVALID_VALUE;
    if (d.num_pages > 0 && (k_cache == nullptr || v_cache == nullptr)) return BOLE_ERR_INVALID_VALUE;
    const size_t need = bole::prefix_workspace(d);
    if (need > 0 && (workspace == nullptr || reinterpret_cast<uintptr_t>(workspace) % 16 != 0 ||
                     workspace_bytes < need))
        return BOLE_ERR_INVALID_VALUE;
    const hipError_t e = bole::launch_prefix(q, k, v, k_cache, v_cache, prefix_table, prefix_len,
                                             group_offsets, page_table, cache_len, parent, node_offsets,
                                             out, workspace, d, seq_status,
                                             reinterpret_cast<hipStream_t>(stream));
    return e == hipSuccess ? BOLE_OK : BOLE_ERR_HIP;
}

}  // extern "C"
