// window_attention.hip - attention with a sliding window and visible first tokens over a
// paged cache: a row at position p sees keys at s <= p on its own path with p - s < window
// or s < sinks;   out = sum_s w_s v_s,  w = softmax(scale q . k_s).
#include "window_device.h"
#include "launch.h"

namespace bole {

// Any width up to 256 and either type: one wavefront per (row, query head). Keys come 64 at a
// time, a key a lane, with a running maximum and sum; a lane then owns output dimensions
// lane, lane + 64, .. and adds the keys' values. Only seen keys and values are loaded.
template <typename T>
__global__ __launch_bounds__(64) void window_generic_kernel(const WindowArgs a) {
    const WindowShape &s = a.s;
    const int row = blockIdx.x, h = blockIdx.y, hk = h / (s.H / s.HK), lane = lane_id();
    const bool ordered = offsets_ordered(a.offsets, s.B, s.T);
    if (row == 0 && h == 0 && a.status)
        for (int b = lane; b < s.B; b += 64)
            if (!ordered || a.offsets[b + 1] == a.offsets[b])
                a.status[b] = ordered ? BOLE_TREE_OK : BOLE_TREE_BAD_SIZE;
    if (!ordered) return;
    const int b = sequence_of(a.offsets, s.B, row);
    const int lo = a.offsets[b], n = a.offsets[b + 1] - lo, i = row - lo;
    if (i < 0 || i >= n) return;
    const int len = a.cache_len[b];
    int st = a.parent && n > kMaxTree ? BOLE_TREE_BAD_SIZE : BOLE_TREE_OK;
    uint64_t mask = 0;
    int depth = 0;
    if (a.parent && st == BOLE_TREE_OK) {
        const WaveTopo t = wave_topology(a.parent + lo, n);
        st = t.bad;
        mask = shfl_u64(t.mask, i);
        depth = t.depth;
    }
    if (st == BOLE_TREE_OK) st = length_status(s, len);
    if (st == BOLE_TREE_OK) st = pages_status(a, b, len);
    if (i == 0 && h == 0 && lane == 0 && a.status) a.status[b] = st;
    T *o = static_cast<T *>(a.out) + ((size_t)row * s.H + h) * s.D;
    if (st != BOLE_TREE_OK) {
        if (st != BOLE_TREE_BAD_SIZE)
            for (int e = lane; e < s.D; e += 64) o[e] = (T)__builtin_nanf("");
        return;
    }
    const T *q = static_cast<const T *>(a.q) + ((size_t)row * s.H + h) * s.D;
    const int32_t *table = a.page_table + (size_t)b * s.max_pages;
    const int ps = 1 << s.page_shift;
    // element offset of key x: of a cached position, or of an own row
    auto at = [&](bool own, int x) -> size_t {
        if (own) return ((size_t)(lo + x) * s.HK + hk) * s.D;
        return (((size_t)table[x >> s.page_shift] * s.HK + hk) * ps + (x & (ps - 1))) * s.D;
    };
    float m = -INFINITY, sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    auto block = [&](bool own, int x0, bool seen) {
        const T *kp = static_cast<const T *>(own ? a.k : a.k_cache);
        const T *vp = static_cast<const T *>(own ? a.v : a.v_cache);
        float z = -INFINITY;
        const size_t mine = seen ? at(own, x0 + lane) : 0;
        if (seen) {
            z = 0.f;
            for (int e = 0; e < s.D; ++e) z = fmaf(to_f32(q[e]), to_f32(kp[mine + e]), z);
            z *= s.scale;
        }
        float top = z;
        for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
        const uint64_t live = __ballot(seen);
        if (live == 0) return;
        const float next = fmaxf(m, top), keep = m == -INFINITY ? 0.f : expf(m - next);
        const float p = seen ? expf(z - next) : 0.f;
        float add = p;
        for (int d = 1; d < 64; d <<= 1) add += __shfl_xor(add, d, 64);
        sum = sum * keep + add;
        m = next;
        for (int j = 0; j < 4; ++j) acc[j] *= keep;
        for (uint64_t l = live; l; l &= l - 1) {
            const int x = __ffsll((unsigned long long)l) - 1;
            const float w = __shfl(p, x, 64);
            const size_t off = (size_t)shfl_u64(mine, x);
            for (int j = 0; j < 4; ++j)
                if (lane + 64 * j < s.D) acc[j] = fmaf(w, to_f32(vp[off + lane + 64 * j]), acc[j]);
        }
    };
    auto range = [&](bool own, int x0, int x1) {
        for (int x = x0; x < x1; x += 64) block(own, x, x + lane < x1);
    };
    const int pos = a.parent ? len + __popcll(mask) - 1 : len + i;
    const int edge = pos - s.window + 1;  // the first position inside the window
    const int sink = min(s.sinks, len);
    range(false, 0, sink);
    range(false, max(sink, edge), len);
    if (a.parent) {
        const int at_j = len + depth - 1;
        block(true, 0, ((mask >> lane) & 1ull) && (at_j >= edge || at_j < s.sinks));
    } else {
        const int own_sink = min(max(0, s.sinks - len), i + 1);
        range(true, 0, own_sink);
        range(true, max(own_sink, edge - len), i + 1);
    }
    for (int j = 0; j < 4; ++j)
        if (lane + 64 * j < s.D) o[lane + 64 * j] = (T)(acc[j] / sum);
}

hipError_t launch_window(const void *q, const void *k, const void *v, const void *k_cache,
                         const void *v_cache, const int32_t *page_table, const int32_t *cache_len,
                         const int32_t *parent, const int32_t *node_offsets, void *out,
                         void *workspace, const bole_window_dims_t &d, int32_t *seq_status,
                         hipStream_t stream) {
    const WindowArgs a = {q, k, v, k_cache, v_cache, page_table, cache_len, parent, node_offsets, out,
                          seq_status,
                          {d.batch, d.heads, d.kv_heads, d.head_dim, d.total_rows, d.num_pages,
                           __builtin_ctz((unsigned)d.page_size), d.max_pages, d.window, d.sinks,
                           d.scale}};
    if (window_mfma_applies(d, a)) return launch_window_mfma(a, d, workspace, stream);
    const dim3 grid((unsigned)(d.total_rows > 0 ? d.total_rows : 1), (unsigned)d.heads);
    if (d.dtype == BOLE_DTYPE_F32)
        window_generic_kernel<float><<<grid, dim3(64), 0, stream>>>(a);
    else
        window_generic_kernel<__bf16><<<grid, dim3(64), 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace bole
