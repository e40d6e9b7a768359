// append.hip - new tokens into a paged cache: all rows of each sequence, or the rows of its
// accepted path, behind its cached tokens.
//
// A bad sequence adds nothing, so each of its rows has to know: a wavefront that finds a row's place
// checks every page that its sequence's new tokens go to. Rows are on their way meanwhile: bound by
// the copy, or, for accepted paths, by the chain offsets - path - pages - rows (64 of them 4.9 us).
#include "delta_device.h"
#include "launch.h"

namespace bole {

struct AppendArgs {
    const void *k, *v;
    void *k_cache, *v_cache;
    const int32_t *page_table, *cache_len, *parent, *offsets, *accepted_idx, *accepted_len;
    int32_t *new_len, *status;
    int B, HK, D, T, pages, page_shift, max_pages, max_path;
    int64_t k_stride, v_stride;
    bool paths;
};

// Whether n tokens fit behind len, into pages that exist. One wavefront.
__device__ __forceinline__ int room_status(const AppendArgs &a, int b, int len, int n) {
    if (len < 0 || (int64_t)len + n > ((int64_t)a.max_pages << a.page_shift)) return BOLE_TREE_BAD_CACHE;
    if (n == 0) return BOLE_TREE_OK;
    const int32_t *table = a.page_table + (size_t)b * a.max_pages;
    bool bad = false;
    for (int i = (len >> a.page_shift) + lane_id(); i <= (len + n - 1) >> a.page_shift; i += 64)
        bad |= (unsigned)table[i] >= (unsigned)a.pages;
    return __any(bad) ? BOLE_TREE_BAD_CACHE : BOLE_TREE_OK;
}

constexpr size_t kNowhere = ~(size_t)0;

// Byte offset in either cache of position `at` of sequence b, head 0.
__device__ __forceinline__ size_t place_of(const AppendArgs &a, int size, int b, int at) {
    const int page = a.page_table[(size_t)b * a.max_pages + (at >> a.page_shift)];
    return ((((size_t)page * a.HK) << a.page_shift) + (at & ((1 << a.page_shift) - 1))) * a.D * size;
}

// One piece, of V (a power of two) bytes, of a row's keys (the first half of 2 n pieces) or values.
template <typename V>
struct Piece {
    const char *from;
    char *to;
    size_t stride, head;  // bytes between rows; from the row's place in the cache on
    __device__ __forceinline__ Piece(const AppendArgs &a, int size, int e, int n) {
        const bool value = e >= n;
        e -= value ? n : 0;
        const int per = a.D * size / (int)sizeof(V), h = e / per, c = e - h * per;
        from = static_cast<const char *>(value ? a.v : a.k) + (size_t)e * sizeof(V);
        to = static_cast<char *>(value ? a.v_cache : a.k_cache);
        stride = (size_t)(value ? a.v_stride : a.k_stride) * size;
        head = (((size_t)h << a.page_shift) * a.D) * size + (size_t)c * sizeof(V);
    }
    __device__ __forceinline__ V load(int row) const { return *reinterpret_cast<const V *>(from + row * stride); }
    __device__ __forceinline__ void store(size_t place, V x) const { *reinterpret_cast<V *>(to + place + head) = x; }
};

// A workgroup ROWS neighbouring rows: eight from 2048 rows on, whose loads are in flight together while
// their places are found (8 heads of 128 in bf16: 16384 rows 28.4 us, 4.7 TB/s, with one row each 34.9; 4096
// 8.8 and 9.2; 2048 5.7 and 5.5). Fewer rows take one each, so that more CUs have work.
template <typename V, int ROWS>
__global__ __launch_bounds__(256) void append_rows_kernel(const AppendArgs a, int size) {
    __shared__ size_t s_place[ROWS];
    const int row0 = blockIdx.x * ROWS, rows = min(ROWS, a.T - row0), lane = lane_id(), wave = threadIdx.x >> 6;
    const int n = a.HK * (a.D * size / (int)sizeof(V));
    V x[ROWS];
    if (rows > 0) {
        const Piece<V> p(a, size, min((int)threadIdx.x, 2 * n - 1), n);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) x[r] = p.load(row0 + min(r, rows - 1));
    }
    constexpr int EACH = (ROWS + 3) / 4;
    RowOwner o = {false, true, -1, 0, 0};
    int len = 0, st = BOLE_TREE_OK;
    for (int i = 0; i < EACH; ++i) {
        const int r = wave * EACH + i, row = row0 + r;
        if (r >= ROWS || (r >= rows && row != 0)) break;
        if (!o.found || row >= o.lo + o.n) {
            o = owner_of(a.offsets, a.B, a.T, row);
            if (o.found) {
                len = a.cache_len[o.b];
                st = room_status(a, o.b, len, o.n);
            }
        }
        if (row == 0)  // sequences without rows, and all of them if offsets are unordered
            for (int b = lane; b < a.B; b += 64)
                if (!o.ordered || a.offsets[b + 1] == a.offsets[b]) {
                    const int have = a.cache_len[b];
                    const int bad = !o.ordered ? BOLE_TREE_BAD_SIZE
                                    : have < 0 || have > ((int64_t)a.max_pages << a.page_shift) ? BOLE_TREE_BAD_CACHE
                                                                                              : BOLE_TREE_OK;
                    if (a.status) a.status[b] = bad;
                    if (a.new_len) a.new_len[b] = have;
                }
        if (o.found && row == o.lo && lane == 0) {
            if (a.status) a.status[o.b] = st;
            if (a.new_len) a.new_len[o.b] = st == BOLE_TREE_OK ? len + o.n : len;
        }
        if (lane == 0)
            s_place[r] = o.found && r < rows && st == BOLE_TREE_OK ? place_of(a, size, o.b, len + row - o.lo) : kNowhere;
    }
    if (rows <= 0) return;  // (a call without rows only reports)
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * n; e += 256) {
        const Piece<V> p(a, size, e, n);
        if (e != (int)threadIdx.x) {
#pragma unroll
            for (int r = 0; r < ROWS; ++r) x[r] = p.load(row0 + min(r, rows - 1));
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
            if (r < rows && s_place[r] != kNowhere) p.store(s_place[r], x[r]);
    }
}

// A workgroup a node of an accepted path.
template <typename V>
__global__ __launch_bounds__(256) void append_path_kernel(const AppendArgs a, int size) {
    const int b = blockIdx.x, m = blockIdx.y;
    const WavePath w = wave_path(a.parent, a.offsets, a.accepted_idx, a.accepted_len, b, a.T, a.max_path);
    const int len = a.cache_len[b];
    int st = w.status;
    if (st == BOLE_TREE_OK) st = room_status(a, b, len, w.len);
    if (m == 0 && threadIdx.x == 0) {
        if (a.status) a.status[b] = st;
        if (a.new_len) a.new_len[b] = st == BOLE_TREE_OK ? len + w.len : len;
    }
    if (st != BOLE_TREE_OK || m >= w.len) return;
    const int row = __builtin_amdgcn_readlane(w.row, m), n = a.HK * (a.D * size / (int)sizeof(V));
    const size_t place = place_of(a, size, b, len + m);
    for (int e = threadIdx.x; e < 2 * n; e += 256) {
        const Piece<V> p(a, size, e, n);
        p.store(place, p.load(row));
    }
}

template <typename V>
static hipError_t launch_pieces(const AppendArgs &a, int size, hipStream_t stream) {
    if (a.paths) {
        const dim3 grid((unsigned)a.B, (unsigned)(a.max_path > 0 ? a.max_path : 1));
        append_path_kernel<V><<<grid, dim3(256), 0, stream>>>(a, size);
    } else {
        if (a.T >= 2048) append_rows_kernel<V, 8><<<dim3((unsigned)((a.T + 7) / 8)), dim3(256), 0, stream>>>(a, size);
        else append_rows_kernel<V, 1><<<dim3((unsigned)(a.T > 0 ? a.T : 1)), dim3(256), 0, stream>>>(a, size);
    }
    return hipGetLastError();
}

hipError_t launch_append(const void *k, const void *v, void *k_cache, void *v_cache,
                         const int32_t *page_table, const int32_t *cache_len, const int32_t *parent,
                         const int32_t *node_offsets, const int32_t *accepted_idx,
                         const int32_t *accepted_len, int32_t *new_len, const bole_append_dims_t &d,
                         int32_t *seq_status, hipStream_t stream) {
    const AppendArgs a = {k, v, k_cache, v_cache, page_table, cache_len, parent, node_offsets,
                          accepted_idx, accepted_len, new_len, seq_status, d.batch, d.kv_heads, d.head_dim,
                          d.total_rows, d.num_pages, __builtin_ctz((unsigned)d.page_size), d.max_pages,
                          d.max_path, d.k_stride, d.v_stride, accepted_len != nullptr};
    const int size = d.dtype == BOLE_DTYPE_F32 ? 4 : 2;
    uintptr_t bits = (uintptr_t)d.head_dim * size | (uintptr_t)d.k_stride * size | (uintptr_t)d.v_stride * size;
    for (const void *p : {k, v, static_cast<const void *>(k_cache), static_cast<const void *>(v_cache)})
        bits |= reinterpret_cast<uintptr_t>(p);
    if (bits % 16 == 0) return launch_pieces<uint4>(a, size, stream);
    return size == 4 ? launch_pieces<uint32_t>(a, size, stream) : launch_pieces<uint16_t>(a, size, stream);
}

}  // namespace bole

extern "C" {

bole_status_t bole_append_check_dims(const bole_append_dims_t *d) {
    if (d == nullptr) return BOLE_ERR_INVALID_VALUE;
    if (d->batch < 0 || d->kv_heads < 1 || d->head_dim < 1 || d->total_rows < 0 || d->num_pages < 0 ||
        d->max_pages < 0 || d->max_path < 0 || d->flags != 0)
        return BOLE_ERR_INVALID_VALUE;
    if (d->page_size < 1 || (d->page_size & (d->page_size - 1)) != 0) return BOLE_ERR_INVALID_VALUE;
    if (d->dtype != BOLE_DTYPE_BF16 && d->dtype != BOLE_DTYPE_F32) return BOLE_ERR_INVALID_VALUE;
    if (d->k_stride < (int64_t)d->kv_heads * d->head_dim || d->v_stride < (int64_t)d->kv_heads * d->head_dim)
        return BOLE_ERR_INVALID_VALUE;
    if (d->head_dim > 256 || d->page_size > 1024 || d->kv_heads > 65535 || d->max_path > bole::kMaxTreeNodesHost)
        return BOLE_ERR_UNSUPPORTED;
    // positions fit 31 bits, and a launch has fewer than 2^32 threads
    if ((int64_t)d->max_pages * d->page_size + d->total_rows > 0x7fffffffLL || d->total_rows >= 1 << 24 ||
        (int64_t)d->batch * (d->max_path > 0 ? d->max_path : 1) >= 1 << 24)
        return BOLE_ERR_UNSUPPORTED;
    return BOLE_OK;
}

bole_status_t bole_cache_append(const void *k, const void *v, void *k_cache, void *v_cache,
                                const int32_t *page_table, const int32_t *cache_len,
                                const int32_t *parent, const int32_t *node_offsets,
                                const int32_t *accepted_idx, const int32_t *accepted_len,
                                int32_t *new_len, const bole_append_dims_t *dims,
                                int32_t *seq_status, bole_stream_t stream) {
    const bole_status_t st = bole_append_check_dims(dims);
    if (st != BOLE_OK) return st;
    const bole_append_dims_t &d = *dims;
    const bool paths = accepted_len != nullptr;
    // a path comes with its trees, its rows' indices (none if max_path is 0) and its lengths
    if ((accepted_idx != nullptr && !paths) || (paths && d.max_path > 0 && accepted_idx == nullptr) ||
        (!paths && (parent != nullptr || d.max_path > 0)))
        return BOLE_ERR_INVALID_VALUE;
    if (d.batch == 0) return BOLE_OK;
    if (cache_len == nullptr || node_offsets == nullptr || (d.max_pages > 0 && page_table == nullptr))
        return BOLE_ERR_INVALID_VALUE;
    if (d.total_rows > 0 && (k == nullptr || v == nullptr || (paths && parent == nullptr)))
        return BOLE_ERR_INVALID_VALUE;
    if (d.num_pages > 0 && (k_cache == nullptr || v_cache == nullptr)) return BOLE_ERR_INVALID_VALUE;
    const hipError_t e = bole::launch_append(k, v, k_cache, v_cache, page_table, cache_len, parent,
                                             node_offsets, accepted_idx, accepted_len, new_len, d,
                                             seq_status, reinterpret_cast<hipStream_t>(stream));
    return e == hipSuccess ? BOLE_OK : BOLE_ERR_HIP;
}

}  // extern "C"
