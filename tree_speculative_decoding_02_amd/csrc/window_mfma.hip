// window_mfma.hip - windowed attention on the matrix cores, bf16, head widths 64, 96 and 128.
//
// A sequence's rows and the G = H / H_kv query heads that share a key head are packed as
// rows R = i G + g, so one pass over the keys serves all of them. With the transposed score
// tile S^T = K Q^T (keys down, queries across), a lane holds one query: its running maximum
// and sum are lane-local up to a last exchange between the lanes that share the query, and
// the exponentials, rounded to bf16, already lie as the B operand of O^T = V^T P^T (a
// permutation of the keys within a product, the same for both operands). V^T comes from
// row-major LDS through the transposing read.
//
// The keys a tile of rows can see are one virtual list: the cached first tokens, the cached
// window behind the tile's first row, the call's own first tokens, the call's own rows. Tiles
// of 64 keys that every row sees are taken without tests; the others test each key. Slots
// past the end repeat the last key, so nothing that no row of the sequence sees is read, and
// no load depends on a branch.
//
// Two shapes of workgroup:
//  - rows: 128 rows, 32 a wavefront, keys and values staged in LDS for all four wavefronts
//    (two buffers, one barrier a tile). For prompts and draft trees.
//  - tokens: 16 rows, the key tiles dealt to the four wavefronts, each with its own softmax
//    state, merged at the end; keys go straight to registers. For single tokens, where the
//    cache's bytes set the time.
// With few rows in the whole call the key list is also split over workgroups; a second kernel
// merges the parts.
#include "window_device.h"
#include "launch.h"

namespace bole {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kKeys = 64;        // keys a tile
constexpr int kRowTile = 128;    // rows a workgroup, rows form
constexpr int kTokenTile = 16;   // rows a workgroup, tokens form

// Where the unnormalised parts of a split call go: O [parts][tiles][MT][D], then (m, l)
// [parts][tiles][MT][2]. A part's m is NaN for a sequence whose rows become NaN and +inf for
// one that is not touched.
struct WindowParts {
    float *o, *ml;
    int n;         // parts of the key list
};

// Row tile of a workgroup and the key list it runs over.
struct RowTile {
    int b, lo, n, tile, slot0;       // sequence, its rows, tile within it, its first slot
    int status, len;
    int i0, i1;                      // rows (before packing) of the tile: [i0, i1)
    int n1, n2, n3, n4, w0, o2;      // key list: sinks, window from w0, own sinks, own rows from o2
    int total, all_from;             // keys; first position every row's window holds
};

__device__ __forceinline__ void key_list(const WindowShape &s, bool tree, RowTile &t) {
    const int p0 = tree ? t.len : t.len + t.i0;                      // first and last position
    const int p1 = tree ? t.len + t.n - 1 : t.len + t.i1 - 1;        // (a bound for trees)
    const int edge = p0 - s.window + 1;
    t.all_from = p1 - s.window + 1;
    t.n1 = min(s.sinks, t.len);
    t.w0 = max(t.n1, edge);
    t.n2 = max(0, t.len - t.w0);
    t.n3 = tree ? 0 : min(max(0, s.sinks - t.len), t.i1);
    t.o2 = tree ? 0 : max(t.n3, edge - t.len);
    t.n4 = tree ? t.n : max(0, t.i1 - t.o2);
    t.total = t.n1 + t.n2 + t.n3 + t.n4;
}

// Finds the workgroup's tile and all that is wrong with its sequence but its pages. Every
// wavefront computes the same. mask: of a tree, lane i's node's visible own nodes (its path, cut
// to the window); depth: its depth. False: no rows here.
template <int MT>
__device__ __forceinline__ bool find_tile(const WindowArgs &a, int G, int slot, bool report,
                                          RowTile &t, uint64_t &mask, int &depth) {
    const WindowShape &s = a.s;
    const int lane = lane_id();
    t.status = BOLE_TREE_OK;
    const Located l = locate(a.offsets, a.cache_len, s.B, s.T, G, MT, slot);
    if (!l.found) {
        if (!l.ordered && report && slot == 0 && a.status)
            for (int b = lane; b < s.B; b += 64) a.status[b] = BOLE_TREE_BAD_SIZE;
        return false;
    }
    t.b = l.b, t.lo = l.lo, t.n = l.n, t.slot0 = l.slot0, t.len = l.per;
    t.tile = slot - t.slot0;
    if (t.n == 0 && t.tile == 0 && report && lane == 0 && a.status) a.status[t.b] = BOLE_TREE_OK;
    if (t.tile * MT >= t.n * G) return false;
    t.i0 = t.tile * MT / G;
    t.i1 = min(t.n, (t.tile * MT + MT + G - 1) / G);
    if (a.parent) {
        if (t.n > kMaxTree) {
            t.status = BOLE_TREE_BAD_SIZE;
        } else {
            const WaveTopo w = wave_topology(a.parent + t.lo, t.n);
            t.status = w.bad;
            mask = w.mask;
            depth = w.depth;
        }
    }
    if (t.status == BOLE_TREE_OK) t.status = length_status(s, t.len);
    if (t.status != BOLE_TREE_OK) return true;
    if (a.parent && s.window < kMaxTree) {
        // path nodes that the window has left behind, unless they are first tokens
        for (int j = 0; j < t.n; ++j) {
            const int dj = __builtin_amdgcn_readlane(depth, j);
            if (depth - dj >= s.window && t.len + dj - 1 >= s.sinks) mask &= ~(1ull << j);
        }
    }
    key_list(s, a.parent != nullptr, t);
    if (t.n1 + t.n2 > 0 && s.pages == 0) t.status = BOLE_TREE_BAD_CACHE;
    return true;
}

__device__ __forceinline__ int cached_position(const RowTile &t, int x) {
    return x < t.n1 ? x : t.w0 + (x - t.n1);
}

__device__ __forceinline__ int own_row(const RowTile &t, int x) {
    const int j = x - t.n1 - t.n2;
    return j < t.n3 ? j : t.o2 + (j - t.n3);
}

// Page of key x as the table has it; 0 for the call's own rows.
__device__ __forceinline__ int key_page(const WindowShape &s, const int32_t *__restrict__ table,
                                        const RowTile &t, int x) {
    x = min(x, t.total - 1);
    return x < t.n1 + t.n2 ? table[cached_position(t, x) >> s.page_shift] : 0;
}

// A page that is not in the cache stands for its last one: the first loads go out before the
// sequence's pages are known to be valid, and are dropped if they are not.
// Row (of D elements) of key x: in the cache's [page][head][slot] order, or in the call's k and
// v. At 128 bytes a row and more, 32 bits number more rows than memory holds.
__device__ __forceinline__ uint32_t key_row(const WindowShape &s, const RowTile &t, int hk, int x,
                                            int page) {
    if (x < t.n1 + t.n2) {
        const uint32_t slot = cached_position(t, x) & ((1 << s.page_shift) - 1);
        return ((min((uint32_t)page, (uint32_t)s.pages - 1) * s.HK + hk) << s.page_shift) + slot;
    }
    return (uint32_t)(t.lo + own_row(t, x)) * s.HK + hk;
}

// Whether every row of the tile sees all 64 keys from x0 on.
__device__ __forceinline__ bool tile_open(const RowTile &t, bool tree, int x0) {
    const int x1 = x0 + kKeys, c = t.n1 + t.n2;
    if (x1 <= t.n1) return true;
    if (x0 >= t.n1 && x1 <= c) return t.w0 + (x0 - t.n1) >= t.all_from;
    if (!tree && x0 >= c + t.n3 && x1 <= t.total) {
        const int j = own_row(t, x0);
        return j + kKeys - 1 <= t.i0 && t.len + j >= t.all_from;
    }
    return false;
}

__device__ __forceinline__ uint64_t bits_below(int n) {
    return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}

// The keys x0 .. x0 + 63 that a query sees, as bits: row i of its sequence, window from position
// qe on, own nodes qmask for trees. Each part of the list shows it an interval (or the path).
__device__ __forceinline__ uint64_t seen_keys(const RowTile &t, bool tree, int i, int qe, uint64_t qmask,
                                              int x0) {
    const int c = t.n1 + t.n2 - x0, from = max(qe, 0);
    uint64_t m = bits_below(c) & ~bits_below(t.n1 - x0 + max(0, from - t.w0));
    m |= bits_below(t.n1 - x0);
    if (tree) {
        if (c > -64 && c < 64) m |= (c >= 0 ? qmask << c : qmask >> -c) & bits_below(c + t.n4);
    } else {
        const int own = c + t.n3;
        m |= bits_below(c + min(t.n3, i + 1)) & ~bits_below(c);
        m |= bits_below(own + min(t.n4, i + 1 - t.o2)) & ~bits_below(own + max(0, from - t.len - t.o2));
    }
    return m;
}

// LDS row strides in elements: K rows 16 bytes past a multiple of 256 apart or an odd number
// of 16-byte pieces (16 rows' pieces in distinct banks), V rows 64 or 192 bytes past one (the
// four rows of a transposing read in distinct quarters).
template <int D> struct Pad {
    static constexpr int K = D + 8;
    static constexpr int V = D == 128 ? 160 : 96;
};

constexpr float kLog2e = 1.4426950408889634f;

template <int D>
__global__ __launch_bounds__(256, 2) void window_rows_kernel(const WindowArgs a, const WindowParts parts,
                                                             int slots) {
    constexpr int CH = D / 8, PER = kKeys * CH / 256, KP = Pad<D>::K, VP = Pad<D>::V;
    __shared__ __align__(16) __bf16 s_k[2][kKeys * KP];
    __shared__ __align__(16) __bf16 s_v[2][kKeys * VP];
    const WindowShape &s = a.s;
    const int tid = threadIdx.x, lane = lane_id(), wave = tid >> 6, G = s.H / s.HK;
    const int hk = blockIdx.x % s.HK, slot = blockIdx.x / s.HK, part = blockIdx.y;
    const bool tree = a.parent != nullptr;
    RowTile t;
    uint64_t node_mask = 0;
    int node_depth = 0;
    const bool work = find_tile<kRowTile>(a, G, slot, hk == 0 && part == 0 && wave == 0, t, node_mask,
                                          node_depth);
    if (!work) return;
    const int col = lane & 31, hh = lane >> 5;
    const int R = t.tile * kRowTile + wave * 32 + col;
    const bool live = R < t.n * G;
    const int i = live ? R / G : 0, gq = live ? R - i * G : 0;
    const size_t row_off = ((size_t)(t.lo + i) * s.H + hk * G + gq) * D;
    __bf16 *out = static_cast<__bf16 *>(a.out) + row_off;
    const size_t part_row = ((size_t)part * slots * s.HK + blockIdx.x) * kRowTile + wave * 32 + col;
    auto give_up = [&]() {
        const bool fill = t.status != BOLE_TREE_BAD_SIZE;
        if (parts.n > 1) {
            if (live && hh == 0) parts.ml[part_row * 2] = fill ? __builtin_nanf("") : INFINITY;
        } else if (live && fill) {
            for (int e = hh; e < D; e += 2) out[e] = (__bf16)__builtin_nanf("");
        }
    };
    const bool report = hk == 0 && part == 0 && t.tile == 0 && tid == 0 && a.status;
    if (t.status != BOLE_TREE_OK) {
        if (report) a.status[t.b] = t.status;
        give_up();
        return;
    }
    const uint64_t qmask = tree ? shfl_u64(node_mask, i) : 0;
    const int qpos = tree ? t.len + __shfl(node_depth, i, 64) - 1 : t.len + i;
    const int qe = qpos - s.window + 1;
    bf16x8 qf[D / 16];
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
        qf[ks] = (bf16x8)(__bf16)0.f;
        if (live) qf[ks] = load16(static_cast<const __bf16 *>(a.q) + row_off + 16 * ks + 8 * hh);
    }
    const int32_t *table = a.page_table + (size_t)t.b * s.max_pages;
    const int tiles = (t.total + kKeys - 1) / kKeys;
    const int first = (int)((int64_t)tiles * part / parts.n);
    const int last = (int)((int64_t)tiles * (part + 1) / parts.n);

    // lane x holds the page (one tile ahead of the loads) and then the row of the tile's key x
    int page = -1;
    bf16x8 kr[PER], vr[PER];
    auto fetch = [&](int tile) {
        const uint32_t mine = key_row(s, t, hk, min(tile * kKeys + lane, t.total - 1), page);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int e = tid + 256 * j, x = min(tile * kKeys + e / CH, t.total - 1), c = e % CH;
            const size_t off = (size_t)(uint32_t)__shfl((int)mine, e / CH, 64) * D + 8 * c;
            const bool own = x >= t.n1 + t.n2;
            kr[j] = load16(static_cast<const __bf16 *>(own ? a.k : a.k_cache) + off);
            vr[j] = load16(static_cast<const __bf16 *>(own ? a.v : a.v_cache) + off);
        }
    };
    auto stage = [&](int buf) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int e = tid + 256 * j, r = e / CH, c = e % CH;
            *reinterpret_cast<bf16x8 *>(&s_k[buf][r * KP + 8 * c]) = kr[j];
            *reinterpret_cast<bf16x8 *>(&s_v[buf][r * VP + 8 * c]) = vr[j];
        }
    };
    f32x16 acc[D / 32];
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt) acc[dt] = (f32x16)0.f;
    float m = -INFINITY, l = 0.f;
    const float c2 = s.scale * kLog2e;
    const bool busy = t.tile * kRowTile + wave * 32 < t.n * G;  // else it only stages
    if (first < last) {
        page = key_page(s, table, t, first * kKeys + lane);
        fetch(first);
        page = key_page(s, table, t, (first + 1) * kKeys + lane);
    }
    t.status = pages_status(a, t.b, t.len);
    if (report) a.status[t.b] = t.status;
    if (t.status != BOLE_TREE_OK) {
        give_up();
        return;
    }
    if (first < last) {
        stage(0);
        lds_barrier();
    // (a do loop, entered only from here: a loop that could also be reached around these loads
    // would have to wait for every load in flight in each of its turns)
    int tile = first;
    do {
        const int buf = (tile - first) & 1;
        if (tile + 1 < last) {
            fetch(tile + 1);
            page = key_page(s, table, t, (tile + 2) * kKeys + lane);
        }
        const int x0 = tile * kKeys;
        if (busy) {
        f32x16 z[2];
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
            z[sub] = (f32x16)0.f;
            const __bf16 *kp = &s_k[buf][(sub * 32 + col) * KP + 8 * hh];
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
                z[sub] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(load16(kp + 16 * ks), qf[ks], z[sub],
                                                                 0, 0, 0);
        }
        float top = -INFINITY;
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) z[sub] *= c2;
        if (!tile_open(t, tree, x0)) {
            const uint64_t seen = seen_keys(t, tree, i, qe, qmask, x0) >> (4 * hh);
#pragma unroll
            for (int sub = 0; sub < 2; ++sub)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    z[sub][r] = ((uint32_t)(seen >> (32 * sub)) >> (8 * (r >> 2) + (r & 3))) & 1u
                                    ? z[sub][r] : -INFINITY;
        }
#pragma unroll
        for (int sub = 0; sub < 2; ++sub)
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, z[sub][r]);
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const float next = fmaxf(m, top);
        // nothing seen so far: keep every exponential at 0
        const float base = next == -INFINITY ? 0.f : next;
        if (__any(next > m)) {
            const float keep = __builtin_amdgcn_exp2f(m - base);
            l *= keep;
#pragma unroll
            for (int dt = 0; dt < D / 32; ++dt) acc[dt] *= keep;
            m = next;
        }
#pragma unroll
        for (int sub = 0; sub < 2; ++sub)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                z[sub][r] = __builtin_amdgcn_exp2f(z[sub][r] - base);
                l += z[sub][r];
            }
        const int sl = lane & 15;
        const __bf16 *vp = &s_v[buf][(4 * hh + (sl >> 2)) * VP + ((lane >> 4) & 1) * 16 + (sl & 3) * 4];
#pragma unroll
        for (int sub = 0; sub < 2; ++sub)
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                bf16x8 p;
#pragma unroll
                for (int j = 0; j < 8; ++j) p[j] = (__bf16)z[sub][8 * kk + j];
                const __bf16 *v0 = vp + (sub * 32 + kk * 16) * VP;
#pragma unroll
                for (int dt = 0; dt < D / 32; ++dt) {
                    const bf16x8 v = join(read_transposed(v0 + dt * 32), read_transposed(v0 + 8 * VP + dt * 32));
                    acc[dt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, p, acc[dt], 0, 0, 0);
                }
            }
        }
        if (tile + 1 < last) stage(buf ^ 1);
        lds_barrier();
    } while (++tile < last);
    }
    l += __shfl_xor(l, 32, 64);
    if (!live) return;
    if (parts.n > 1) {
        if (hh == 0) {
            parts.ml[part_row * 2] = m;
            parts.ml[part_row * 2 + 1] = l;
        }
        float *o = parts.o + part_row * D;
#pragma unroll
        for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
            for (int r = 0; r < 16; r += 4)
                *reinterpret_cast<f32x4 *>(o + dt * 32 + 2 * r + 4 * hh) =
                    f32x4{acc[dt][r], acc[dt][r + 1], acc[dt][r + 2], acc[dt][r + 3]};
        return;
    }
    const float inv = 1.f / l;
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
            bf16x4 y;
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = (__bf16)(acc[dt][r + j] * inv);
            *reinterpret_cast<bf16x4 *>(out + dt * 32 + 2 * r + 4 * hh) = y;
        }
}

template <int D>
__global__ __launch_bounds__(256, 1) void window_tokens_kernel(const WindowArgs a, const WindowParts parts,
                                                               int slots) {
    constexpr int CH = D / 8, VP = Pad<D>::V, VPER = kKeys * CH / 64;
    constexpr int JOIN = 4 * 16 * (D + 4) * 4;  // the last merge: sums, then (m, l), over the values
    static_assert(JOIN + 4 * 16 * 2 * 4 <= 4 * kKeys * VP * 2, "LDS");
    __shared__ __align__(16) char s_mem[4 * kKeys * VP * 2];
    float(*s_ml)[16][2] = reinterpret_cast<float(*)[16][2]>(s_mem + JOIN);
    const WindowShape &s = a.s;
    const int tid = threadIdx.x, lane = lane_id(), wave = tid >> 6, G = s.H / s.HK;
    const int hk = blockIdx.x % s.HK, slot = blockIdx.x / s.HK, part = blockIdx.y;
    const bool tree = a.parent != nullptr;
    RowTile t;
    uint64_t node_mask = 0;
    int node_depth = 0;
    const bool work = find_tile<kTokenTile>(a, G, slot, hk == 0 && part == 0 && wave == 0, t, node_mask,
                                            node_depth);
    if (!work) return;
    const int col = lane & 15, g = lane >> 4;
    auto row_offset = [&](int R) {
        const int i = R / G;
        return ((size_t)(t.lo + i) * s.H + hk * G + (R - i * G)) * D;
    };
    const int R = t.tile * kTokenTile + col, rows = t.n * G;
    const bool live = R < rows;
    const int i = live ? R / G : 0;
    const size_t part_tile = ((size_t)part * slots * s.HK + blockIdx.x) * kTokenTile;
    auto give_up = [&]() {
        const bool fill = t.status != BOLE_TREE_BAD_SIZE;
        if (parts.n > 1) {
            if (live && g == 0 && wave == 0)
                parts.ml[(part_tile + col) * 2] = fill ? __builtin_nanf("") : INFINITY;
        } else if (live && fill) {
            __bf16 *o = static_cast<__bf16 *>(a.out) + row_offset(R);
            for (int e = wave * 4 + g; e < D; e += 16) o[e] = (__bf16)__builtin_nanf("");
        }
    };
    const bool report = hk == 0 && part == 0 && t.tile == 0 && tid == 0 && a.status;
    if (t.status != BOLE_TREE_OK) {
        if (report) a.status[t.b] = t.status;
        give_up();
        return;
    }
    const uint64_t qmask = tree ? shfl_u64(node_mask, i) : 0;
    const int qpos = tree ? t.len + __shfl(node_depth, i, 64) - 1 : t.len + i;
    const int qe = qpos - s.window + 1;
    bf16x8 qf[D / 32];
#pragma unroll
    for (int ks = 0; ks < D / 32; ++ks) {
        qf[ks] = (bf16x8)(__bf16)0.f;
        if (live) qf[ks] = load16(static_cast<const __bf16 *>(a.q) + row_offset(R) + 32 * ks + 8 * g);
    }
    const int32_t *table = a.page_table + (size_t)t.b * s.max_pages;
    const int tiles = (t.total + kKeys - 1) / kKeys;
    const int first = (int)((int64_t)tiles * part / parts.n) + wave;
    const int last = (int)((int64_t)tiles * (part + 1) / parts.n);
    __bf16 *s_v = reinterpret_cast<__bf16 *>(s_mem) + wave * kKeys * VP;

    // a lane's keys: for K, key 16 r + col of the tile (r = 0..3), 16-byte pieces 4 ks + g; for
    // V, piece e = lane + 64 j of the tile's kKeys x CH pieces
    bf16x8 kf[4][D / 32], vr[VPER];
    int page = -1;
    auto fetch = [&](int tile) {
        const int x0 = tile * kKeys, cached = t.n1 + t.n2;
        const uint32_t mine = key_row(s, t, hk, min(x0 + lane, t.total - 1), page);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int x = min(x0 + 16 * r + col, t.total - 1);
            const size_t off = (size_t)(uint32_t)__shfl((int)mine, 16 * r + col, 64) * D + 8 * g;
            const __bf16 *p = static_cast<const __bf16 *>(x >= cached ? a.k : a.k_cache) + off;
#pragma unroll
            for (int ks = 0; ks < D / 32; ++ks) kf[r][ks] = load16(p + 32 * ks);
        }
#pragma unroll
        for (int j = 0; j < VPER; ++j) {
            const int e = lane + 64 * j, x = min(x0 + e / CH, t.total - 1);
            const size_t off = (size_t)(uint32_t)__shfl((int)mine, e / CH, 64) * D + 8 * (e % CH);
            vr[j] = load16(static_cast<const __bf16 *>(x >= cached ? a.v : a.v_cache) + off);
        }
    };
    f32x4 acc[D / 16];
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt) acc[dt] = (f32x4)0.f;
    float m = -INFINITY, l = 0.f;
    const float c2 = s.scale * kLog2e;
    if (first < last) {
        page = key_page(s, table, t, first * kKeys + lane);
        fetch(first);
        page = key_page(s, table, t, (first + 4) * kKeys + lane);
    }
    t.status = pages_status(a, t.b, t.len);
    if (report) a.status[t.b] = t.status;
    if (t.status != BOLE_TREE_OK) {
        give_up();
        return;
    }
    if (first < last) {
    int tile = first;
    do {
        const int x0 = tile * kKeys;
        f32x4 z[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            z[r] = (f32x4)0.f;
#pragma unroll
            for (int ks = 0; ks < D / 32; ++ks) z[r] = mfma16_bf16(kf[r][ks], qf[ks], z[r]);
        }
#pragma unroll
        for (int j = 0; j < VPER; ++j) {
            const int e = lane + 64 * j;
            *reinterpret_cast<bf16x8 *>(s_v + (e / CH) * VP + 8 * (e % CH)) = vr[j];
        }
        if (tile + 4 < last) {
            fetch(tile + 4);
            page = key_page(s, table, t, (tile + 8) * kKeys + lane);
        }
        float top = -INFINITY;
#pragma unroll
        for (int r = 0; r < 4; ++r) z[r] *= c2;
        if (!tile_open(t, tree, x0)) {
            const uint64_t seen = seen_keys(t, tree, i, qe, qmask, x0) >> (4 * g);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    z[r][e] = ((uint32_t)(seen >> (32 * (r >> 1))) >> (16 * (r & 1) + e)) & 1u ? z[r][e]
                                                                                            : -INFINITY;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e) top = fmaxf(top, z[r][e]);
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const float next = fmaxf(m, top), base = next == -INFINITY ? 0.f : next;
        const float keep = __builtin_amdgcn_exp2f(m - base);
        m = next;
        l *= keep;
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt) acc[dt] *= keep;
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                z[r][e] = __builtin_amdgcn_exp2f(z[r][e] - base);
                l += z[r][e];
            }
        asm volatile("" ::: "memory");  // the wavefront's own stores to s_v come first
        const __bf16 *vp = s_v + (4 * g + (col >> 2)) * VP + (col & 3) * 4;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            bf16x8 p;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                p[e] = (__bf16)z[2 * half][e];
                p[4 + e] = (__bf16)z[2 * half + 1][e];
            }
            const __bf16 *v0 = vp + half * 32 * VP;
#pragma unroll
            for (int dt = 0; dt < D / 16; ++dt)
                acc[dt] = mfma16_bf16(join(read_transposed(v0 + dt * 16), read_transposed(v0 + 16 * VP + dt * 16)),
                                      p, acc[dt]);
        }
        asm volatile("" ::: "memory");
    } while ((tile += 4) < last);
    }
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);

    // the four wavefronts' parts: O^T as [wave][row][D + 4]
    lds_barrier();
    float *s_o = reinterpret_cast<float *>(s_mem);
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt)
        *reinterpret_cast<f32x4 *>(s_o + (wave * 16 + col) * (D + 4) + dt * 16 + 4 * g) = acc[dt];
    if (g == 0) {
        s_ml[wave][col][0] = m;
        s_ml[wave][col][1] = l;
    }
    lds_barrier();
    const int r = tid >> 4, d0 = (tid & 15) * (D / 16);  // a row's 16 threads
    if (t.tile * kTokenTile + r >= rows) return;
    float mm = -INFINITY, ll = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) mm = fmaxf(mm, s_ml[w][r][0]);
    const float base = mm == -INFINITY ? 0.f : mm;
    float o[D / 16];
#pragma unroll
    for (int e = 0; e < D / 16; ++e) o[e] = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const float f = __builtin_amdgcn_exp2f(s_ml[w][r][0] - base);
        ll += f * s_ml[w][r][1];
#pragma unroll
        for (int e = 0; e < D / 16; ++e) o[e] += f * s_o[(w * 16 + r) * (D + 4) + d0 + e];
    }
    if (parts.n > 1) {
        if (d0 == 0) {
            parts.ml[(part_tile + r) * 2] = mm;
            parts.ml[(part_tile + r) * 2 + 1] = ll;
        }
#pragma unroll
        for (int e = 0; e < D / 16; ++e) parts.o[(part_tile + r) * D + d0 + e] = o[e];
        return;
    }
    __bf16 *dst = static_cast<__bf16 *>(a.out) + row_offset(t.tile * kTokenTile + r) + d0;
    const float inv = 1.f / ll;
#pragma unroll
    for (int e = 0; e < D / 16; ++e) dst[e] = (__bf16)(o[e] * inv);
}

// Joins the parts of a split call (at most 64): a workgroup a row, wavefront w takes parts w,
// w + 4, .., a lane two or fewer dimensions; sums in a fixed order.
template <int D, int MT>
__global__ __launch_bounds__(256) void window_join_kernel(const WindowArgs a, const WindowParts parts,
                                                          int slots) {
    __shared__ float s_o[4][D];
    const WindowShape &s = a.s;
    const int G = s.H / s.HK, hk = blockIdx.x % s.HK, slot = blockIdx.x / s.HK, r = blockIdx.y;
    const int lane = lane_id(), wave = threadIdx.x >> 6;
    const size_t stride = (size_t)slots * s.HK * MT, at = (size_t)blockIdx.x * MT + r;
    // every part's maximum and sum, a part a lane (the rows of unused tiles are never read)
    const Located t = locate(a.offsets, nullptr, s.B, s.T, G, MT, slot);
    const int R = (slot - t.slot0) * MT + r;
    if (!t.found || R >= t.n * G) return;
    float m = -INFINITY, l = 0.f;
    if (lane < parts.n) {
        m = parts.ml[(lane * stride + at) * 2];
        l = parts.ml[(lane * stride + at) * 2 + 1];
    }
    // all parts of a bad sequence say the same: NaN rows, or (+inf) untouched ones
    const float m0 = readlane_f(m, 0);
    if (m0 == INFINITY) return;
    float top = m;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
    const float f = __builtin_amdgcn_exp2f(m - top);  // top is finite: some part sees the row itself
    float sum = f * l;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d, 64);
    constexpr int E = (D + 63) / 64;
    float o[E] = {};
#pragma unroll 4
    for (int p = wave; p < parts.n; p += 4) {
        const float fp = __shfl(f, p, 64);
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (lane + 64 * e < D) o[e] += fp * parts.o[(p * stride + at) * D + lane + 64 * e];
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (lane + 64 * e < D) s_o[wave][lane + 64 * e] = o[e];
    __syncthreads();
    const int d = threadIdx.x, i = R / G;
    if (d >= D) return;
    const float y = ((s_o[0][d] + s_o[1][d]) + (s_o[2][d] + s_o[3][d])) / sum;
    static_cast<__bf16 *>(a.out)[((size_t)(t.lo + i) * s.H + hk * G + (R - i * G)) * D + d] =
        (__bf16)(m0 == m0 ? y : m0);
}

// ---- host

static bool covers(const bole_window_dims_t &d) {
    return d.dtype == BOLE_DTYPE_BF16 && !(d.flags & BOLE_FLAG_FORCE_GENERIC) &&
           (d.head_dim == 64 || d.head_dim == 96 || d.head_dim == 128) && d.batch > 0;
}

// Form and split of a call, from its sizes alone: the tokens form up to 32 packed rows a
// sequence on average; parts so that 512 workgroups (two a CU) run, each with 256 keys or more.
struct WindowPlan {
    bool tokens;
    int tile, slots, parts;
};

static WindowPlan plan(const bole_window_dims_t &d) {
    WindowPlan p;
    const int64_t G = d.heads / d.kv_heads, rows = d.total_rows * G;
    p.tokens = rows <= 32LL * d.batch;
    p.tile = p.tokens ? kTokenTile : kRowTile;
    p.slots = (int)(rows / p.tile + d.batch);
    const int64_t cached = (int64_t)d.max_pages * d.page_size;
    const int64_t seen = (cached < (int64_t)d.window + d.sinks ? cached : (int64_t)d.window + d.sinks) + 1;
    const int64_t base = (int64_t)p.slots * d.kv_heads;
    int64_t n = (512 + base - 1) / base;
    if (n > (seen + 255) / 256) n = (seen + 255) / 256;
    p.parts = (int)(n > 64 ? 64 : n < 1 ? 1 : n);
    return p;
}

size_t window_workspace(const bole_window_dims_t &d) {
    if (!covers(d)) return 0;
    const WindowPlan p = plan(d);
    if (p.parts == 1) return 0;
    return (size_t)p.parts * p.slots * d.kv_heads * p.tile * (d.head_dim + 2) * sizeof(float);
}

bool window_mfma_applies(const bole_window_dims_t &d, const WindowArgs &a) {
    uintptr_t bits = 0;
    for (const void *p : {a.q, a.k, a.v, a.k_cache, a.v_cache, static_cast<const void *>(a.out)})
        bits |= reinterpret_cast<uintptr_t>(p);
    return covers(d) && bits % 16 == 0;
}

template <int D>
static hipError_t launch_width(const WindowArgs &a, const bole_window_dims_t &d, const WindowPlan &p,
                               const WindowParts &parts, hipStream_t stream) {
    const dim3 grid((unsigned)(p.slots * d.kv_heads), (unsigned)p.parts), block(256);
    if (p.tokens)
        window_tokens_kernel<D><<<grid, block, 0, stream>>>(a, parts, p.slots);
    else
        window_rows_kernel<D><<<grid, block, 0, stream>>>(a, parts, p.slots);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && p.parts > 1) {
        if (p.tokens)
            window_join_kernel<D, kTokenTile><<<dim3(grid.x, kTokenTile), block, 0, stream>>>(a, parts, p.slots);
        else
            window_join_kernel<D, kRowTile><<<dim3(grid.x, kRowTile), block, 0, stream>>>(a, parts, p.slots);
        e = hipGetLastError();
    }
    return e;
}

hipError_t launch_window_mfma(const WindowArgs &a, const bole_window_dims_t &d, void *workspace,
                              hipStream_t stream) {
    const WindowPlan p = plan(d);
    WindowParts parts = {static_cast<float *>(workspace), nullptr, p.parts};
    if (p.parts > 1)
        parts.ml = parts.o + (size_t)p.parts * p.slots * d.kv_heads * p.tile * d.head_dim;
    switch (d.head_dim) {
        case 64: return launch_width<64>(a, d, p, parts, stream);
        case 96: return launch_width<96>(a, d, p, parts, stream);
        default: return launch_width<128>(a, d, p, parts, stream);
    }
}

}  // namespace bole
