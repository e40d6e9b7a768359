// window_tile.h - what the matrix-core kernels of windowed attention share: the row tiles of a
// call, the list of keys a tile runs over, who sees which of them, and the parts of a split call.
#pragma once

#include "window_device.h"

namespace bole {

constexpr int kKeys = 64;        // keys a tile

// Where the unnormalised parts of a split call go: O [parts][tiles][MT][D], then (m, l)
// [parts][tiles][MT][2]. In place of a sum, which is not negative, stands kNanRow for a sequence
// whose rows become NaN and kLeftRow for one that is not touched.
constexpr float kNanRow = -1.f, kLeftRow = -2.f;
struct WindowParts {
    float *o, *ml;
    int n;         // parts of the key list
};

// How a call runs: form, rows a workgroup, row tiles (slots), parts of the key list.
struct WindowPlan {
    bool f32, tokens;
    int tile, slots, parts;
};

hipError_t launch_window_f32(const WindowArgs &a, const WindowPlan &p, const WindowParts &parts,
                             hipStream_t stream);

// Row tile of a workgroup and the key list it runs over.
struct RowTile {
    int b, lo, n, tile, slot0;       // sequence, its rows, tile within it, its first slot
    int status, len;
    int i0, i1;                      // rows (before packing) of the tile: [i0, i1)
    int n1, n2, n3, n4, w0, o2;      // key list: sinks, window from w0, own sinks, own rows from o2
    int own0, total, all_from;       // first own key (on a tile's edge), keys; first position every
                                     // row's window holds
};

// A value that every lane has, as a scalar: divisions end in vector registers, and all that is
// worked out from them would.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

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
    t.own0 = (t.n1 + t.n2 + kKeys - 1) & ~(kKeys - 1);
    t.total = t.own0 + t.n3 + t.n4;
}

// Row tile `slot` of a call: sequence b's tiles (MT packed rows, G to a row; at least one) lie
// behind those of the sequences before it, so the slots that are nobody's are the last ones. (In
// turn with the others they cost more than their exit: 64 sequences of one whole tile and one spare
// slot each took 251 us, against 190 of one.) per: the sequence's cached tokens.
struct Slot {
    bool found, ordered;            // found: b owns the slot; ordered: the offsets are
    int b, lo, n, slot0, per;       // sequence, its rows, its first slot
};

template <int MT>
__device__ __forceinline__ Slot find_slot(const WindowArgs &a, int G, int slot) {
    const int B = a.s.B;
    bool bad = false;
    Slot l = {false, true, 0, 0, 0, 0, 0};
    int before = 0;
    for (int c0 = 0; c0 < B; c0 += 64 * kAtOnce) {
        int lo[kAtOnce], hi[kAtOnce], len[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int x = min(c0 + 64 * j + lane_id(), B - 1);
            lo[j] = a.offsets[x], hi[j] = a.offsets[x + 1], len[j] = a.cache_len[x];
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int c = c0 + 64 * j;
            if (c >= B) break;
            bad |= lo[j] < 0 || hi[j] < lo[j] || hi[j] > a.s.T;
            const int own = c + lane_id() < B ? max(1, (int)(((uint32_t)(hi[j] - lo[j]) * G + MT - 1) / MT)) : 0;
            const int end = before + wave_sum_up(own);
            const int at = uniform((int)__popcll(__ballot(c + lane_id() < B && end <= slot)));
            if (!l.found && at < min(64, B - c)) {
                l.found = true;
                l.b = c + at;
                l.lo = __builtin_amdgcn_readlane(lo[j], at);
                l.n = __builtin_amdgcn_readlane(hi[j], at) - l.lo;
                l.slot0 = __builtin_amdgcn_readlane(end - own, at);
                l.per = __builtin_amdgcn_readlane(len[j], at);
            }
            before = __builtin_amdgcn_readlane(end, 63);
        }
    }
    l.ordered = !__any(bad);
    l.found = l.found && l.ordered;
    return l;
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
    const Slot l = find_slot<MT>(a, G, slot);
    if (!l.found) {
        if (!l.ordered && report && slot == 0 && a.status)
            for (int b = lane; b < s.B; b += 64) a.status[b] = BOLE_TREE_BAD_SIZE;
        return false;
    }
    t.b = l.b, t.lo = l.lo, t.n = l.n, t.slot0 = l.slot0, t.len = l.per;
    t.tile = slot - t.slot0;
    if (t.n == 0 && t.tile == 0 && report && lane == 0 && a.status) a.status[t.b] = BOLE_TREE_OK;
    if (t.tile * MT >= t.n * G) return false;
    t.i0 = uniform(t.tile * MT / G);
    t.i1 = min(t.n, uniform((t.tile * MT + MT + G - 1) / G));
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

// Where part `part` of `n` of the tiles begins (n <= 64, and fewer than 2^25 tiles).
__device__ __forceinline__ int part_edge(int tiles, int part, int n) {
    return uniform((int)((uint32_t)tiles * (uint32_t)part / (uint32_t)n));
}

__device__ __forceinline__ int cached_position(const RowTile &t, int x) {
    return x < t.n1 ? x : t.w0 + (x - t.n1);
}

__device__ __forceinline__ int own_row(const RowTile &t, int x) {
    const int j = x - t.own0;
    return j < t.n3 ? j : t.o2 + (j - t.n3);
}

// Page of the lane's key of the tile from x0 on, as the table has it; 0 for the call's own rows.
__device__ __forceinline__ int key_page(const WindowShape &s, const int32_t *__restrict__ table,
                                        const RowTile &t, int x0) {
    if (x0 >= t.own0) return 0;
    return table[cached_position(t, min(x0 + lane_id(), t.n1 + t.n2 - 1)) >> s.page_shift];
}

// Row (of D elements) of the lane's key of the tile from x0 on: in the cache's [page][head][slot]
// order, or in the call's k and v. Slots past the end of either part repeat its last key. A page
// that is not in the cache stands for its last one: the first loads go out before the sequence's
// pages are known to be valid, and are dropped if they are not. At 128 bytes a row and more, 32
// bits number more rows than memory holds.
__device__ __forceinline__ uint32_t key_row(const WindowShape &s, const RowTile &t, int hk, int x0,
                                            int page) {
    const int x = x0 + lane_id();
    if (x0 >= t.own0) return (uint32_t)(t.lo + own_row(t, min(x, t.total - 1))) * s.HK + hk;
    const uint32_t slot = cached_position(t, min(x, t.n1 + t.n2 - 1)) & ((1 << s.page_shift) - 1);
    return ((min((uint32_t)page, (uint32_t)s.pages - 1) * s.HK + hk) << s.page_shift) + slot;
}

// Where a tile's keys and values are: in the call, or in the cache. (The addresses are pinned to
// registers: the compiler would choose between their places in memory instead, and load one in
// every tile.) k, v: sixteen bytes at element `off`.
template <typename T>
struct KeySides {
    typedef T piece __attribute__((ext_vector_type(16 / sizeof(T))));
    uint64_t k0, v0, k1, v1;
    __device__ __forceinline__ explicit KeySides(const WindowArgs &a)
        : k0((uint64_t)a.k_cache), v0((uint64_t)a.v_cache), k1((uint64_t)a.k), v1((uint64_t)a.v) {
        asm volatile("" : "+s"(k0), "+s"(v0), "+s"(k1), "+s"(v1));
    }
    static __device__ __forceinline__ piece load(uint64_t base, size_t off) {
        return *(const __attribute__((address_space(1))) piece *)(base + off * sizeof(T));
    }
    __device__ __forceinline__ piece k(bool own, size_t off) const { return load(own ? k1 : k0, off); }
    __device__ __forceinline__ piece v(bool own, size_t off) const { return load(own ? v1 : v0, off); }
};

// Lane `from`'s value of x.
__device__ __forceinline__ uint32_t lane_value(uint32_t x, int from) {
    return (uint32_t)__builtin_amdgcn_ds_bpermute(4 * from, (int)x);
}

// Whether every row of the tile sees all 64 keys from x0 on.
__device__ __forceinline__ bool tile_open(const RowTile &t, bool tree, int x0) {
    const int x1 = x0 + kKeys;
    if (x0 < t.own0)
        return x1 <= t.n1 || (x0 >= t.n1 && x1 <= t.n1 + t.n2 && t.w0 + (x0 - t.n1) >= t.all_from);
    if (tree || x0 < t.own0 + t.n3 || x1 > t.total) return false;
    const int j = own_row(t, x0);
    return j + kKeys - 1 <= t.i0 && t.len + j >= t.all_from;
}

__device__ __forceinline__ uint64_t bits_below(int n) {
    return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}

// The keys x0 .. x0 + 63 that a query sees, as bits: row i of its sequence, window from position
// qe on, own nodes qmask for trees. Each part of the list shows it an interval (or the path).
__device__ __forceinline__ uint64_t seen_keys(const RowTile &t, bool tree, int i, int qe, uint64_t qmask,
                                              int x0) {
    const int from = max(qe, 0);
    if (x0 < t.own0)
        return bits_below(t.n1 - x0) |
               (bits_below(t.n1 + t.n2 - x0) & ~bits_below(t.n1 - x0 + max(0, from - t.w0)));
    if (tree) return qmask;  // at most 64 nodes: one tile
    const int sink = t.own0 - x0, own = sink + t.n3;
    return (bits_below(sink + min(t.n3, i + 1)) & ~bits_below(sink)) |
           (bits_below(own + min(t.n4, i + 1 - t.o2)) & ~bits_below(own + max(0, from - t.len - t.o2)));
}

constexpr float kLog2e = 1.4426950408889634f;

// Joins the parts of a split call (at most 64): a workgroup a row, wavefront w takes parts w,
// w + 4, .., a lane two or fewer dimensions; sums in a fixed order.
template <typename T, int D, int MT>
__global__ __launch_bounds__(256) void window_join_kernel(const WindowArgs a, const WindowParts parts,
                                                          int slots) {
    __shared__ float s_o[4][D];
    const WindowShape &s = a.s;
    const int G = s.H / s.HK, hk = blockIdx.x % s.HK, slot = blockIdx.x / s.HK, r = blockIdx.y;
    const int lane = lane_id(), wave = threadIdx.x >> 6;
    const size_t stride = (size_t)slots * s.HK * MT, at = (size_t)blockIdx.x * MT + r;
    // every part's maximum and sum, a part a lane (the rows of unused tiles are never read)
    const Slot t = find_slot<MT>(a, G, slot);
    const int R = (slot - t.slot0) * MT + r;
    if (!t.found || R >= t.n * G) return;
    float m = -INFINITY, l = 0.f;
    if (lane < parts.n) {
        m = parts.ml[(lane * stride + at) * 2];
        l = parts.ml[(lane * stride + at) * 2 + 1];
    }
    // (all parts of a bad sequence say the same)
    const float l0 = readlane_f(l, 0);
    if (l0 == kLeftRow) return;
    float top = m;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
    const float f = __builtin_amdgcn_exp2f(m - top);
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
    static_cast<T *>(a.out)[((size_t)(t.lo + i) * s.H + hk * G + (R - i * G)) * D + d] =
        (T)(l0 == kNanRow ? __builtin_nanf("") : y);
}

}  // namespace bole
