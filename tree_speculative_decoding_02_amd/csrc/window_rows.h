// window_rows.h - the two forms of workgroup of bf16 attention over a paged cache (window_mfma.hip),
// for windowed attention and for attention behind shared prefixes. Which rows a workgroup has and
// which keys they see is `Keys`:
//   args(), find<MT>(..) (the row tile of a slot and its key list), table(b) (its pages),
//   pages_status(t, x0, x1) (whether the pages of its keys exist, at least of entries x0 .. x1 - 1 of
//   the list);  kOwnRows: the rows' own sequences and what they see beyond the shared
//   prefix;  kSplit: results always go to the parts, [part][row][head], for another kernel to join.
#pragma once

#include "window_tile.h"

namespace bole {

typedef float f32x16 __attribute__((ext_vector_type(16)));

// LDS row strides in elements: K rows 16 bytes past a multiple of 256 apart or an odd number
// of 16-byte pieces (16 rows' pieces in distinct banks), V rows 64 or 192 bytes past one (the
// four rows of a transposing read in distinct quarters).
template <int D> struct Pad {
    static constexpr int K = D + 8;
    static constexpr int V = D == 128 ? 160 : 96;
};

// The factor of q . k in the exponent, positive, so that the largest product is the largest score:
// a scale's sign goes to the query (and a scale of 0 makes it 0).
template <int N>
__device__ __forceinline__ float query_scale(float scale, bf16x8 (&q)[N]) {
    if (scale > 0.f) return scale * kLog2e;
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = scale < 0.f ? -q[i] : q[i] * (__bf16)0.f;
    return scale < 0.f ? -scale * kLog2e : 1.f;
}

// Exponentials are taken from a reference m, which moves to the row's largest score so far once
// that is 8 above it: until then they stay below 2^8, which costs neither their bf16 roundings
// nor the fp32 sums anything, and most tiles do not touch the accumulators.
template <typename A, int N>
__device__ __forceinline__ void move_reference(float top, float &m, float &l, A (&acc)[N]) {
    const float next = fmaxf(m, top);
    if (!__any(next > m + 8.f)) return;
    const float keep = __builtin_amdgcn_exp2f(m - (next == -INFINITY ? 0.f : next));
    l *= keep;
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] *= keep;
    m = next;
}

// Also built for two prompts of 8192 tokens, at 361 to 367 us this way: one tile's exponentials
// between the next one's score products (391, with fewer loads in flight), eight wavefronts for 256
// rows (366), keys stored to LDS before or amid the second product (370), and without reading K's
// pieces ahead (376).
template <int D>
constexpr int kRowsLds = 2 * kKeys * (Pad<D>::K + Pad<D>::V) * 2;  // bytes

template <int D, class Keys>
__device__ __forceinline__ void rows_body(const Keys &keys, const WindowParts &parts, int slots, int block,
                                          int part, char *lds) {
    constexpr int CH = D / 8, PER = kKeys * CH / 256, KP = Pad<D>::K, VP = Pad<D>::V;
    __bf16(*s_k)[kKeys * KP] = reinterpret_cast<__bf16(*)[kKeys * KP]>(lds);
    __bf16(*s_v)[kKeys * VP] = reinterpret_cast<__bf16(*)[kKeys * VP]>(lds + 2 * kKeys * KP * 2);
    const WindowArgs &a = keys.args();
    const WindowShape &s = a.s;
    const int tid = threadIdx.x, lane = lane_id(), wave = uniform(tid >> 6), G = s.H / s.HK;
    const int slot = uniform(block / s.HK), hk = block - slot * s.HK;
    const bool tree = Keys::kOwnRows && a.parent != nullptr;
    RowTile t;
    uint64_t node_mask = 0;
    int node_depth = 0;
    const bool work = keys.template find<kRowTile>(G, slot, hk == 0 && part == 0 && wave == 0, t, node_mask,
                                                   node_depth);
    if (!work) return;
    const int col = lane & 31, hh = lane >> 5;
    const int R = t.tile * kRowTile + wave * 32 + col;
    const bool live = R < t.n * G;
    const int i = live ? R / G : 0, gq = live ? R - i * G : 0;
    const size_t row_off = ((size_t)(t.lo + i) * s.H + hk * G + gq) * D;
    __bf16 *out = static_cast<__bf16 *>(a.out) + row_off;
    const size_t part_row = Keys::kSplit ? part * (size_t)s.T * s.H + row_off / D
                                         : ((size_t)part * slots * s.HK + block) * kRowTile + wave * 32 + col;
    auto give_up = [&]() {
        const bool fill = t.status != BOLE_TREE_BAD_SIZE;
        if (Keys::kSplit || parts.n > 1) {
            if (live && hh == 0) parts.ml[part_row * 2 + 1] = fill ? kNanRow : kLeftRow;
        } else if (live && fill) {
            for (int e = hh; e < D; e += 2) out[e] = (__bf16)__builtin_nanf("");
        }
    };
    const bool report = Keys::kOwnRows && hk == 0 && part == 0 && t.tile == 0 && tid == 0 && a.status;
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
    const int32_t *table = keys.table(t.b);
    const int tiles = (t.total + kKeys - 1) / kKeys;
    const int first = part_edge(tiles, part, parts.n), last = part_edge(tiles, part + 1, parts.n);

    // Lane x holds the page and then the row of the tile's key x, `row` the rows that the thread
    // brings: pages two tiles ahead of the loads, rows one, as each is a trip through memory or LDS.
    const KeySides<__bf16> sides(a);
    int page = 0;
    uint32_t row[PER];
    bf16x8 kr[PER], vr[PER];
    auto find_rows = [&](int tile) {
        const uint32_t mine = key_row(s, t, hk, tile * kKeys, page);
#pragma unroll
        for (int j = 0; j < PER; ++j) row[j] = lane_value(mine, (tid + 256 * j) / CH);
        page = key_page(s, table, t, (tile + 1) * kKeys);
    };
    auto fetch = [&](int tile) {
        const bool own = tile * kKeys >= t.own0;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const size_t off = (size_t)row[j] * D + 8 * ((tid + 256 * j) % CH);
            kr[j] = sides.k(own, off);
            vr[j] = sides.v(own, off);
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
    float m = -INFINITY, l = 0.f;  // the exponentials' reference, and their sum
    const float c2 = query_scale(s.scale, qf);
    const bool busy = t.tile * kRowTile + wave * 32 < t.n * G;  // else it only stages
    if (first < last) {
        page = key_page(s, table, t, first * kKeys);
        find_rows(first);
        fetch(first);
        find_rows(min(first + 1, last - 1));
    }
    t.status = keys.pages_status(t, part_edge(tiles, part, parts.n) * kKeys, part_edge(tiles, part + 1, parts.n) * kKeys);
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
            if (tile + 1 < last) fetch(tile + 1);
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
                // K's pieces are read four products ahead
                __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
                for (int k = 0; k < D / 8 - 4; ++k) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                }
                __builtin_amdgcn_sched_group_barrier(0x008, 4, 0);
                float top = -INFINITY;
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
                top = max32(top);
                move_reference(top * c2, m, l, acc);
                const float base = m == -INFINITY ? 0.f : m;  // (nothing seen: exponentials of 0)
#pragma unroll
                for (int sub = 0; sub < 2; ++sub)
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        z[sub][r] = __builtin_amdgcn_exp2f(fmaf(z[sub][r], c2, -base));
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
            if (tile + 1 < last) {
                stage(buf ^ 1);
                find_rows(min(tile + 2, last - 1));
            }
            lds_barrier();
        } while (++tile < last);
    }
    l = sum32(l);
    if (!live) return;
    if (Keys::kSplit || parts.n > 1) {
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

// Two workgroups a CU: 8 single tokens 29 us against 36 with registers for one, 64 of them equal.
template <int D>
constexpr int kTokensLds = 4 * kKeys * Pad<D>::V * 2;  // bytes

template <int D, class Keys>
__device__ __forceinline__ void tokens_body(const Keys &keys, const WindowParts &parts, int slots, int block,
                                            int part, char *s_mem) {
    constexpr int CH = D / 8, VP = Pad<D>::V, VPER = kKeys * CH / 64;
    constexpr int JOIN = 4 * 16 * (D + 4) * 4;  // the last merge: sums, then (m, l), over the values
    static_assert(JOIN + 4 * 16 * 2 * 4 <= kTokensLds<D>, "LDS");
    float(*s_ml)[16][2] = reinterpret_cast<float(*)[16][2]>(s_mem + JOIN);
    const WindowArgs &a = keys.args();
    const WindowShape &s = a.s;
    const int tid = threadIdx.x, lane = lane_id(), wave = uniform(tid >> 6), G = s.H / s.HK;
    const int slot = uniform(block / s.HK), hk = block - slot * s.HK;
    const bool tree = Keys::kOwnRows && a.parent != nullptr;
    RowTile t;
    uint64_t node_mask = 0;
    int node_depth = 0;
    const bool work = keys.template find<kTokenTile>(G, slot, hk == 0 && part == 0 && wave == 0, t, node_mask,
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
    // row r of the tile (row R of the sequence) in the parts
    auto part_row = [&](int r, int R) {
        return Keys::kSplit ? part * (size_t)s.T * s.H + row_offset(R) / D
                            : ((size_t)part * slots * s.HK + block) * kTokenTile + r;
    };
    auto give_up = [&]() {
        const bool fill = t.status != BOLE_TREE_BAD_SIZE;
        if (Keys::kSplit || parts.n > 1) {
            if (live && g == 0 && wave == 0)
                parts.ml[part_row(col, R) * 2 + 1] = fill ? kNanRow : kLeftRow;
        } else if (live && fill) {
            __bf16 *o = static_cast<__bf16 *>(a.out) + row_offset(R);
            for (int e = wave * 4 + g; e < D; e += 16) o[e] = (__bf16)__builtin_nanf("");
        }
    };
    const bool report = Keys::kOwnRows && hk == 0 && part == 0 && t.tile == 0 && tid == 0 && a.status;
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
    const int32_t *table = keys.table(t.b);
    const int tiles = (t.total + kKeys - 1) / kKeys;
    const int first = part_edge(tiles, part, parts.n) + wave, last = part_edge(tiles, part + 1, parts.n);
    __bf16 *s_v = reinterpret_cast<__bf16 *>(s_mem) + wave * kKeys * VP;

    // a lane's keys: for K, key 16 r + col of the tile (r = 0..3), 16-byte pieces 4 ks + g; for
    // V, piece e = lane + 64 j of the tile's kKeys x CH pieces
    bf16x8 kf[4][D / 32], vr[VPER];
    int page = -1;
    const KeySides<__bf16> sides(a);
    auto fetch = [&](int tile) {
        const bool own = tile * kKeys >= t.own0;
        const uint32_t mine = key_row(s, t, hk, tile * kKeys, page);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const size_t off = (size_t)lane_value(mine, 16 * r + col) * D + 8 * g;
#pragma unroll
            for (int ks = 0; ks < D / 32; ++ks) kf[r][ks] = sides.k(own, off + 32 * ks);
        }
#pragma unroll
        for (int j = 0; j < VPER; ++j) {
            const int e = lane + 64 * j;
            vr[j] = sides.v(own, (size_t)lane_value(mine, e / CH) * D + 8 * (e % CH));
        }
    };
    f32x4 acc[D / 16];
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt) acc[dt] = (f32x4)0.f;
    float m = -INFINITY, l = 0.f;  // the exponentials' reference, and their sum
    const float c2 = query_scale(s.scale, qf);
    if (first < last) {
        page = key_page(s, table, t, first * kKeys);
        fetch(first);
        page = key_page(s, table, t, (first + 4) * kKeys);
    }
    t.status = keys.pages_status(t, part_edge(tiles, part, parts.n) * kKeys, part_edge(tiles, part + 1, parts.n) * kKeys);
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
                page = key_page(s, table, t, (tile + 8) * kKeys);
            }
            float top = -INFINITY;
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
            top = max16(top);
            top = max32(top);
            move_reference(top * c2, m, l, acc);
            const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    z[r][e] = __builtin_amdgcn_exp2f(fmaf(z[r][e], c2, -base));
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
    l = sum16(l);
    l = sum32(l);

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
    if (Keys::kSplit || parts.n > 1) {
        const size_t at = part_row(r, t.tile * kTokenTile + r);
        if (d0 == 0) {
            parts.ml[at * 2] = mm;
            parts.ml[at * 2 + 1] = ll;
        }
#pragma unroll
        for (int e = 0; e < D / 16; ++e) parts.o[at * D + d0 + e] = o[e];
        return;
    }
    __bf16 *dst = static_cast<__bf16 *>(a.out) + row_offset(t.tile * kTokenTile + r) + d0;
    const float inv = 1.f / ll;
#pragma unroll
    for (int e = 0; e < D / 16; ++e) dst[e] = (__bf16)(o[e] * inv);
}

}  // namespace bole
