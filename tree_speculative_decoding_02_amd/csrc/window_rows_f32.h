// window_rows_f32.h - the workgroup of fp32 attention over a paged cache (window_mfma_f32.hip), for
// windowed attention and for attention behind shared prefixes; `Keys` as in window_rows.h.
#pragma once

#include "window_tile.h"

namespace bole {

template <int D>
constexpr int kF32Lds = 2 * kKeys * (D + 4) * 4;  // bytes

template <int D, class Keys>
__device__ __forceinline__ void f32_body(const Keys &keys, const WindowParts &parts, int slots, int block,
                                         int part, char *lds) {
    // row strides: 16 rows' 16-byte pieces (K), and four rows a multiple of four apart (V), lie in
    // distinct banks
    constexpr int CH = D / 4, PER = kKeys * CH / 256, ST = D + 4;
    float *s_k = reinterpret_cast<float *>(lds), *s_v = s_k + kKeys * ST;
    const WindowArgs &a = keys.args();
    const WindowShape &s = a.s;
    const int tid = threadIdx.x, lane = lane_id(), wave = uniform(tid >> 6), G = s.H / s.HK;
    const int slot = uniform(block / s.HK), hk = block - slot * s.HK;
    const bool tree = Keys::kOwnRows && a.parent != nullptr;
    RowTile t;
    uint64_t node_mask = 0;
    int node_depth = 0;
    if (!keys.template find<kF32Tile>(G, slot, hk == 0 && part == 0 && wave == 0, t, node_mask, node_depth))
        return;
    const int col = lane & 15, g = lane >> 4;
    const int R = t.tile * kF32Tile + wave * 16 + col;
    const bool live = R < t.n * G;
    const int i = live ? R / G : 0;
    const size_t row_off = ((size_t)(t.lo + i) * s.H + hk * G + (live ? R - i * G : 0)) * D;
    float *out = static_cast<float *>(a.out) + row_off;
    const size_t part_row = Keys::kSplit ? part * (size_t)s.T * s.H + row_off / D
                                         : ((size_t)part * slots * s.HK + block) * kF32Tile + wave * 16 + col;
    auto give_up = [&]() {
        const bool fill = t.status != BOLE_TREE_BAD_SIZE;
        if (Keys::kSplit || parts.n > 1) {
            if (live && g == 0) parts.ml[part_row * 2 + 1] = fill ? kNanRow : kLeftRow;
        } else if (live && fill) {
            for (int e = g; e < D; e += 4) out[e] = __builtin_nanf("");
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
    f32x4 qf[D / 16];
#pragma unroll
    for (int d = 0; d < D / 16; ++d) {
        qf[d] = (f32x4)0.f;
        if (live) qf[d] = *reinterpret_cast<const f32x4 *>(static_cast<const float *>(a.q) + row_off + 16 * d + 4 * g);
    }
    const int32_t *table = keys.table(t.b);
    const int tiles = (t.total + kKeys - 1) / kKeys;
    const int first = part_edge(tiles, part, parts.n), last = part_edge(tiles, part + 1, parts.n);

    int page = 0;
    f32x4 kr[PER], vr[PER];
    const KeySides<float> sides(a);
    auto fetch = [&](int tile) {
        const bool own = tile * kKeys >= t.own0;
        const uint32_t mine = key_row(s, t, hk, tile * kKeys, page);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int e = tid + 256 * j;
            const size_t off = (size_t)lane_value(mine, e / CH) * D + 4 * (e % CH);
            kr[j] = sides.k(own, off);
            vr[j] = sides.v(own, off);
        }
    };
    auto stage = [&]() {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int e = tid + 256 * j, at = (e / CH) * ST + 4 * (e % CH);
            *reinterpret_cast<f32x4 *>(&s_k[at]) = kr[j];
            *reinterpret_cast<f32x4 *>(&s_v[at]) = vr[j];
        }
    };
    f32x4 acc[D / 16];
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt) acc[dt] = (f32x4)0.f;
    float m = -INFINITY, l = 0.f;
    const float c2 = s.scale * kLog2e;
    const bool busy = t.tile * kF32Tile + wave * 16 < t.n * G;  // else it only stages
    if (first < last) {
        page = key_page(s, table, t, first * kKeys);
        fetch(first);
        page = key_page(s, table, t, (first + 1) * kKeys);
    }
    t.status = keys.pages_status(t, first * kKeys, last * kKeys);
    if (report) a.status[t.b] = t.status;
    if (t.status != BOLE_TREE_OK) {
        give_up();
        return;
    }
    if (first < last) {
        int tile = first;
        do {
            lds_barrier();  // the last tile is read
            stage();
            lds_barrier();
            if (tile + 1 < last) {
                fetch(tile + 1);
                page = key_page(s, table, t, (tile + 2) * kKeys);
            }
            if (!busy) continue;
            const int x0 = tile * kKeys;
            f32x4 z[4];
#pragma unroll
            for (int kt = 0; kt < 4; ++kt) {
                z[kt] = (f32x4)0.f;
                const float *kp = &s_k[(16 * kt + col) * ST + 4 * g];
#pragma unroll
                for (int d = 0; d < D / 16; ++d) {
                    const f32x4 x = *reinterpret_cast<const f32x4 *>(kp + 16 * d);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        z[kt] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[r], qf[d][r], z[kt], 0, 0, 0);
                }
                z[kt] *= c2;
            }
            if (!tile_open(t, tree, x0)) {
                const uint64_t seen = seen_keys(t, tree, i, qe, qmask, x0) >> (4 * g);
#pragma unroll
                for (int kt = 0; kt < 4; ++kt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        z[kt][e] = ((uint32_t)(seen >> (32 * (kt >> 1))) >> (16 * (kt & 1) + e)) & 1u
                                       ? z[kt][e] : -INFINITY;
            }
            float top = -INFINITY;
#pragma unroll
            for (int kt = 0; kt < 4; ++kt)
#pragma unroll
                for (int e = 0; e < 4; ++e) top = fmaxf(top, z[kt][e]);
            top = max16(top);
            top = max32(top);
            const float next = fmaxf(m, top), base = next == -INFINITY ? 0.f : next;
            const float keep = __builtin_amdgcn_exp2f(m - base);
            m = next;
            l *= keep;
#pragma unroll
            for (int dt = 0; dt < D / 16; ++dt) acc[dt] *= keep;
#pragma unroll
            for (int kt = 0; kt < 4; ++kt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    z[kt][e] = __builtin_amdgcn_exp2f(z[kt][e] - base);
                    l += z[kt][e];
                }
#pragma unroll
            for (int kt = 0; kt < 4; ++kt)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float *vp = &s_v[(16 * kt + 4 * g + r) * ST + col];
#pragma unroll
                    for (int dt = 0; dt < D / 16; ++dt)
                        acc[dt] = __builtin_amdgcn_mfma_f32_16x16x4f32(vp[16 * dt], z[kt][r], acc[dt], 0, 0, 0);
                }
        } while (++tile < last);
    }
    l = sum16(l);
    l = sum32(l);
    if (!live) return;
    if (Keys::kSplit || parts.n > 1) {
        if (g == 0) {
            parts.ml[part_row * 2] = m;
            parts.ml[part_row * 2 + 1] = l;
        }
        float *o = parts.o + part_row * D;
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt) *reinterpret_cast<f32x4 *>(o + 16 * dt + 4 * g) = acc[dt];
        return;
    }
    const float inv = 1.f / l;
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt) *reinterpret_cast<f32x4 *>(out + 16 * dt + 4 * g) = acc[dt] * inv;
}

}  // namespace bole
