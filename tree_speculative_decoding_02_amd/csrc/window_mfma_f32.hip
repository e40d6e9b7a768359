// window_mfma_f32.hip - windowed attention on the fp32 matrix instructions, head widths 64, 96
// and 128. The same shape as the bf16 rows form (window_mfma.hip): S^T = K Q^T, a query a lane
// group of 16 lanes' column, and the exponentials in registers are the right operand of
// O^T = V^T P^T as they are: of v_mfma_f32_16x16x4_f32's results lane group g holds rows
// 4 g .. 4 g + 3, and with step r of a product taking keys {4 g + r} from every group, register
// r is that step's operand.
//
// One workgroup: 64 rows, 16 a wavefront, keys and values staged in LDS 64 at a time, the next
// 64 in registers meanwhile. The fp32 matrix rate (a sixteenth of bf16's) bounds prompts and
// trees, the cache's bytes single tokens: 32 heads over 8 of 128, a window of 4096, 64 single
// tokens 442 us (4.2 TB/s), 64 trees of up to 32 nodes 1077 us (45 TFLOP/s, the matrix instructions
// at work half of the time); two prompts of 2048 tokens, window 1024, 679 us (102 TFLOP/s).
#include "window_tile.h"
#include "launch.h"

namespace bole {

constexpr int kF32Tile = 64;

template <int D>
__global__ __launch_bounds__(256, 2) void window_f32_kernel(const WindowArgs a, const WindowParts parts,
                                                            int slots) {
    // row strides: 16 rows' 16-byte pieces (K), and four rows a multiple of four apart (V), lie in
    // distinct banks
    constexpr int CH = D / 4, PER = kKeys * CH / 256, ST = D + 4;
    __shared__ __align__(16) float s_k[kKeys * ST];
    __shared__ __align__(16) float s_v[kKeys * ST];
    const WindowShape &s = a.s;
    const int tid = threadIdx.x, lane = lane_id(), wave = uniform(tid >> 6), G = s.H / s.HK;
    const int slot = uniform(blockIdx.x / s.HK), hk = blockIdx.x - slot * s.HK, part = blockIdx.y;
    const bool tree = a.parent != nullptr;
    RowTile t;
    uint64_t node_mask = 0;
    int node_depth = 0;
    if (!find_tile<kF32Tile>(a, G, slot, hk == 0 && part == 0 && wave == 0, t, node_mask, node_depth))
        return;
    const int col = lane & 15, g = lane >> 4;
    const int R = t.tile * kF32Tile + wave * 16 + col;
    const bool live = R < t.n * G;
    const int i = live ? R / G : 0;
    const size_t row_off = ((size_t)(t.lo + i) * s.H + hk * G + (live ? R - i * G : 0)) * D;
    float *out = static_cast<float *>(a.out) + row_off;
    const size_t part_row = ((size_t)part * slots * s.HK + blockIdx.x) * kF32Tile + wave * 16 + col;
    auto give_up = [&]() {
        const bool fill = t.status != BOLE_TREE_BAD_SIZE;
        if (parts.n > 1) {
            if (live && g == 0) parts.ml[part_row * 2 + 1] = fill ? kNanRow : kLeftRow;
        } else if (live && fill) {
            for (int e = g; e < D; e += 4) out[e] = __builtin_nanf("");
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
    f32x4 qf[D / 16];
#pragma unroll
    for (int d = 0; d < D / 16; ++d) {
        qf[d] = (f32x4)0.f;
        if (live) qf[d] = *reinterpret_cast<const f32x4 *>(static_cast<const float *>(a.q) + row_off + 16 * d + 4 * g);
    }
    const int32_t *table = a.page_table + (size_t)t.b * s.max_pages;
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
    t.status = pages_status(a, t.b, t.len);
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
    if (parts.n > 1) {
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

template <int D>
static hipError_t launch_width(const WindowArgs &a, const WindowPlan &p, const WindowParts &parts,
                               hipStream_t stream) {
    const unsigned tiles = (unsigned)(p.slots * a.s.HK);
    window_f32_kernel<D><<<dim3(tiles, (unsigned)p.parts), dim3(256), 0, stream>>>(a, parts, p.slots);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && p.parts > 1) {
        window_join_kernel<float, D, kF32Tile><<<dim3(tiles, kF32Tile), dim3(256), 0, stream>>>(a, parts, p.slots);
        e = hipGetLastError();
    }
    return e;
}

hipError_t launch_window_f32(const WindowArgs &a, const WindowPlan &p, const WindowParts &parts,
                             hipStream_t stream) {
    switch (a.s.D) {
        case 64: return launch_width<64>(a, p, parts, stream);
        case 96: return launch_width<96>(a, p, parts, stream);
        default: return launch_width<128>(a, p, parts, stream);
    }
}

}  // namespace bole
