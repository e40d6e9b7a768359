// delta_device.h - device helpers shared by the gated delta rule's kernels: cumulative
// log-decays in fp64, sequence offsets, accepted paths.
//
// Gated delta rule, one head, state H [d_k][d_v]:
//     H' = a H,   u = b (v - H'^T k),   H <- H' + k u^T,   o = H^T q.
#pragma once

#include "bole_device.h"
#include "mfma_util.h"

namespace bole {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

typedef short s16x4 __attribute__((ext_vector_type(4)));

// Transposing LDS read: of each 16 lanes, lane i gets column i, rows 0..3, of the 4 x 16 block
// whose row r, columns 4c .. 4c + 3 lane 4r + c points to (8 bytes a lane).
__device__ __forceinline__ bf16x4 read_transposed(const __bf16 *p) {
    const s16x4 r = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4 *)(__attribute__((address_space(3))) void *)p);
    return __builtin_bit_cast(bf16x4, r);
}

__device__ __forceinline__ bf16x8 join(bf16x4 a, bf16x4 b) {
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// x of this lane and of the lane with bit 3, 4 or 5 of its number flipped, added up or the larger
// one: one or two vector instructions each, where a shuffle takes a round trip through LDS.
__device__ __forceinline__ float flip8(float x) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x128, 0xf, 0xf, false));
}

__device__ __forceinline__ float2 pair16(float x) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return {__uint_as_float(p[0]), __uint_as_float(p[1])};
}

__device__ __forceinline__ float2 pair32(float x) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return {__uint_as_float(p[0]), __uint_as_float(p[1])};
}

__device__ __forceinline__ float sum8(float x) { return x + flip8(x); }
__device__ __forceinline__ float sum16(float x) { const float2 p = pair16(x); return p.x + p.y; }
__device__ __forceinline__ float sum32(float x) { const float2 p = pair32(x); return p.x + p.y; }
__device__ __forceinline__ float max16(float x) { const float2 p = pair16(x); return fmaxf(p.x, p.y); }
__device__ __forceinline__ float max32(float x) { const float2 p = pair32(x); return fmaxf(p.x, p.y); }

// Barrier for data in LDS alone. __syncthreads also waits for every global load in flight, and
// with it a prefetch for the next step would end at the first barrier of this one.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

struct DeltaShape {
    int B, H, HK, DK, DV, T;  // sequences, value heads, key heads, widths, packed rows
};

// log2 of a decay. A decay of 0 (a reset) becomes 2^-10000: every product across it is 0 in
// fp32, and no difference of logarithms is infinity minus infinity. A NaN stays one.
__device__ __forceinline__ float log2_decay(float a) {
    const float l = log2f(a);
    return l < -10000.f ? -10000.f : l;
}

// How key rows are laid out for loads: of any width and address; in 16-byte parts, on 16-byte
// addresses; and of d_k = 8 RPL as well. (Parts against single elements, 128 steps of 32 heads:
// 96 x 96 in bf16 59.8 -> 55.2 us, 72 x 40 29.2 -> 23.1; one step 5.6 -> 3.7 and 6.4 -> 4.5.)
enum { kAnyRow = 0, kParts = 1, kExact = 2 };

// Lane's RPL key-row values, row rg RPL + i (zero past d_k).
template <typename TF, int RPL, int ROW>
struct RowPiece {
    TF x[RPL];
    __device__ __forceinline__ void load(const TF *p, int r0, int DK) {
        if constexpr (ROW != kAnyRow) {
            constexpr int V = 16 / sizeof(TF);
            typedef TF vec __attribute__((ext_vector_type(V)));
#pragma unroll
            for (int i = 0; i < RPL; i += V) {
                const bool in = ROW == kExact || r0 + i < DK;
                const vec t = *reinterpret_cast<const vec *>(p + (in ? r0 + i : 0));
#pragma unroll
                for (int j = 0; j < V; ++j) x[i + j] = in ? t[j] : (TF)0.f;
            }
        } else {
#pragma unroll
            for (int i = 0; i < RPL; ++i) x[i] = r0 + i < DK ? p[r0 + i] : (TF)0.f;
        }
    }
};

// Topology and cumulative log2-decay of a tree whose node i has parent p_loaded in lane i
// (as wave_topology_cumlog), the sum in fp64: pair weights are exponentials of differences
// of these sums, and after strong decays the sums are large while later differences are
// small (in fp32 a sum of 600 leaves an error of 3e-5 in every later pair weight).
struct WaveTopoD {
    uint64_t mask;
    int bad;
    double L;
};

__device__ __forceinline__ double shfl_f64(double x, int src) {
    const long long v = __double_as_longlong(x);
    return __longlong_as_double((long long)shfl_u64((uint64_t)v, src));
}

__device__ __forceinline__ WaveTopoD wave_topology_cumlog_f64(int p_loaded, float lg, int n) {
    const int lane = lane_id();
    const int p = lane < n ? p_loaded : -1;
    const bool bad_lane = lane < n && (p < -1 || p >= lane);
    WaveTopoD t;
    t.bad = __any(bad_lane) ? BOLE_TREE_BAD_PARENT : BOLE_TREE_OK;
    const bool live = lane < n && !t.bad;
    uint64_t m = live ? (1ull << lane) : 0ull;
    double acc = live ? (double)lg : 0.0;
    int anc = live ? p : -1;
    for (int r = 0; r < 6 && __any(anc >= 0); ++r) {
        const int src = anc < 0 ? lane : anc;
        const uint64_t m_up = shfl_u64(m, src);
        const double acc_up = shfl_f64(acc, src);
        const int anc_up = __shfl(anc, src, 64);
        if (anc >= 0) {
            m |= m_up;
            acc += acc_up;
            anc = anc_up;
        }
    }
    t.mask = m;
    t.L = acc;
    return t;
}

// Inclusive sum over lanes 0 .. lane, in fp64.
__device__ __forceinline__ double wave_sum_up_f64(double x) {
    const int lane = lane_id();
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double y = shfl_f64(x, lane >= d ? lane - d : lane);
        if (lane >= d) x += y;
    }
    return x;
}

// Inclusive sum over lanes 0 .. lane, in fp64, by moves within the vector registers.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_f64(double x) {
    const long long v = __double_as_longlong(x);
    const int lo = __builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false);
    const int hi = __builtin_amdgcn_update_dpp(0, (int)(v >> 32), CTRL, ROWS, 0xf, false);
    return __longlong_as_double(((long long)hi << 32) | (unsigned)lo);
}
__device__ __forceinline__ double scan_f64(double x) {
    x += dpp_f64<0x111, 0xf>(x);  // from 1, 2, 4 and 8 lanes before, within rows of 16
    x += dpp_f64<0x112, 0xf>(x);
    x += dpp_f64<0x114, 0xf>(x);
    x += dpp_f64<0x118, 0xf>(x);
    x += dpp_f64<0x142, 0xa>(x);  // a row's last lane to the next row,
    x += dpp_f64<0x143, 0xc>(x);  // lane 31 to the upper half
    return x;
}

// Inclusive sum over lanes 0 .. lane.
__device__ __forceinline__ int wave_sum_up(int x) {
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);  // from 1, 2, 4 and 8 lanes before,
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);  // within rows of 16
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);  // a row's last lane to the next row,
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);  // lane 31 to the upper half
    return x;
}

// Every workgroup looks through all offsets, 64 a load, so many loads at a time: attention of 1024
// single tokens over 256 cached ones 322 us with one, 306 with two, 293 with four, 289 with eight;
// of one token 10.9 and, with eight, 11.1.
constexpr int kAtOnce = 4;

// Whether all B + 1 offsets are ordered and inside [0, T] (wave-uniform; all lanes active).
__device__ __forceinline__ bool offsets_ordered(const int32_t *__restrict__ off, int B, int T) {
    bool bad = false;
    for (int c = 0; c < B; c += 64 * kAtOnce) {
        int lo[kAtOnce], hi[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int x = min(c + 64 * j + lane_id(), B - 1);
            lo[j] = off[x], hi[j] = off[x + 1];
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) bad |= lo[j] < 0 || hi[j] < lo[j] || hi[j] > T;
    }
    return !__any(bad);
}

// Tile `slot` of the packed rows, MT rows a tile: sequence b owns slots from floor(off[b] / MT) + b,
// at least one each (slots before the first sequence's are nobody's).
struct Located {
    bool found, ordered;       // found: b owns the slot; ordered: the offsets are
    int b, lo, n, slot0;       // sequence, its rows, its first slot
};

__device__ __forceinline__ Located locate(const int32_t *__restrict__ off, int B, int T, int MT, int slot) {
    bool bad = false;
    Located l = {false, true, -1, 0, 0, 0};
    for (int c0 = 0; c0 < B; c0 += 64 * kAtOnce) {
        int lo[kAtOnce], hi[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int x = min(c0 + 64 * j + lane_id(), B - 1);
            lo[j] = off[x], hi[j] = off[x + 1];
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int c = c0 + 64 * j;
            if (c >= B) break;
            bad |= lo[j] < 0 || hi[j] < lo[j] || hi[j] > T;
            // the sequences that start at or before the slot are the first ones
            const int many = (int)__popcll(__ballot(c + lane_id() < B && lo[j] / MT + c + lane_id() <= slot));
            if (many > 0) {
                const int at = __builtin_amdgcn_readfirstlane(many - 1);
                l.b = c + at;
                l.lo = __builtin_amdgcn_readlane(lo[j], at);
                l.n = __builtin_amdgcn_readlane(hi[j], at) - l.lo;
            }
        }
    }
    l.ordered = !__any(bad);
    l.found = l.ordered && l.b >= 0;
    l.slot0 = l.lo / MT + l.b;
    return l;
}

// Sequence that owns a packed row (ordered offsets), all lanes of a wavefront active.
struct RowOwner {
    bool found, ordered;
    int b, lo, n;
};

__device__ __forceinline__ RowOwner owner_of(const int32_t *__restrict__ off, int B, int T, int row) {
    bool bad = false;
    RowOwner o = {false, true, -1, 0, 0};
    for (int c0 = 0; c0 < B; c0 += 64 * kAtOnce) {
        int lo[kAtOnce], hi[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int x = min(c0 + 64 * j + lane_id(), B - 1);
            lo[j] = off[x], hi[j] = off[x + 1];
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int c = c0 + 64 * j;
            if (c >= B) break;
            bad |= lo[j] < 0 || hi[j] < lo[j] || hi[j] > T;
            // the sequences that start at or before the row are the first ones
            const int many = (int)__popcll(__ballot(c + lane_id() < B && lo[j] <= row));
            if (many > 0) {
                const int at = __builtin_amdgcn_readfirstlane(many - 1);
                o.b = c + at;
                o.lo = __builtin_amdgcn_readlane(lo[j], at);
                o.n = __builtin_amdgcn_readlane(hi[j], at) - o.lo;
            }
        }
    }
    o.ordered = !__any(bad);
    o.found = o.ordered && o.b >= 0 && row - o.lo < o.n;
    return o;
}

// The accepted path of tree b, validated by one wavefront with the rules of commit_kernel:
// lane m gets the packed row of path node m (-1 past the path), len is 0 for a bad tree.
struct WavePath {
    int row, len, status;
};

__device__ __forceinline__ WavePath wave_path(const int32_t *__restrict__ parent,
                                              const int32_t *__restrict__ node_offsets,
                                              const int32_t *__restrict__ accepted_idx,
                                              const int32_t *__restrict__ accepted_len, int b,
                                              int T, int max_path) {
    const int lane = lane_id();
    const TreeRange tr = tree_range(node_offsets, b, T);
    const int len_raw = accepted_len[b];
    int st = tr.status, len = 0, x = -1;
    if (st == BOLE_TREE_OK) {
        const int n = tr.n;
        const int p = lane < n ? parent[tr.lo + lane] : -1;
        const bool len_ok = len_raw >= 0 && len_raw <= max_path && len_raw <= n;
        x = (len_ok && lane < len_raw) ? accepted_idx[(size_t)b * max_path + lane] : -1;
        if (__any(lane < n && (p < -1 || p >= lane))) {
            st = BOLE_TREE_BAD_PARENT;
        } else if (!len_ok) {
            st = BOLE_TREE_BAD_PATH;
        } else {
            len = len_raw;
            const int px = __shfl(p, (x >= 0 && x < n) ? x : 0, 64);
            const int before = __shfl(x, lane > 0 ? lane - 1 : 0, 64);
            const int prev = lane == 0 ? -1 : before;
            if (__any(lane < len && (x < 0 || x >= n || px != prev))) st = BOLE_TREE_BAD_PATH;
        }
    }
    WavePath w;
    w.status = st;
    w.len = st == BOLE_TREE_OK ? len : 0;
    w.row = lane < w.len ? tr.lo + x : -1;
    return w;
}

}  // namespace bole
