// delta_walk.hip - the gated delta rule token by token: the single-token step, the commit of
// an accepted path, and prompts of shapes that the chunked kernels do not take.
//
// One token, from state H (all in fp32):
//     w = H^T k, z = H^T q, u = b (v - a w), o = a z + (q . k) u, H <- a H + k u^T.
// Both products read the old state, so a token costs one pass over it; o needs no second one.
//
// A wavefront owns 8 CPL columns of one state and keeps all of their rows in registers: lane
// (rg, cg) = (lane / 8, lane % 8) holds rows rg RPL .. rg RPL + RPL - 1 of columns cg CPL ..
// cg CPL + CPL - 1. w and z are summed over the lane's rows, then over the eight row groups
// with three cross-lane steps. Nothing is shared between wavefronts: no LDS, no barrier.
// The state is read once and written once whatever the number of tokens, with non-temporal
// 16-byte accesses (a row's eight lanes cover 128 contiguous bytes).
//
// Step and commit are bound by the state's round trip through HBM: 128 sequences of 32 heads with
// 128 x 128 states, one token each, 95 us (5.7 TB/s), 64 accepted paths of trees of up to 64 nodes
// 42 us (5.2 TB/s); one sequence's step, a chain of loads and sums, 3.4 us in a graph. Tokens of a sequence
// cannot overlap here, so long prompts are bound by the chain of a token's products and
// exchanges; the chunked kernels take the shapes where that matters.
#include "delta_device.h"
#include "launch.h"

namespace bole {

enum { kWalkStep = 0, kWalkCommit = 1, kWalkPrefill = 2 };

struct WalkArgs {
    float *H0;
    const void *q, *k, *v;
    const float *gate, *beta;
    const int32_t *parent, *offsets, *accepted_idx, *accepted_len;
    void *out;
    int32_t *path_nodes, *status;
    DeltaShape s;
    int max_path;
};

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

template <int MODE, typename TF, int RPL, int CPL, int ROW>
__global__ __launch_bounds__(256) void delta_walk_kernel(const WalkArgs a, int units, int blocks) {
    typedef float hvec __attribute__((ext_vector_type(CPL)));
    const int lane = lane_id();
    const int wave = blockIdx.x * 4 + (threadIdx.x >> 6);
    const int unit = wave / blocks, cb = wave - unit * blocks;
    if (unit >= units) return;
    const int H = a.s.H, DK = a.s.DK, DV = a.s.DV;
    const int b = unit / H, h = unit - b * H, hk = h / (H / a.s.HK);

    const int rg = lane >> 3, c0 = (cb * 8 + (lane & 7)) * CPL, r0 = rg * RPL;
    const bool live = c0 < DV;  // CPL divides d_v: a lane's columns exist or do not together
    float *Hu = a.H0 + (size_t)unit * DK * DV + c0;
    hvec hr[RPL];
    auto load_state = [&]() {
#pragma unroll
        for (int i = 0; i < RPL; ++i) {
            hr[i] = (hvec)0.f;
            if (live && (ROW == kExact || r0 + i < DK))
                hr[i] = __builtin_nontemporal_load(
                    reinterpret_cast<const hvec *>(Hu + (size_t)(r0 + i) * DV));
        }
    };

    // the tokens: `row` of lane m is the m-th of a path, lo + m for the other modes
    int lo = b, n = 1, path_row = -1;
    if constexpr (MODE == kWalkCommit) {
        // the state is on its way while the path is checked (it is read for nothing if that fails)
        if (a.accepted_len[b] > 0) load_state();
        const WavePath p = wave_path(a.parent, a.offsets, a.accepted_idx, a.accepted_len, b, a.s.T,
                                     a.max_path);
        n = p.len;
        path_row = p.row;
        if (h == 0 && cb == 0) {
            if (lane == 0 && a.status) a.status[b] = p.status;
            if (a.path_nodes && lane < a.max_path)
                a.path_nodes[(size_t)b * a.max_path + lane] = p.row;
        }
    } else if constexpr (MODE == kWalkPrefill) {
        const bool ok = offsets_ordered(a.offsets, a.s.B, a.s.T);
        if (h == 0 && cb == 0 && lane == 0 && a.status)
            a.status[b] = ok ? BOLE_TREE_OK : BOLE_TREE_BAD_SIZE;
        lo = a.offsets[b];
        n = ok ? a.offsets[b + 1] - lo : 0;
    }
    if (n <= 0) return;

    const TF *q = static_cast<const TF *>(a.q), *k = static_cast<const TF *>(a.k),
             *v = static_cast<const TF *>(a.v);
    if constexpr (MODE != kWalkCommit) load_state();
    constexpr bool OUT = MODE != kWalkCommit;
    const size_t sk = (size_t)a.s.HK * DK, sv = (size_t)H * DV;
    RowPiece<TF, RPL, ROW> kn, qn;
    float vn[CPL], an, bn;
    auto fetch = [&](int t) {
        const int row = MODE == kWalkCommit ? __builtin_amdgcn_readlane(path_row, t) : lo + t;
        kn.load(k + row * sk + (size_t)hk * DK, r0, DK);
        if constexpr (OUT) qn.load(q + row * sk + (size_t)hk * DK, r0, DK);
#pragma unroll
        for (int c = 0; c < CPL; ++c)
            vn[c] = live ? to_f32(v[row * sv + (size_t)h * DV + c0 + c]) : 0.f;
        an = a.gate[(size_t)row * H + h];
        bn = a.beta[(size_t)row * H + h];
    };
    fetch(0);
    for (int t = 0; t < n; ++t) {
        RowPiece<TF, RPL, ROW> kc = kn, qc = qn;
        float vc[CPL], w[CPL], z[CPL], kq = 0.f;
        const float ac = an, bc = bn;
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            vc[c] = vn[c];
            w[c] = z[c] = 0.f;
        }
        if (t + 1 < n) fetch(t + 1);
#pragma unroll
        for (int i = 0; i < RPL; ++i) {
            const float kk = to_f32(kc.x[i]), qq = OUT ? to_f32(qc.x[i]) : 0.f;
            if constexpr (OUT) kq = fmaf(kk, qq, kq);
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                w[c] = fmaf(hr[i][c], kk, w[c]);
                if constexpr (OUT) z[c] = fmaf(hr[i][c], qq, z[c]);
            }
        }
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            w[c] = sum32(sum16(sum8(w[c])));
            if constexpr (OUT) z[c] = sum32(sum16(sum8(z[c])));
        }
        if constexpr (OUT) kq = sum32(sum16(sum8(kq)));
        float u[CPL];
#pragma unroll
        for (int c = 0; c < CPL; ++c) u[c] = bc * (vc[c] - ac * w[c]);
#pragma unroll
        for (int i = 0; i < RPL; ++i) {
            const float kk = to_f32(kc.x[i]);
#pragma unroll
            for (int c = 0; c < CPL; ++c) hr[i][c] = fmaf(kk, u[c], ac * hr[i][c]);
        }
        if constexpr (OUT) {
            if (rg == 0 && live) {
                TF *o = static_cast<TF *>(a.out) + (size_t)(lo + t) * sv + (size_t)h * DV + c0;
#pragma unroll
                for (int c = 0; c < CPL; ++c) o[c] = (TF)fmaf(ac, z[c], kq * u[c]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < RPL; ++i)
        if (live && (ROW == kExact || r0 + i < DK))
            __builtin_nontemporal_store(hr[i], reinterpret_cast<hvec *>(Hu + (size_t)(r0 + i) * DV));
}

static bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <int MODE, typename TF, int RPL, int CPL>
static hipError_t launch_columns(const WalkArgs &a, hipStream_t stream) {
    const int units = a.s.B * a.s.H, cols = 8 * CPL, blocks = (a.s.DV + cols - 1) / cols;
    const bool parts = a.s.DK * sizeof(TF) % 16 == 0 && aligned16(a.k) && (MODE == kWalkCommit || aligned16(a.q));
    const dim3 grid((unsigned)(((int64_t)units * blocks + 3) / 4)), block(256);
    if (parts && a.s.DK == 8 * RPL)
        delta_walk_kernel<MODE, TF, RPL, CPL, kExact><<<grid, block, 0, stream>>>(a, units, blocks);
    else if (parts)
        delta_walk_kernel<MODE, TF, RPL, CPL, kParts><<<grid, block, 0, stream>>>(a, units, blocks);
    else
        delta_walk_kernel<MODE, TF, RPL, CPL, kAnyRow><<<grid, block, 0, stream>>>(a, units, blocks);
    return hipGetLastError();
}

// Four columns a lane (16-byte accesses), or one and four times the wavefronts where four would
// leave the chip unfilled: a token's chain is then a quarter as long, the accesses 32 bytes wide.
// Steps, which move a state for one token's chain, gain below 512 wide wavefronts (128 x 128
// states of 32 heads, bf16: 3.4 against 4.0 us for one sequence, 5.4 against 5.0 for four), paths
// and prompts below 2048 (paths of up to 10 nodes, 8 sequences: 10.9 against 13.2 us; 16: equal).
template <int MODE, typename TF, int RPL>
static hipError_t launch_rows(const WalkArgs &a, hipStream_t stream) {
    const bool wide = a.s.DV % 4 == 0 && aligned16(a.H0);
    if (wide && (int64_t)a.s.B * a.s.H * ((a.s.DV + 31) / 32) >= (MODE == kWalkStep ? 512 : 2048))
        return launch_columns<MODE, TF, RPL, 4>(a, stream);
    return launch_columns<MODE, TF, RPL, 1>(a, stream);
}

template <int MODE, typename TF>
static hipError_t launch_typed(const WalkArgs &a, hipStream_t stream) {
    if (a.s.DK <= 64) return launch_rows<MODE, TF, 8>(a, stream);
    if (a.s.DK <= 128) return launch_rows<MODE, TF, 16>(a, stream);
    return launch_rows<MODE, TF, 32>(a, stream);
}

template <int MODE>
static hipError_t launch_walk(const WalkArgs &a, int32_t dtype, hipStream_t stream) {
    return dtype == BOLE_DTYPE_F32 ? launch_typed<MODE, float>(a, stream)
                                   : launch_typed<MODE, __bf16>(a, stream);
}

static DeltaShape shape(const bole_delta_dims_t &d) {
    return {d.batch, d.heads, d.key_heads, d.d_k, d.d_v, d.total_tokens};
}

hipError_t launch_delta_step(float *H0, const void *q, const void *k, const void *v,
                             const float *gate, const float *beta, void *out,
                             const bole_delta_dims_t &d, hipStream_t stream) {
    const WalkArgs a = {H0, q, k, v, gate, beta, nullptr, nullptr, nullptr, nullptr,
                        out, nullptr, nullptr, shape(d), 0};
    return launch_walk<kWalkStep>(a, d.factor_dtype, stream);
}

hipError_t launch_delta_commit(float *H0, const void *k, const void *v, const float *gate,
                               const float *beta, const int32_t *parent,
                               const int32_t *node_offsets, const int32_t *accepted_idx,
                               const int32_t *accepted_len, const bole_delta_dims_t &d,
                               int32_t *path_nodes, int32_t *tree_status, hipStream_t stream) {
    const WalkArgs a = {H0, nullptr, k, v, gate, beta, parent, node_offsets, accepted_idx,
                        accepted_len, nullptr, path_nodes, tree_status, shape(d), d.max_path};
    return launch_walk<kWalkCommit>(a, d.factor_dtype, stream);
}

hipError_t launch_delta_prefill_walk(float *H0, const void *q, const void *k, const void *v,
                                     const float *gate, const float *beta,
                                     const int32_t *seq_offsets, void *out,
                                     const bole_delta_dims_t &d, int32_t *seq_status,
                                     hipStream_t stream) {
    const WalkArgs a = {H0, q, k, v, gate, beta, nullptr, seq_offsets, nullptr, nullptr,
                        out, nullptr, seq_status, shape(d), 0};
    return launch_walk<kWalkPrefill>(a, d.factor_dtype, stream);
}

}  // namespace bole
