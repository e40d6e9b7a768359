// linear_walk.hip - linear attention with a decay token by token: the single-token step, and
// prompts of shapes and gates that the chunked kernels do not take.
//
// One token, from state H (all in fp32):   H <- a H + k v^T,   o = H^T q.
//
// A wavefront owns 8 CPL columns of one state and keeps all of their rows in registers: lane
// (rg, cg) = (lane / 8, lane % 8) holds rows rg RPL .. rg RPL + RPL - 1 of columns cg CPL ..
// cg CPL + CPL - 1. o is summed over the lane's rows as they are updated, then over the eight row
// groups with three cross-lane steps. Nothing is shared between wavefronts: no LDS, no barrier.
// The state is read once and written once whatever the number of tokens, with non-temporal
// 16-byte accesses (a row's eight lanes cover 128 contiguous bytes).
#include "linear_device.h"
#include "launch.h"

namespace bole {

// CHANNEL: a decay for each key channel, in place of one a head.
template <bool PROMPTS, typename TF, bool CHANNEL, int RPL, int CPL, int ROW>
__global__ __launch_bounds__(256) void linear_walk_kernel(const LinearArgs a, int units, int blocks) {
    typedef float hvec __attribute__((ext_vector_type(CPL)));
    const int lane = lane_id();
    const int wave = blockIdx.x * 4 + (threadIdx.x >> 6);
    const int unit = wave / blocks, cb = wave - unit * blocks;
    if (unit >= units) return;
    const int H = a.s.H, DK = a.s.DK, DV = a.s.DV;
    const int b = unit / H, h = unit - b * H, hk = h / (H / a.s.HK);
    const int rg = lane >> 3, c0 = (cb * 8 + (lane & 7)) * CPL, r0 = rg * RPL;
    const bool live = c0 < DV;  // CPL divides d_v: a lane's columns exist or do not together
    int lo = b, n = 1;
    if constexpr (PROMPTS) {
        const bool ok = offsets_ordered(a.offsets, a.s.B, a.s.T);
        if (h == 0 && cb == 0 && lane == 0 && a.status)
            a.status[b] = ok ? BOLE_TREE_OK : BOLE_TREE_BAD_SIZE;
        lo = a.offsets[b];
        n = ok ? a.offsets[b + 1] - lo : 0;
        if (n <= 0) return;
    }
    float *Hu = a.H0 + (size_t)unit * DK * DV + c0;
    hvec hr[RPL];
#pragma unroll
    for (int i = 0; i < RPL; ++i) {
        hr[i] = (hvec)0.f;
        if (live && (ROW == kExact || r0 + i < DK))
            hr[i] = __builtin_nontemporal_load(reinterpret_cast<const hvec *>(Hu + (size_t)(r0 + i) * DV));
    }
    const TF *q = static_cast<const TF *>(a.q), *k = static_cast<const TF *>(a.k),
             *v = static_cast<const TF *>(a.v);
    const size_t sk = (size_t)a.s.HK * DK, sv = (size_t)H * DV;
    RowPiece<TF, RPL, ROW> kn, qn;
    RowPiece<float, CHANNEL ? RPL : 1, CHANNEL ? ROW : kAnyRow> gn;
    float vn[CPL];
    auto fetch = [&](int t) {
        const size_t row = (size_t)lo + t;
        kn.load(k + row * sk + (size_t)hk * DK, r0, DK);
        qn.load(q + row * sk + (size_t)hk * DK, r0, DK);
#pragma unroll
        for (int c = 0; c < CPL; ++c)
            vn[c] = live ? to_f32(v[row * sv + (size_t)h * DV + c0 + c]) : 0.f;
        if constexpr (CHANNEL) gn.load(a.gate + (row * H + h) * DK, r0, DK);
        else gn.x[0] = a.gate[row * H + h];
    };
    fetch(0);
    for (int t = 0; t < n; ++t) {
        const RowPiece<TF, RPL, ROW> kc = kn, qc = qn;
        const auto gc = gn;
        float vc[CPL], z[CPL];
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
            vc[c] = vn[c];
            z[c] = 0.f;
        }
        if (t + 1 < n) fetch(t + 1);
#pragma unroll
        for (int i = 0; i < RPL; ++i) {
            const float kk = to_f32(kc.x[i]), qq = to_f32(qc.x[i]), g = gc.x[CHANNEL ? i : 0];
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                hr[i][c] = fmaf(kk, vc[c], g * hr[i][c]);
                z[c] = fmaf(hr[i][c], qq, z[c]);
            }
        }
#pragma unroll
        for (int c = 0; c < CPL; ++c) z[c] = sum32(sum16(sum8(z[c])));
        if (rg == 0 && live) {
            TF *o = static_cast<TF *>(a.out) + ((size_t)lo + t) * sv + (size_t)h * DV + c0;
#pragma unroll
            for (int c = 0; c < CPL; ++c) o[c] = (TF)z[c];
        }
    }
#pragma unroll
    for (int i = 0; i < RPL; ++i)
        if (live && (ROW == kExact || r0 + i < DK))
            __builtin_nontemporal_store(hr[i], reinterpret_cast<hvec *>(Hu + (size_t)(r0 + i) * DV));
}

static bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <bool PROMPTS, typename TF, bool CHANNEL, int RPL, int CPL>
static hipError_t launch_columns(const LinearArgs &a, hipStream_t stream) {
    const int units = a.s.B * a.s.H, cols = 8 * CPL, blocks = (a.s.DV + cols - 1) / cols;
    const bool parts = a.s.DK * sizeof(TF) % 16 == 0 && aligned16(a.k) && aligned16(a.q) &&
                       (!CHANNEL || aligned16(a.gate));
    const dim3 grid((unsigned)(((int64_t)units * blocks + 3) / 4)), block(256);
    if (parts && a.s.DK == 8 * RPL)
        linear_walk_kernel<PROMPTS, TF, CHANNEL, RPL, CPL, kExact><<<grid, block, 0, stream>>>(a, units, blocks);
    else if (parts)
        linear_walk_kernel<PROMPTS, TF, CHANNEL, RPL, CPL, kParts><<<grid, block, 0, stream>>>(a, units, blocks);
    else
        linear_walk_kernel<PROMPTS, TF, CHANNEL, RPL, CPL, kAnyRow><<<grid, block, 0, stream>>>(a, units, blocks);
    return hipGetLastError();
}

// Four columns a lane (16-byte accesses), or one and four times the wavefronts where four would
// leave the chip unfilled.
template <bool PROMPTS, typename TF, bool CHANNEL, int RPL>
static hipError_t launch_rows(const LinearArgs &a, hipStream_t stream) {
    const bool wide = a.s.DV % 4 == 0 && aligned16(a.H0);
    if (wide && (int64_t)a.s.B * a.s.H * ((a.s.DV + 31) / 32) >= (PROMPTS ? 2048 : 512))
        return launch_columns<PROMPTS, TF, CHANNEL, RPL, 4>(a, stream);
    return launch_columns<PROMPTS, TF, CHANNEL, RPL, 1>(a, stream);
}

template <bool PROMPTS, typename TF, bool CHANNEL>
static hipError_t launch_typed(const LinearArgs &a, hipStream_t stream) {
    if (a.s.DK <= 64) return launch_rows<PROMPTS, TF, CHANNEL, 8>(a, stream);
    if (a.s.DK <= 128) return launch_rows<PROMPTS, TF, CHANNEL, 16>(a, stream);
    return launch_rows<PROMPTS, TF, CHANNEL, 32>(a, stream);
}

template <bool PROMPTS>
static hipError_t launch_gated(const LinearArgs &a, const bole_linear_dims_t &d, hipStream_t stream) {
    const bool channel = d.gate_kind == BOLE_GATE_VECTOR;
    if (d.factor_dtype == BOLE_DTYPE_F32)
        return channel ? launch_typed<PROMPTS, float, true>(a, stream)
                       : launch_typed<PROMPTS, float, false>(a, stream);
    return channel ? launch_typed<PROMPTS, __bf16, true>(a, stream)
                   : launch_typed<PROMPTS, __bf16, false>(a, stream);
}

hipError_t launch_linear_walk(const LinearArgs &a, const bole_linear_dims_t &d, bool prompts,
                              hipStream_t stream) {
    return prompts ? launch_gated<true>(a, d, stream) : launch_gated<false>(a, d, stream);
}

}  // namespace bole
