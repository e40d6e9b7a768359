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
//
// Measured, 32 heads of 128 x 64 states, bf16: a token of each of 128 sequences 50 us (5.4 TB/s: the
// states' way through HBM), of one sequence 4.0 to 4.6 us (launch, and one chain of loads and sums).
#include "linear_device.h"
#include "launch.h"

namespace bole {

// Step and prompt alike are bound by the state's round trip through HBM where they are many; a long
// prompt by the chain of its tokens, so prompts are cut into segments: a first kernel walks each
// segment from nothing, a second runs over a sequence's segments and leaves the state that each starts
// from, a third walks them again, with outputs. (Two prompts of up to 600 tokens, 32 heads of 128 x 64
// states, decays a channel: 86 to 89 us - 26, 20 and 39 - and 606 in one chain.)
//
// A segment's decays are multiplied in fp64, as their products may leave fp32 where what they scale is
// small or zero, and kept below infinity, as zero has to stay that. A product in fp32's range goes on as
// it is, one above or below as its root with a minus sign.
struct WalkSpace {
    float *s;      // [slot][H][d_k][d_v]
    float *decay;  // [slot][H], or [slot][H][d_k]
    int seg;       // tokens a segment; 0: whole sequences
};

__device__ __forceinline__ float kept_decay(double x) {
    if (x == 0.0 || (x >= 0x1p-126 && x <= 0x1p126)) return (float)x;
    const double root = sqrt(x);
    return root > 0x1p127 ? -0x1p127f : -(float)root;
}

enum { kWalkStep = 0, kWalkLocal = 1, kWalkMain = 2 };

// CHANNEL: a decay for each key channel, in place of one a head.
template <int MODE, typename TF, bool CHANNEL, int RPL, int CPL, int ROW>
__global__ __launch_bounds__(256) void linear_walk_kernel(const LinearArgs a, const WalkSpace w, int units, int blocks) {
    typedef float hvec __attribute__((ext_vector_type(CPL)));
    constexpr bool OUT = MODE != kWalkLocal;
    const int lane = lane_id();
    const int wave = blockIdx.x * 4 + (threadIdx.x >> 6);
    const int unit = wave / blocks, cb = wave - unit * blocks;
    if (unit >= units) return;
    const int H = a.s.H, DK = a.s.DK, DV = a.s.DV;
    int b = unit / H;
    const int h = unit - b * H, hk = h / (H / a.s.HK);
    const int rg = lane >> 3, c0 = (cb * 8 + (lane & 7)) * CPL, r0 = rg * RPL;
    const bool live = c0 < DV;  // CPL divides d_v: a lane's columns exist or do not together
    int lo = b, n = 1;
    const float *from = nullptr;
    float *to = nullptr;        // the state's place after the last token, if it has one
    size_t space = 0;
    if constexpr (MODE != kWalkStep) {
        Located l = {};
        int i = 0;
        if (w.seg > 0) {
            l = locate(a.offsets, a.s.B, a.s.T, w.seg, b);
            i = b - l.slot0;
        } else {
            l.ordered = offsets_ordered(a.offsets, a.s.B, a.s.T);
            l.found = l.ordered, l.b = b, l.lo = a.offsets[b], l.n = a.offsets[b + 1] - l.lo;
        }
        if (OUT && h == 0 && cb == 0 && a.status) {
            if (!l.ordered) {
                if (b == 0)
                    for (int x = lane; x < a.s.B; x += 64) a.status[x] = BOLE_TREE_BAD_SIZE;
            } else if (l.found && i == 0 && lane == 0) {
                a.status[l.b] = BOLE_TREE_OK;
            }
        }
        if (!l.found) return;
        const int t0 = i * w.seg;
        if (t0 >= l.n || (!OUT && t0 + w.seg >= l.n)) return;
        const bool cut = w.seg > 0 && l.n > w.seg;
        n = cut ? min(w.seg, l.n - t0) : l.n;
        b = l.b, lo = l.lo + t0;
        space = cut ? space_slot(l.lo, w.seg, i) * H + h : 0;
        float *state = a.H0 + (size_t)(b * H + h) * DK * DV;
        from = cut ? w.s + space * DK * DV : state;
        to = !OUT ? w.s + space * DK * DV : t0 + n == l.n ? state : nullptr;
    } else {
        to = a.H0 + (size_t)unit * DK * DV;
        from = to;
    }
    hvec hr[RPL];
#pragma unroll
    for (int i = 0; i < RPL; ++i) {
        hr[i] = (hvec)0.f;
        if (OUT && live && (ROW == kExact || r0 + i < DK))
            hr[i] = __builtin_nontemporal_load(reinterpret_cast<const hvec *>(from + c0 + (size_t)(r0 + i) * DV));
    }
    const TF *q = static_cast<const TF *>(a.q), *k = static_cast<const TF *>(a.k),
             *v = static_cast<const TF *>(a.v);
    const size_t sk = (size_t)a.s.HK * DK, sv = (size_t)H * DV;
    // Decays that the lane multiplies up: the head's, or its share of the row group's.
    constexpr int SHARE = CHANNEL ? RPL / 8 : 1;
    const int s0 = CHANNEL ? r0 + (lane & 7) * SHARE : 0;
    struct Token {
        RowPiece<TF, RPL, ROW> k, q;
        RowPiece<float, CHANNEL ? RPL : 1, CHANNEL ? ROW : kAnyRow> g;
        float v[CPL];
        float share[SHARE];
    };
    // this token and the next one: with three or four the registers leave fewer wavefronts (7000 tokens of
    // 32 heads with decays a channel 0.60 ms, 0.98 and 1.01)
    constexpr int AHEAD = MODE == kWalkStep ? 1 : 2;
    Token x[AHEAD];
    double all[SHARE];
#pragma unroll
    for (int i = 0; i < SHARE; ++i) all[i] = 1.0;
    auto fetch = [&](int t, Token &y) {
        const size_t row = (size_t)lo + min(t, n - 1);
        y.k.load(k + row * sk + (size_t)hk * DK, r0, DK);
        if constexpr (OUT) y.q.load(q + row * sk + (size_t)hk * DK, r0, DK);
#pragma unroll
        for (int c = 0; c < CPL; ++c)
            y.v[c] = live ? to_f32(v[row * sv + (size_t)h * DV + c0 + c]) : 0.f;
        if constexpr (CHANNEL) y.g.load(a.gate + (row * H + h) * DK, r0, DK);
        else y.g.x[0] = a.gate[row * H + h];
        if constexpr (!OUT) {
#pragma unroll
            for (int i = 0; i < SHARE; ++i)
                y.share[i] = !CHANNEL ? y.g.x[0] : ROW == kExact || s0 + i < DK ? a.gate[(row * H + h) * DK + s0 + i] : 1.f;
        }
    };
    auto token = [&](int t, const Token &y) {
        float z[CPL];
#pragma unroll
        for (int c = 0; c < CPL; ++c) z[c] = 0.f;
        if constexpr (!OUT) {
#pragma unroll
            for (int i = 0; i < SHARE; ++i) all[i] *= (double)y.share[i];
        }
#pragma unroll
        for (int i = 0; i < RPL; ++i) {
            const float kk = to_f32(y.k.x[i]), qq = OUT ? to_f32(y.q.x[i]) : 0.f, g = y.g.x[CHANNEL ? i : 0];
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                hr[i][c] = fmaf(kk, y.v[c], g * hr[i][c]);
                if constexpr (OUT) z[c] = fmaf(hr[i][c], qq, z[c]);
            }
        }
        if constexpr (OUT) {
#pragma unroll
            for (int c = 0; c < CPL; ++c) z[c] = sum32(sum16(sum8(z[c])));
            if (rg == 0 && live) {
                TF *o = static_cast<TF *>(a.out) + ((size_t)lo + t) * sv + (size_t)h * DV + c0;
#pragma unroll
                for (int c = 0; c < CPL; ++c) o[c] = (TF)z[c];
            }
        }
    };
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) fetch(u, x[u]);
    if constexpr (MODE == kWalkStep) {
        token(0, x[0]);
    } else {
        int t = 0;
        for (; t + AHEAD <= n; t += AHEAD) {
            if constexpr (!OUT) {  // (two decays more stay below infinity)
                static_assert(AHEAD == 2, "range");
#pragma unroll
                for (int i = 0; i < SHARE; ++i) all[i] = all[i] > 0x1p700 ? 0x1p700 : all[i];
            }
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                token(t + u, x[u]);
                fetch(t + u + AHEAD, x[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            if (t + u < n) token(t + u, x[u]);
    }
    if (to) {
#pragma unroll
        for (int i = 0; i < RPL; ++i)
            if (live && (ROW == kExact || r0 + i < DK))
                __builtin_nontemporal_store(hr[i], reinterpret_cast<hvec *>(to + c0 + (size_t)(r0 + i) * DV));
    }
    if constexpr (!OUT) {
        if (cb == 0) {
            if constexpr (CHANNEL) {
#pragma unroll
                for (int i = 0; i < SHARE; ++i)
                    if (s0 + i < DK) w.decay[space * DK + s0 + i] = kept_decay(all[i]);
            } else if (lane == 0) {
                w.decay[space] = kept_decay(all[0]);
            }
        }
    }
}

// Over a sequence's segments: each one's contribution gives way to the state that it starts from. A
// thread an element, eight segments' loads in flight.
__global__ __launch_bounds__(256) void linear_walk_carry_kernel(const LinearArgs a, const WalkSpace w, bool channel) {
    const DeltaShape &s = a.s;
    const int unit = blockIdx.x, b = unit / s.H, h = unit - b * s.H;
    if (!offsets_ordered(a.offsets, s.B, s.T)) return;
    const int lo = a.offsets[b], n = a.offsets[b + 1] - lo, e = blockIdx.y * 256 + threadIdx.x;
    if (n <= w.seg || e >= s.DK * s.DV) return;
    const int count = (n + w.seg - 1) / w.seg, row = e / s.DV;
    float S = a.H0[(size_t)unit * s.DK * s.DV + e];
    const size_t first = space_slot(lo, w.seg, 0) * s.H + h, step = (size_t)s.H * s.DK * s.DV;
    float *x = w.s + first * s.DK * s.DV + e;
    const float *d = channel ? w.decay + first * s.DK + row : w.decay + first;
    const size_t dstep = channel ? (size_t)s.H * s.DK : s.H;
    for (int i = 0; i < count; i += 8) {
        float own[8], decay[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int at = min(i + k, count - 2);  // (the last segment's is not needed, and not there)
            own[k] = x[at * step];
            decay[k] = d[at * dstep];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (i + k >= count) break;
            x[(i + k) * step] = S;
            const float by = fabsf(decay[k]);
            S = fmaf(decay[k] < 0.f ? S * by : S, by, own[k]);
        }
    }
}

static bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <int MODE, typename TF, bool CHANNEL, int RPL, int CPL>
static hipError_t launch_columns(const LinearArgs &a, const WalkSpace &w, int units, hipStream_t stream) {
    const int cols = 8 * CPL, blocks = (a.s.DV + cols - 1) / cols;
    const bool parts = a.s.DK * sizeof(TF) % 16 == 0 && aligned16(a.k) && aligned16(a.q) &&
                       (!CHANNEL || aligned16(a.gate));
    const dim3 grid((unsigned)(((int64_t)units * blocks + 3) / 4)), block(256);
    if (parts && a.s.DK == 8 * RPL)
        linear_walk_kernel<MODE, TF, CHANNEL, RPL, CPL, kExact><<<grid, block, 0, stream>>>(a, w, units, blocks);
    else if (parts)
        linear_walk_kernel<MODE, TF, CHANNEL, RPL, CPL, kParts><<<grid, block, 0, stream>>>(a, w, units, blocks);
    else
        linear_walk_kernel<MODE, TF, CHANNEL, RPL, CPL, kAnyRow><<<grid, block, 0, stream>>>(a, w, units, blocks);
    return hipGetLastError();
}

// Four columns a lane (16-byte accesses), so that a token's key, query and decays are loaded once for
// four; or one and four times the wavefronts for steps that would leave the chip unfilled (a token of each
// of 4 sequences of 32 heads 5.2 against 5.4 us, of 8 6.1 against 5.9, of 128 123 against 50).
template <int MODE, typename TF, bool CHANNEL, int RPL>
static hipError_t launch_rows(const LinearArgs &a, const WalkSpace &w, int units, hipStream_t stream) {
    const bool wide = a.s.DV % 4 == 0 && aligned16(a.H0);
    if (wide && (MODE != kWalkStep || (int64_t)units * ((a.s.DV + 31) / 32) >= 512))
        return launch_columns<MODE, TF, CHANNEL, RPL, 4>(a, w, units, stream);
    return launch_columns<MODE, TF, CHANNEL, RPL, 1>(a, w, units, stream);
}

template <int MODE, typename TF, bool CHANNEL>
static hipError_t launch_typed(const LinearArgs &a, const WalkSpace &w, int units, hipStream_t stream) {
    if (a.s.DK <= 64) return launch_rows<MODE, TF, CHANNEL, 8>(a, w, units, stream);
    if (a.s.DK <= 128) return launch_rows<MODE, TF, CHANNEL, 16>(a, w, units, stream);
    return launch_rows<MODE, TF, CHANNEL, 32>(a, w, units, stream);
}

template <int MODE>
static hipError_t launch_gated(const LinearArgs &a, const WalkSpace &w, int units, const bole_linear_dims_t &d,
                               hipStream_t stream) {
    const bool channel = d.gate_kind == BOLE_GATE_VECTOR;
    if (d.factor_dtype == BOLE_DTYPE_F32)
        return channel ? launch_typed<MODE, float, true>(a, w, units, stream)
                       : launch_typed<MODE, float, false>(a, w, units, stream);
    return channel ? launch_typed<MODE, __bf16, true>(a, w, units, stream)
                   : launch_typed<MODE, __bf16, false>(a, w, units, stream);
}

hipError_t launch_linear_step_walk(const LinearArgs &a, const bole_linear_dims_t &d, hipStream_t stream) {
    return launch_gated<kWalkStep>(a, {nullptr, nullptr, 0}, a.s.B * a.s.H, d, stream);
}

// Tokens a segment (0: sequences stay whole), from a call's sizes alone: segments so that 2048
// wavefronts run, of at least 16 tokens, since each costs a state's way through memory (two prompts of
// up to 600 tokens 86 us, with at least 32 103; four heads' 46 and 67).
static int walk_segment(const bole_linear_dims_t &d) {
    const int64_t blocks = d.d_v % 4 == 0 ? (d.d_v + 31) / 32 : (d.d_v + 7) / 8;
    if ((int64_t)d.batch * d.heads * blocks >= 2048) return 0;
    int64_t seg = ((int64_t)d.total_tokens * d.heads * blocks + 2047) / 2048;
    if (seg < 16) seg = 16;
    return seg < d.total_tokens ? (int)seg : 0;
}

size_t linear_walk_workspace(const bole_linear_dims_t &d) {
    const int seg = walk_segment(d);
    if (seg == 0) return 0;
    const size_t each = (size_t)d.d_k * d.d_v + (d.gate_kind == BOLE_GATE_VECTOR ? d.d_k : 1);
    return (space_slots(d.total_tokens, seg) * d.heads * each * sizeof(float) + 15) / 16 * 16;
}

hipError_t launch_linear_walk(const LinearArgs &a, const bole_linear_dims_t &d, void *workspace,
                              hipStream_t stream) {
    const int seg = walk_segment(d);
    if (seg == 0) return launch_gated<kWalkMain>(a, {nullptr, nullptr, 0}, a.s.B * a.s.H, d, stream);
    float *s = static_cast<float *>(workspace);
    const WalkSpace w = {s, s + space_slots(d.total_tokens, seg) * d.heads * d.d_k * d.d_v, seg};
    const int units = (d.total_tokens / seg + d.batch) * d.heads;
    hipError_t e = launch_gated<kWalkLocal>(a, w, units, d, stream);
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)(a.s.B * a.s.H), (unsigned)((d.d_k * d.d_v + 255) / 256));
    linear_walk_carry_kernel<<<grid, dim3(256), 0, stream>>>(a, w, d.gate_kind == BOLE_GATE_VECTOR);
    e = hipGetLastError();
    return e != hipSuccess ? e : launch_gated<kWalkMain>(a, w, units, d, stream);
}

}  // namespace bole
