// delta_prefill.hip - prompts through the gated delta rule, 64 tokens at a time.
//
// Within a chunk the updates U of all tokens solve one triangular system (delta_mfma.h), and
// with the chunk's start state S, start_i = 2^{L_i} and end_i = 2^{L_C - L_i}:
//     R = V - diag(start) K S,   U = X diag(b) R,   O = diag(start) Q S + P U,
//     S <- start_C S + K^T diag(end) U.
// X and P do not depend on the state: a first kernel forms them for every chunk and head at
// once and writes them to the workspace. A second one walks each sequence's chunks in order
// with the state in registers, a workgroup per (sequence, value head, 16 NT columns).
//
// The state is kept to fp32: K is exact in bf16, and S, R, X and end U are taken as three bf16
// terms each (2^-25 left). What only the output sees may be rounded harder: S and U in two
// terms, P in one (half a step of bf16 of each pair weight, once, before an output that is
// rounded to bf16 itself).
#include "delta_mfma.h"
#include "launch.h"

namespace bole {

// Workspace of one chunk and value head: operand pieces in the order the second kernel's lanes
// load them, 64 lanes times 8 values a piece. Row tiles 0 and 1 have one piece (tokens 0..31),
// tiles 2 and 3 two; what lies right of the diagonal is zero and not stored.
constexpr int kPieces = 6;
struct ChunkSystem {
    float x[kPieces][64][8];     // X diag(b)
    __bf16 p[kPieces][64][8];    // P
    float start[kChunk], end[kChunk];
};

__device__ __forceinline__ int piece_of(int m, int s) { return s == 0 ? m : 2 + m; }

struct PrefillArgs {
    float *H0;
    const __bf16 *q, *k, *v;
    const float *gate, *beta;
    const int32_t *offsets;
    __bf16 *out;
    int32_t *status;
    ChunkSystem *ws;
    DeltaShape s;
};

template <int DK>
__global__ __launch_bounds__(256, 2) void delta_chunk_kernel(const PrefillArgs a) {
    __shared__ DeltaTokens t;
    const DeltaShape &s = a.s;
    const int h = blockIdx.x % s.H, slot = blockIdx.x / s.H, hk = h / (s.H / s.HK);
    const int tid = threadIdx.x, lane = lane_id(), wave = tid >> 6, col = lane & 15, g = lane >> 4;
    int b, slot0;
    bool ordered;
    if (!locate(a.offsets, s.B, s.T, 1, kChunk, slot, b, slot0, ordered)) return;
    const int lo = a.offsets[b] + (slot - slot0) * kChunk, n = min(kChunk, a.offsets[b + 1] - lo);
    if (n <= 0) return;
    ChunkSystem &w = a.ws[(size_t)slot * s.H + h];
    if (tid < 64) {
        const bool in = tid < n;
        const size_t at = (size_t)(lo + tid) * s.H + h;
        const WaveTopoD c = wave_topology_cumlog_f64(tid - 1, in ? log2_decay(a.gate[at]) : 0.f, n);
        t.mask[tid] = c.mask;
        t.L[tid] = c.L;
        t.beta[tid] = in ? a.beta[at] : 0.f;
        const double all = shfl_f64(c.L, n - 1);
        w.start[tid] = in ? __builtin_amdgcn_exp2f((float)c.L) : 0.f;
        w.end[tid] = in ? __builtin_amdgcn_exp2f((float)(all - c.L)) : 0.f;
    }
    lds_barrier();
    const size_t sk = (size_t)s.HK * DK, at = (size_t)lo * sk + (size_t)hk * DK;
    delta_system<DK>(t, a.k + at, a.q + at, sk, n);
#pragma unroll
    for (int sb = 0; sb < 2; ++sb) {
        if (sb > (wave >> 1)) continue;
        const int f = piece_of(wave, sb);
        f32x4 x, y;
        x_piece(t, tile_token(wave, col), sb, g, x, y);
        *reinterpret_cast<f32x4 *>(&w.x[f][lane][0]) = x;
        *reinterpret_cast<f32x4 *>(&w.x[f][lane][4]) = y;
        p_piece(t, tile_token(wave, col), sb, g, x, y);
        bf16x8 p[1];
        split_terms8<1>(x, y, p);
        *reinterpret_cast<bf16x8 *>(&w.p[f][lane][0]) = p[0];
    }
}

// One workgroup: four wavefronts, 16 NT state columns. Wavefront w has the tokens of row tile
// w and the state rows of d_k / 64 row tiles; what it computes becomes the others' operand
// through LDS (S, then R, then U; three barriers a chunk). In operand order every exchange is
// a lane's own 8 or 16 bytes. The next chunk's rows and system are in flight meanwhile.
template <int DK, int NT>
__global__ __launch_bounds__(256, 2) void delta_scan_kernel(const PrefillArgs a, int units, int groups) {
    constexpr int KS = DK / 32, TILES = DK / 64, CH = DK / 8, PER = kChunk * CH / 256, KP = DK + 8;
    __shared__ __align__(16) __bf16 s_k[2][kChunk * KP];
    __shared__ __align__(16) __bf16 s_s[3][NT][KS][64][8];   // state, three terms
    __shared__ __align__(16) __bf16 s_r[3][NT][2][64][8];    // R
    __shared__ __align__(16) __bf16 s_e[3][NT][2][64][8];    // end U, for the state
    __shared__ __align__(16) __bf16 s_u[2][NT][2][64][8];    // U, for the output
    const DeltaShape &s = a.s;
    // the column groups of a unit go to one XCD (workgroups are dealt to the eight in turn):
    // they read the same rows and systems, and fill each other's output lines
    const int unit = (int)(blockIdx.x / 8 / groups) * 8 + (int)(blockIdx.x % 8);
    const int cg = (int)(blockIdx.x / 8) % groups;
    if (unit >= units) return;
    const int tid = threadIdx.x, lane = lane_id(), wave = tid >> 6, col = lane & 15, g = lane >> 4;
    const int b = unit / s.H, h = unit - b * s.H, hk = h / (s.H / s.HK);
    const bool ordered = offsets_ordered(a.offsets, s.B, s.T);
    if (h == 0 && cg == 0 && tid == 0 && a.status)
        a.status[b] = ordered ? BOLE_TREE_OK : BOLE_TREE_BAD_SIZE;
    if (!ordered) return;
    const int lo = a.offsets[b], n = a.offsets[b + 1] - lo;
    if (n == 0) return;
    const int chunks = (n + kChunk - 1) / kChunk;
    const size_t sk = (size_t)s.HK * DK, sv = (size_t)s.H * s.DV;
    const int c0 = 16 * NT * cg + col;   // + 16 c
    const ChunkSystem *ws = a.ws + ((size_t)(lo / kChunk + b)) * s.H + h;
    const __bf16 *kb = a.k + (size_t)lo * sk + (size_t)hk * DK, *qb = a.q + (size_t)lo * sk + (size_t)hk * DK;
    const size_t v0 = (size_t)lo * sv + (size_t)h * s.DV + c0;

    // state row of register e of row tile j: tiles are numbered and laid out as tokens are
    const int m0 = wave * TILES;
    float *Hu = a.H0 + (size_t)unit * DK * s.DV + c0;
    f32x4 st[TILES][NT];
#pragma unroll
    for (int j = 0; j < TILES; ++j)
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                st[j][c][e] = Hu[(size_t)tile_token(m0 + j, 4 * g + e) * s.DV + 16 * c];

    // a row tile's four values a lane, as the terms of the B operand
    auto put = [&](const f32x4 &x, int m, auto &dst, int c) {
        constexpr int N = sizeof(dst) / sizeof(dst[0]);
        bf16x4 y[N];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            __bf16 t[N];
            split_terms<N>(x[e], t);
#pragma unroll
            for (int i = 0; i < N; ++i) y[i][e] = t[i];
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
            *reinterpret_cast<bf16x4 *>(&dst[i][c][m >> 1][lane][4 * (m & 1)]) = y[i];
    };
    // The next chunk's loads, raw: nothing waits for them before they are used. Rows past the
    // last token repeat it: their columns of X diag(b) and their `end` are zero, and their
    // outputs are not stored.
    bf16x8 kr[PER], qn[KS], pn[2];
    f32x4 xn[2][2];
    __bf16 vn[4][NT];
    float startn[4], endn[4], decayn;
    const int my_row = tile_token(wave, col);
    auto fetch = [&](int chunk) {
        const int t0 = chunk * kChunk, last = min(kChunk, n - t0) - 1;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int e = tid + 256 * j;
            kr[j] = load16(kb + (size_t)(t0 + min(e / CH, last)) * sk + 8 * (e % CH));
        }
        const __bf16 *qrow = qb + (size_t)(t0 + min(my_row, last)) * sk + 8 * g;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) qn[ks] = load16(qrow + 32 * ks);
        const ChunkSystem &w = ws[(size_t)chunk * s.H];
#pragma unroll
        for (int sb = 0; sb < 2; ++sb) {
            // the first two wavefronts have one piece: they load it twice
            const int f = piece_of(wave, min(sb, wave >> 1));
            xn[sb][0] = *reinterpret_cast<const f32x4 *>(&w.x[f][lane][0]);
            xn[sb][1] = *reinterpret_cast<const f32x4 *>(&w.x[f][lane][4]);
            pn[sb] = *reinterpret_cast<const bf16x8 *>(&w.p[f][lane][0]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = tile_token(wave, 4 * g + e);
            startn[e] = w.start[i];
            endn[e] = w.end[i];
#pragma unroll
            for (int c = 0; c < NT; ++c) vn[e][c] = a.v[v0 + (size_t)(t0 + min(i, last)) * sv + 16 * c];
        }
        decayn = w.start[last];
    };
    auto stage = [&](int buf) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int e = tid + 256 * j;
            *reinterpret_cast<bf16x8 *>(&s_k[buf][(e / CH) * KP + 8 * (e % CH)]) = kr[j];
        }
    };
    auto put_state = [&]() {
#pragma unroll
        for (int j = 0; j < TILES; ++j)
#pragma unroll
            for (int c = 0; c < NT; ++c) put(st[j][c], m0 + j, s_s, c);
    };
    fetch(0);
    stage(0);
    put_state();
    lds_barrier();
    for (int chunk = 0; chunk < chunks; ++chunk) {
        const int buf = chunk & 1, t0 = chunk * kChunk;
        bf16x8 q[KS], p[2];
        bf16x8 x[2][3];
        float v[4][NT], start[4], end[4];
        const float decay = decayn;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) q[ks] = qn[ks];
#pragma unroll
        for (int sb = 0; sb < 2; ++sb) {
            p[sb] = pn[sb];
            split_terms8<3>(xn[sb][0], xn[sb][1], x[sb]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            start[e] = startn[e], end[e] = endn[e];
#pragma unroll
            for (int c = 0; c < NT; ++c) v[e][c] = (float)vn[e][c];
        }
        if (chunk + 1 < chunks) fetch(chunk + 1);

        // ---- K S and Q S for the wavefront's tokens
        f32x4 r[NT], o[NT];
#pragma unroll
        for (int c = 0; c < NT; ++c) r[c] = o[c] = (f32x4)0.f;
        const __bf16 *krow = &s_k[buf][my_row * KP + 8 * g];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const bf16x8 ka = load16(krow + 32 * ks);
#pragma unroll
            for (int c = 0; c < NT; ++c) {
                const bf16x8 s0 = load16(&s_s[0][c][ks][lane][0]), s1 = load16(&s_s[1][c][ks][lane][0]),
                             s2 = load16(&s_s[2][c][ks][lane][0]);
                r[c] = mfma16_bf16(ka, s2, r[c]);
                r[c] = mfma16_bf16(ka, s1, r[c]);
                r[c] = mfma16_bf16(ka, s0, r[c]);
                o[c] = mfma16_bf16(q[ks], s1, o[c]);
                o[c] = mfma16_bf16(q[ks], s0, o[c]);
            }
        }
#pragma unroll
        for (int c = 0; c < NT; ++c) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                r[c][e] = v[e][c] - start[e] * r[c][e];
                o[c][e] *= start[e];
            }
            put(r[c], wave, s_r, c);
        }
        lds_barrier();
        // ---- U = X diag(b) R
        f32x4 u[NT];
#pragma unroll
        for (int c = 0; c < NT; ++c) {
            u[c] = (f32x4)0.f;
#pragma unroll
            for (int sb = 0; sb < 2; ++sb) {
                if (sb > (wave >> 1)) continue;
                const bf16x8 rb[3] = {load16(&s_r[0][c][sb][lane][0]), load16(&s_r[1][c][sb][lane][0]),
                                      load16(&s_r[2][c][sb][lane][0])};
                u[c] = mfma_terms<3>(x[sb], rb, u[c]);
            }
        }
#pragma unroll
        for (int c = 0; c < NT; ++c) {
            put(u[c], wave, s_u, c);
            f32x4 ue;
#pragma unroll
            for (int e = 0; e < 4; ++e) ue[e] = end[e] * u[c][e];
            put(ue, wave, s_e, c);
        }
        lds_barrier();
        // ---- S <- decay S + K^T (end U): K^T through the transposing read
#pragma unroll
        for (int j = 0; j < TILES; ++j) {
#pragma unroll
            for (int c = 0; c < NT; ++c) st[j][c] *= decay;
            const int m = m0 + j;
#pragma unroll
            for (int sb = 0; sb < 2; ++sb) {
                // state rows of lanes 4c .. 4c + 3: 32 (m / 2) + 8 c + 4 (m % 2) ..
                const __bf16 *kt = &s_k[buf][(32 * sb + 8 * g + (col >> 2)) * KP + 32 * (m >> 1) +
                                             8 * (col & 3) + 4 * (m & 1)];
                const bf16x8 ka = join(read_transposed(kt), read_transposed(kt + 4 * KP));
#pragma unroll
                for (int c = 0; c < NT; ++c)
#pragma unroll
                    for (int i = 2; i >= 0; --i)
                        st[j][c] = mfma16_bf16(ka, load16(&s_e[i][c][sb][lane][0]), st[j][c]);
            }
        }
        // ---- O += P U
#pragma unroll
        for (int c = 0; c < NT; ++c) {
#pragma unroll
            for (int sb = 0; sb < 2; ++sb) {
                if (sb > (wave >> 1)) continue;
                o[c] = mfma16_bf16(p[sb], load16(&s_u[1][c][sb][lane][0]), o[c]);
                o[c] = mfma16_bf16(p[sb], load16(&s_u[0][c][sb][lane][0]), o[c]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = t0 + tile_token(wave, 4 * g + e);
                if (i < n) a.out[v0 + (size_t)i * sv + 16 * c] = (__bf16)o[c][e];
            }
        }
        if (chunk + 1 < chunks) {
            stage(buf ^ 1);
            put_state();
            lds_barrier();
        }
    }
#pragma unroll
    for (int j = 0; j < TILES; ++j)
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                Hu[(size_t)tile_token(m0 + j, 4 * g + e) * s.DV + 16 * c] = st[j][c][e];
}

// ---- host

static bool chunked(const bole_delta_dims_t &d) {
    return d.factor_dtype == BOLE_DTYPE_BF16 && !(d.flags & BOLE_FLAG_FORCE_GENERIC) &&
           (d.d_k == 64 || d.d_k == 128) && d.d_v % 16 == 0;
}

static size_t slots_of(const bole_delta_dims_t &d) {
    return (size_t)d.total_tokens / kChunk + (size_t)d.batch;
}

size_t delta_prefill_workspace(const bole_delta_dims_t &d) {
    return chunked(d) ? slots_of(d) * (size_t)d.heads * sizeof(ChunkSystem) : 0;
}

template <int DK, int NT>
static void launch_scan(const PrefillArgs &a, hipStream_t stream) {
    const int units = a.s.B * a.s.H, groups = a.s.DV / (16 * NT);
    const unsigned grid = (unsigned)((units + 7) / 8) * 8u * (unsigned)groups;
    delta_scan_kernel<DK, NT><<<dim3(grid), dim3(256), 0, stream>>>(a, units, groups);
}

template <int DK>
static hipError_t launch_chunked(const PrefillArgs &a, size_t slots, hipStream_t stream) {
    if (a.s.T > 0) {
        delta_chunk_kernel<DK><<<dim3((unsigned)(slots * a.s.H)), dim3(256), 0, stream>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    launch_scan<DK, 1>(a, stream);
    return hipGetLastError();
}

hipError_t launch_delta_prefill(float *H0, const void *q, const void *k, const void *v,
                                const float *gate, const float *beta, const int32_t *seq_offsets,
                                void *out, void *workspace, const bole_delta_dims_t &d,
                                int32_t *seq_status, hipStream_t stream) {
    const bool aligned = (reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k)) % 16 == 0;
    if (!chunked(d) || !aligned)
        return launch_delta_prefill_walk(H0, q, k, v, gate, beta, seq_offsets, out, d, seq_status,
                                         stream);
    const PrefillArgs a = {H0, static_cast<const __bf16 *>(q), static_cast<const __bf16 *>(k),
                           static_cast<const __bf16 *>(v), gate, beta, seq_offsets,
                           static_cast<__bf16 *>(out), seq_status,
                           static_cast<ChunkSystem *>(workspace),
                           {d.batch, d.heads, d.key_heads, d.d_k, d.d_v, d.total_tokens}};
    return d.d_k == 64 ? launch_chunked<64>(a, slots_of(d), stream)
                       : launch_chunked<128>(a, slots_of(d), stream);
}

}  // namespace bole
