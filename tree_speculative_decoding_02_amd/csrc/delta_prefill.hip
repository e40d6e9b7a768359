// delta_prefill.hip - prompts through the gated delta rule, 64 tokens at a time.
//
// Within a chunk the updates U of all tokens solve one triangular system (delta_mfma.h), and
// with the chunk's start state S, start_i = 2^{L_i} and end_i = 2^{L_C - L_i}:
//     R = V - diag(start) K S,   U = X diag(b) R,   O = diag(start) Q S + P U,
//     S <- start_C S + K^T diag(end) U.
// X and P do not depend on the state: a first kernel forms them for every chunk and head at
// once and writes them to the workspace. A second one walks each sequence's chunks in order
// with the state in registers.
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
template <typename TF>
struct ChunkSystem {
    static constexpr int kP = sizeof(TF) == 2 ? 1 : 3;
    __bf16 x[3][kPieces][64][8];  // X diag(b), three terms
    __bf16 p[kP][kPieces][64][8]; // P
    float start[kChunk], end[kChunk];
};

__device__ __forceinline__ int piece_of(int m, int s) { return s == 0 ? m : 2 + m; }

template <typename TF>
struct PrefillArgs {
    float *H0;
    const TF *q, *k, *v;
    const float *gate, *beta;
    const int32_t *offsets;
    TF *out;
    int32_t *status;
    ChunkSystem<TF> *ws;
    DeltaShape s;
};

// One workgroup a chunk and value head. Most of its time is waiting, for rows, sums and the inverse's
// steps, so what counts is how many run: 33 KB of LDS and up to 128 registers are four a CU. (One
// 32768-token prompt of 32 heads, 16384 systems: 199 us, 181 with warm clocks, 0.4 GB written; with P
// in LDS and K's rows from the caches three a CU and 249 us.)
template <typename TF, int DK, bool WHOLE>
__global__ __launch_bounds__(256, sizeof(TF) == 2 ? 4 : 2) void delta_chunk_kernel(const PrefillArgs<TF> a) {
    __shared__ DeltaTokens t;
    const DeltaShape &s = a.s;
    const int h = blockIdx.x % s.H, slot = blockIdx.x / s.H, hk = h / (s.H / s.HK);
    const int tid = threadIdx.x, lane = lane_id(), wave = tid >> 6, col = lane & 15, g = lane >> 4;
    const Located l = locate(a.offsets, s.B, s.T, kChunk, slot);
    if (!l.found) return;
    const int done = (slot - l.slot0) * kChunk, lo = l.lo + done, n = min(kChunk, l.n - done);
    if (n <= 0) return;
    ChunkSystem<TF> &w = a.ws[(size_t)slot * s.H + h];
    const int dk = WHOLE ? DK : s.DK;
    const size_t sk = (size_t)s.HK * dk, row0 = (size_t)lo * sk + (size_t)hk * dk;
    SystemRows<TF, DK, WHOLE, false> rows;
    rows.load(a.k + row0, a.q + row0, sk, dk, n);
    if (tid < 64) {
        // tokens past the last do not decay and have no strength
        const bool in = tid < n;
        const size_t at = (size_t)(lo + min(tid, n - 1)) * s.H + h;
        const double L = wave_sum_up_f64(in ? (double)log2_decay(a.gate[at]) : 0.0);
        t.L[tid] = (float)L;
        t.Lrest[tid] = (float)(L - (double)(float)L);
        t.beta[tid] = in ? a.beta[at] : 0.f;
        const double all = shfl_f64(L, 63);
        w.start[tid] = in ? __builtin_amdgcn_exp2f((float)L) : 0.f;
        w.end[tid] = in ? __builtin_amdgcn_exp2f((float)(all - L)) : 0.f;
    }
    rows.share(t.X);
    lds_barrier();
    f32x4 pair[4];
    pair_products(t, rows, a.k + row0, sk, dk, n, pair);
#pragma unroll
    for (int sb = 0; sb < 2; ++sb) {
        if (sb > (wave >> 1)) continue;
        constexpr int NP = ChunkSystem<TF>::kP;
        bf16x8 p[NP];
        split_terms8<NP>(pair[2 * sb], pair[2 * sb + 1], p);
#pragma unroll
        for (int i = 0; i < NP; ++i)
            *reinterpret_cast<bf16x8 *>(&w.p[i][piece_of(wave, sb)][lane][0]) = p[i];
    }
    lds_barrier();
    invert_system(t, n);
#pragma unroll
    for (int sb = 0; sb < 2; ++sb) {
        if (sb > (wave >> 1)) continue;
        f32x4 x, y;
        x_piece(t, tile_token(wave, col), 32 * sb + 8 * g, 32 * sb + 8 * g + 4, x, y);
        bf16x8 xt[3];
        split_terms8<3>(x, y, xt);
#pragma unroll
        for (int i = 0; i < 3; ++i)
            *reinterpret_cast<bf16x8 *>(&w.x[i][piece_of(wave, sb)][lane][0]) = xt[i];
    }
}

// K in LDS: element (row, 8 c + x) of part c. A row's 16-byte parts are permuted by its number, so
// that an operand's rows (tile_token's order) and the four rows of a transposing read lie in
// distinct banks.
template <int DK>
__device__ __forceinline__ int k_at(int row, int c) {
    return row * DK + 8 * (c ^ (DK == 128 ? ((row & 3) << 2 | ((row >> 2) & 3))
                                          : (((row >> 1) & 1) << 2 | ((row >> 3) & 3))));
}

// One workgroup: eight wavefronts, 16 state columns. What bounds one alone is the chain of a chunk's
// steps (K S, then U, then the state), so four wavefronts do only these: wavefront w has the
// tokens of row tile w and the state rows of d_k / 64 row tiles, and what it computes becomes
// the others' operand through LDS (S, then R, then U; three barriers a chunk). In operand
// order every exchange is a lane's own 8 or 16 bytes. The other four, one more on each SIMD,
// do what nobody waits for: they bring K into one of two LDS buffers and compute and store the
// outputs. Operands are loaded for the next chunk as soon as this one has used them.
//
// Measured, one 32768-token prompt of 32 heads (256 workgroups of 512 chunks): 1.3 us a chunk, of
// which LDS is at work for half and the matrix cores for a quarter; 2.1 us with four wavefronts that
// do everything, 4.6 us with wavefronts that do all 64 tokens of 16 columns of their own and
// exchange nothing, 1.6 us with K S in parts by state rows (no exchange of S, one of the sums).
// A second workgroup on the CU hides nothing: of 8192-token prompts one takes 188 us, two (two
// workgroups a CU) 360, four 706, with the units as busy as before (LDS 49 %, vector ALU 38 %, matrix
// cores 27 %). There the CU's throughput counts: 2.8 us for a step of both.
//
// fp32 factors: K lies in LDS as three bf16 terms, Q, U and P are taken as three too, and every
// product as the six of them that reach 2^-24; one workgroup a CU.
//
// WHOLE: d_k = DK and d_v is a multiple of 16. Otherwise both are multiples of 8; parts of rows
// from d_k on count as zero, lanes past the last column load what they do not store.
template <typename TF, int DK, bool WHOLE>
__global__ __launch_bounds__(512, sizeof(TF) == 2 ? 4 : 2) void delta_scan_kernel(
    const PrefillArgs<TF> a, int units, int groups) {
    typedef ChunkSystem<TF> System;
    typedef TF tf4 __attribute__((ext_vector_type(4)));
    constexpr int NK = Terms<TF>::K, NS = Terms<TF>::S, SZ = sizeof(TF);
    constexpr int KS = DK / 32, TILES = DK / 64, CH = DK / 8, PER = kChunk * CH / 256;
    __shared__ __align__(16) __bf16 s_k[2][NK][kChunk * DK];
    __shared__ __align__(16) __bf16 s_s[3][KS][64][8];   // state, three terms
    __shared__ __align__(16) __bf16 s_r[3][2][64][8];    // R
    __shared__ __align__(16) __bf16 s_e[3][2][64][8];    // end U, for the state
    __shared__ __align__(16) __bf16 s_u[NS][2][64][8];   // U, for the output
    __shared__ __align__(16) TF s_v[2][kChunk * 16];     // V, the workgroup's columns
    __shared__ __align__(16) float s_w[2][2 * kChunk];   // start, end
    const DeltaShape &s = a.s;
    // the column groups of a unit go to one XCD (workgroups are dealt to the eight in turn):
    // they read the same rows and systems, and fill each other's output lines
    const int unit = (int)(blockIdx.x / 8 / groups) * 8 + (int)(blockIdx.x % 8);
    const int cg = (int)(blockIdx.x / 8) % groups;
    if (unit >= units) return;
    const int lane = lane_id(), col = lane & 15, g = lane >> 4, tid = threadIdx.x & 255;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const bool chain = __builtin_amdgcn_readfirstlane((int)threadIdx.x) < 256;
    const int b = unit / s.H, h = unit - b * s.H, hk = h / (s.H / s.HK);
    const bool ordered = offsets_ordered(a.offsets, s.B, s.T);
    if (h == 0 && cg == 0 && threadIdx.x == 0 && a.status)
        a.status[b] = ordered ? BOLE_TREE_OK : BOLE_TREE_BAD_SIZE;
    if (!ordered) return;
    const int lo = __builtin_amdgcn_readfirstlane(a.offsets[b]);
    const int n = __builtin_amdgcn_readfirstlane(a.offsets[b + 1]) - lo;
    if (n == 0) return;
    const int chunks = (n + kChunk - 1) / kChunk;
    // addresses are a chunk's (scalar) plus a lane's 32-bit offset in bytes
    const int dk = WHOLE ? DK : s.DK;
    const uint32_t skb = (uint32_t)s.HK * dk * SZ, svb = (uint32_t)s.H * s.DV * SZ;
    const size_t c0 = ((size_t)h * s.DV + 16 * cg) * SZ;
    const char *ws = reinterpret_cast<const char *>(a.ws + ((size_t)(lo / kChunk + b)) * s.H + h);
    const size_t ws_step = (size_t)s.H * sizeof(System);
    // Rows past the last token repeat it: their columns of X diag(b) and their `end` are zero,
    // and their outputs are not stored. Past the last chunk it is loaded again.
    const int my_row = tile_token(wave, col), my_token = tile_token(wave, 4 * g);

    // a row tile's four values a lane, as the terms of the B operand
    auto put = [&](const f32x4 &x, int m, auto &dst) {
        constexpr int N = sizeof(dst) / sizeof(dst[0]);
        bf16x2 y[2][N];
        split_terms2<N>(__builtin_shufflevector(x, x, 0, 1), y[0]);
        split_terms2<N>(__builtin_shufflevector(x, x, 2, 3), y[1]);
#pragma unroll
        for (int i = 0; i < N; ++i)
            *reinterpret_cast<bf16x4 *>(&dst[i][m >> 1][lane][4 * (m & 1)]) =
                __builtin_shufflevector(y[0][i], y[1][i], 0, 1, 2, 3);
    };

    if (chain) {
        // register e of state row tile j: row tile_token(m0 + j, 4 g + e), as tokens are laid out
        const int m0 = wave * TILES;
        char *Hu = reinterpret_cast<char *>(a.H0 + (size_t)unit * dk * s.DV + 16 * cg);
        const uint32_t hrow = (uint32_t)s.DV * 4;
        auto state_at = [&](int j, int e) -> float & {
            return *reinterpret_cast<float *>(Hu + (uint32_t)tile_token(m0 + j, 4 * g + e) * hrow + 4 * col);
        };
        auto state_has = [&](int j, int e) {
            return WHOLE || (tile_token(m0 + j, 4 * g + e) < dk && 16 * cg + col < s.DV);
        };
        f32x4 st[TILES];
#pragma unroll
        for (int j = 0; j < TILES; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) st[j][e] = state_has(j, e) ? state_at(j, e) : 0.f;
        bf16x8 x[2][3];
        // right of the diagonal X is zero: the first two wavefronts' second piece
#pragma unroll
        for (int i = 0; i < 3; ++i) x[1][i] = (bf16x8)(__bf16)0.f;
        auto fetch_x = [&](int chunk) {
            const System &w = *reinterpret_cast<const System *>(ws + min(chunk, chunks - 1) * ws_step);
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                x[0][i] = load16(&w.x[i][piece_of(wave, 0)][lane][0]);
                if (wave >= 2) x[1][i] = load16(&w.x[i][piece_of(wave, 1)][lane][0]);
            }
        };
        fetch_x(0);
#pragma unroll
        for (int j = 0; j < TILES; ++j) put(st[j], m0 + j, s_s);
        lds_barrier();
        for (int chunk = 0; chunk < chunks; ++chunk) {
            const int buf = chunk & 1;
            // ---- R = V - diag(start) K S for the wavefront's tokens, a sum for each term of S
            f32x4 r[3];
#pragma unroll
            for (int i = 0; i < 3; ++i) r[i] = (f32x4)0.f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                bf16x8 ka[NK];
#pragma unroll
                for (int j = 0; j < NK; ++j) ka[j] = load16(&s_k[buf][j][k_at<DK>(my_row, 4 * ks + g)]);
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    const bf16x8 sb = load16(&s_s[i][ks][lane][0]);
#pragma unroll
                    for (int j = 0; j < NK && i + j < 3; ++j) r[i + j] = mfma16_bf16(ka[j], sb, r[i + j]);
                }
            }
            const f32x4 start = *reinterpret_cast<const f32x4 *>(&s_w[buf][my_token]);
            tf4 v;
            if constexpr (SZ == 2) {
                v = read_transposed(&s_v[buf][(my_token + (col >> 2)) * 16 + 4 * (col & 3)]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = s_v[buf][(my_token + e) * 16 + col];
            }
            r[0] += r[2] + r[1];
#pragma unroll
            for (int e = 0; e < 4; ++e) r[0][e] = fmaf(-start[e], r[0][e], (float)v[e]);
            put(r[0], wave, s_r);
            lds_barrier();
            // ---- U = X diag(b) R, a sum for each size of product and half
            f32x4 u[2][3];
#pragma unroll
            for (int sb = 0; sb < 2; ++sb) {
                bf16x8 rb[3];
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    rb[i] = load16(&s_r[i][sb][lane][0]);
                    u[sb][i] = (f32x4)0.f;
                }
#pragma unroll
                for (int i = 0; i < 3; ++i)
#pragma unroll
                    for (int k = 0; k <= i; ++k) u[sb][i] = mfma16_bf16(x[sb][k], rb[i - k], u[sb][i]);
            }
            const f32x4 end = *reinterpret_cast<const f32x4 *>(&s_w[buf][kChunk + my_token]);
            u[0][0] += u[1][0] + ((u[0][2] + u[1][2]) + (u[0][1] + u[1][1]));
            put(end * u[0][0], wave, s_e);
            put(u[0][0], wave, s_u);
            fetch_x(chunk + 1);
            lds_barrier();
            // ---- S <- decay S + K^T (end U): K^T through the transposing read
            const float d = s_w[buf][min(n - chunk * kChunk, kChunk) - 1];
            bf16x8 eb[2][3];
#pragma unroll
            for (int sb = 0; sb < 2; ++sb)
#pragma unroll
                for (int i = 0; i < 3; ++i) eb[sb][i] = load16(&s_e[i][sb][lane][0]);
#pragma unroll
            for (int j = 0; j < TILES; ++j) {
                const int m = m0 + j;
                f32x4 y[2];
                y[0] = st[j] * d;
                y[1] = (f32x4)0.f;
#pragma unroll
                for (int sb = 0; sb < 2; ++sb) {
                    // state rows of lanes 4c .. 4c + 3: 32 (m / 2) + 8 c + 4 (m % 2) ..
                    const int row = 32 * sb + 8 * g + (col >> 2), c = 4 * (m >> 1) + (col & 3);
                    bf16x8 ka[NK];
#pragma unroll
                    for (int i = 0; i < NK; ++i)
                        ka[i] = join(read_transposed(&s_k[buf][i][k_at<DK>(row, c) + 4 * (m & 1)]),
                                     read_transposed(&s_k[buf][i][k_at<DK>(row + 4, c) + 4 * (m & 1)]));
                    y[sb] = mfma_terms(ka, eb[sb], y[sb]);
                }
                st[j] = y[0] + y[1];
                put(st[j], m, s_s);
            }
            lds_barrier();
        }
#pragma unroll
        for (int j = 0; j < TILES; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (state_has(j, e)) state_at(j, e) = st[j][e];
    } else {
        const char *kb = reinterpret_cast<const char *>(a.k) + (size_t)lo * skb + (size_t)hk * dk * SZ;
        const char *qb = reinterpret_cast<const char *>(a.q) + (size_t)lo * skb + (size_t)hk * dk * SZ;
        const char *vb = reinterpret_cast<const char *>(a.v) + (size_t)lo * svb + c0;
        char *ob = reinterpret_cast<char *>(a.out) + (size_t)lo * svb + c0;
        constexpr int VP = 16 * SZ / 16, VT = kChunk * VP;     // 16-byte parts of a V row, of V
        const bool has_part = WHOLE || 8 * (tid % CH) < dk;    // of K
        const bool has_v = WHOLE || 16 * cg + 16 / SZ * (tid % VP) < s.DV;
        const uint32_t koff = (uint32_t)(tid / CH) * skb + 8 * SZ * (tid % CH), qoff = my_row * skb + 8 * SZ * g,
                       ooff = my_row * svb + 4 * SZ * g;
        RowPart<TF> kr[PER], q[KS];
        bf16x8 p[2][System::kP], vr = (bf16x8)(__bf16)0.f, wr;
#pragma unroll
        for (int j = 0; j < PER; ++j) kr[j].clear();
        // with K: V by the first threads, start and end (512 bytes) by 32 others
        auto fetch_k = [&](int t0, int last, const System &w) {
            const char *k0 = kb + (size_t)t0 * skb;
            constexpr int ROWS = 256 / CH;
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                uint32_t off = koff + ROWS * j * skb;
                if (last < kChunk - 1) off = min(tid / CH + ROWS * j, last) * skb + 8 * SZ * (tid % CH);
                if (has_part) kr[j].load(reinterpret_cast<const TF *>(k0 + off));
            }
            if (tid < VT && has_v)
                vr = load16(reinterpret_cast<const __bf16 *>(
                    vb + (size_t)t0 * svb + (uint32_t)min(tid / VP, last) * svb + 16 * (tid % VP)));
            if (tid >= 224) wr = load16(reinterpret_cast<const __bf16 *>(&w.start[0]) + 8 * (tid - 224));
        };
        auto fetch_q = [&](int t0, int last) {
            const char *q0 = qb + (size_t)t0 * skb;
            uint32_t off = qoff;
            if (last < kChunk - 1) off = min(my_row, last) * skb + 8 * SZ * g;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                if (!WHOLE) q[ks].clear();
                if (WHOLE || 32 * ks + 8 * g < dk) q[ks].load(reinterpret_cast<const TF *>(q0 + off + 32 * SZ * ks));
            }
        };
        auto fetch_p = [&](const System &w) {
#pragma unroll
            for (int i = 0; i < System::kP; ++i) {
                p[0][i] = load16(&w.p[i][piece_of(wave, 0)][lane][0]);
                if (wave >= 2) p[1][i] = load16(&w.p[i][piece_of(wave, 1)][lane][0]);
            }
        };
#pragma unroll
        for (int i = 0; i < System::kP; ++i) p[1][i] = (bf16x8)(__bf16)0.f;
        auto stage = [&](int buf) {
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                bf16x8 y[NK];
                kr[j].terms(y);
#pragma unroll
                for (int i = 0; i < NK; ++i)
                    *reinterpret_cast<bf16x8 *>(&s_k[buf][i][k_at<DK>(tid / CH + 256 / CH * j, tid % CH)]) = y[i];
            }
            if (tid < VT) *reinterpret_cast<bf16x8 *>(reinterpret_cast<char *>(&s_v[buf][0]) + 16 * tid) = vr;
            if (tid >= 224) *reinterpret_cast<bf16x8 *>(&s_w[buf][4 * (tid - 224)]) = wr;
        };
        auto chunk_at = [&](int chunk, int &t0, int &last) -> const System & {
            const int c = min(chunk, chunks - 1);
            t0 = c * kChunk;
            last = min(kChunk, n - t0) - 1;
            return *reinterpret_cast<const System *>(ws + c * ws_step);
        };
        int t1, last;
        {
            const System &w = chunk_at(0, t1, last);
            fetch_k(t1, last, w);
            fetch_q(t1, last);
            fetch_p(w);
            stage(0);
            const System &w1 = chunk_at(1, t1, last);
            fetch_k(t1, last, w1);
        }
        lds_barrier();
        // The lines of a chunk, dealt to the threads of the unit's workgroups: each reads its own
        // kAhead chunks early and drops it, so that what the workgroups load one chunk ahead waits in
        // their XCD's L2 (a load is dropped two chunks later, when it has long arrived). One
        // 32768-token prompt: 932 -> 851 us; what fits the last-level cache gains 0 to 3 %.
        constexpr int kAhead = 3;
        const int line_k = (dk * SZ + 127) / 128, line_v = (s.DV * SZ + 127) / 128, line_w = sizeof(System) / 128;
        const char *touch = ws;
        size_t touch_step = ws_step;
        int line = tid * groups + cg;
        bool touches = true;
        if (line < line_w) {
            touch += 128 * line;
        } else if ((line -= line_w) < 2 * kChunk * line_k) {
            touch_step = (size_t)kChunk * skb;
            touch = line < kChunk * line_k ? kb : qb;
            line %= kChunk * line_k;
            touch += (size_t)(line / line_k) * skb + 128 * (line % line_k);
        } else if ((line -= 2 * kChunk * line_k) < kChunk * line_v) {
            touch_step = (size_t)kChunk * svb;
            touch = reinterpret_cast<const char *>(a.v) + (size_t)lo * svb + (size_t)h * s.DV * SZ +
                    (size_t)(line / line_v) * svb + 128 * (line % line_v);
        } else {
            touches = false;
        }
        uint32_t touched[2] = {};
        auto step = [&](int chunk, uint32_t &mine) {
            const System &w = chunk_at(chunk + 1, t1, last);
            // ---- O^T = S^T Q^T diag(start): a lane has four columns of one token's row (the
            // state's pieces serve as left operands just as they do as right ones)
            f32x4 o = (f32x4)0.f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                bf16x8 sb[NS], qt[NK];
                q[ks].terms(qt);
#pragma unroll
                for (int i = 0; i < NS; ++i) sb[i] = load16(&s_s[i][ks][lane][0]);
#pragma unroll
                for (int i = NS - 1; i >= 0; --i)
#pragma unroll
                    for (int j = 0; j < NK && i + j < NS; ++j) o = mfma16_bf16(sb[i], qt[j], o);
            }
            o *= s_w[chunk & 1][my_row];
            fetch_q(t1, last);
            lds_barrier();
            stage((chunk + 1) & 1);
            const System &w2 = chunk_at(chunk + 2, t1, last);
            fetch_k(t1, last, w2);
            asm volatile("" :: "v"(mine));
            if (touches && (chunk + kAhead + 1) * kChunk <= n)
                mine = *reinterpret_cast<const uint32_t *>(touch + (size_t)(chunk + kAhead) * touch_step);
            lds_barrier();
            // ---- O^T += U^T P^T
#pragma unroll
            for (int sb = 0; sb < 2; ++sb) {
                bf16x8 ub[NS];
#pragma unroll
                for (int i = 0; i < NS; ++i) ub[i] = load16(&s_u[i][sb][lane][0]);
#pragma unroll
                for (int i = NS - 1; i >= 0; --i)
#pragma unroll
                    for (int j = 0; j < System::kP && i + j < NS; ++j) o = mfma16_bf16(ub[i], p[sb][j], o);
            }
            fetch_p(w);
            if (chunk * kChunk + my_row < n && (WHOLE || 16 * cg + 4 * g < s.DV))
                *reinterpret_cast<tf4 *>(ob + (size_t)(chunk * kChunk) * svb + ooff) =
                    __builtin_convertvector(o, tf4);
            lds_barrier();
        };
        for (int chunk = 0; chunk < chunks; ++chunk) {
            step(chunk, touched[0]);
            if (++chunk < chunks) step(chunk, touched[1]);
        }
    }
}

// ---- host

static bool chunked(const bole_delta_dims_t &d) {
    // row offsets within a chunk are 32-bit
    const int64_t row = (int64_t)d.heads * (d.d_v > d.d_k ? d.d_v : d.d_k) * (d.factor_dtype == BOLE_DTYPE_F32 ? 4 : 2);
    return !(d.flags & BOLE_FLAG_FORCE_GENERIC) && d.d_k <= 128 && d.d_k % 8 == 0 && d.d_v % 8 == 0 &&
           row * kChunk <= 0x7fffffffLL;
}

static size_t slots_of(const bole_delta_dims_t &d) {
    return (size_t)d.total_tokens / kChunk + (size_t)d.batch;
}

size_t delta_prefill_workspace(const bole_delta_dims_t &d) {
    if (!chunked(d)) return 0;
    return slots_of(d) * (size_t)d.heads *
           (d.factor_dtype == BOLE_DTYPE_F32 ? sizeof(ChunkSystem<float>) : sizeof(ChunkSystem<__bf16>));
}

template <typename TF, int DK, bool WHOLE>
static hipError_t launch_chunked(const PrefillArgs<TF> &a, size_t slots, hipStream_t stream) {
    if (a.s.T > 0) {
        delta_chunk_kernel<TF, DK, WHOLE><<<dim3((unsigned)(slots * a.s.H)), dim3(256), 0, stream>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const int units = a.s.B * a.s.H, groups = (a.s.DV + 15) / 16;
    const unsigned grid = (unsigned)((units + 7) / 8) * 8u * (unsigned)groups;
    delta_scan_kernel<TF, DK, WHOLE><<<dim3(grid), dim3(512), 0, stream>>>(a, units, groups);
    return hipGetLastError();
}

template <typename TF>
static hipError_t launch_typed(float *H0, const void *q, const void *k, const void *v,
                               const float *gate, const float *beta, const int32_t *seq_offsets,
                               void *out, void *workspace, const bole_delta_dims_t &d,
                               int32_t *seq_status, hipStream_t stream) {
    const PrefillArgs<TF> a = {H0, static_cast<const TF *>(q), static_cast<const TF *>(k),
                               static_cast<const TF *>(v), gate, beta, seq_offsets,
                               static_cast<TF *>(out), seq_status,
                               static_cast<ChunkSystem<TF> *>(workspace),
                               {d.batch, d.heads, d.key_heads, d.d_k, d.d_v, d.total_tokens}};
    const size_t slots = slots_of(d);
    if (d.d_v % 16 == 0 && d.d_k == 64) return launch_chunked<TF, 64, true>(a, slots, stream);
    if (d.d_v % 16 == 0 && d.d_k == 128) return launch_chunked<TF, 128, true>(a, slots, stream);
    return d.d_k <= 64 ? launch_chunked<TF, 64, false>(a, slots, stream)
                       : launch_chunked<TF, 128, false>(a, slots, stream);
}

hipError_t launch_delta_prefill(float *H0, const void *q, const void *k, const void *v,
                                const float *gate, const float *beta, const int32_t *seq_offsets,
                                void *out, void *workspace, const bole_delta_dims_t &d,
                                int32_t *seq_status, hipStream_t stream) {
    const uintptr_t rows = reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) |
                           reinterpret_cast<uintptr_t>(v) | reinterpret_cast<uintptr_t>(out);
    if (!chunked(d) || rows % 16 != 0)
        return launch_delta_prefill_walk(H0, q, k, v, gate, beta, seq_offsets, out, d, seq_status,
                                         stream);
    return d.factor_dtype == BOLE_DTYPE_F32
               ? launch_typed<float>(H0, q, k, v, gate, beta, seq_offsets, out, workspace, d,
                                     seq_status, stream)
               : launch_typed<__bf16>(H0, q, k, v, gate, beta, seq_offsets, out, workspace, d,
                                      seq_status, stream);
}

}  // namespace bole
