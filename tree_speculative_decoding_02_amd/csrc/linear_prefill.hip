// linear_prefill.hip - prompts through linear attention with a decay, 64 tokens at a time.
//
// With L_i the cumulative log2-decay of a chunk's tokens and S the state before them,
//     O = diag(2^L) Q S + P V,   P_ij = 2^{L_i - L_j} (q_i . k_j) for j <= i,
//     S <- 2^{L_64} S + K^T diag(2^{L_64 - L}) V.
// Nothing of this waits for anything but S, and S is linear: a sequence is cut into segments of
// whole chunks. A first kernel forms every segment's own contribution to the state, from nothing; a
// second one runs over each sequence's segments and leaves the state that each starts from; a third
// walks each segment's chunks and has the outputs. Keys and values are read twice by this, so a
// segment is as long as leaves the chip filled, and a sequence of one segment skips both.
//
// A workgroup has a segment, a value head and 64 or 128 state columns, 16 or 32 a wavefront, whose
// rows stay in the accumulators of the matrix cores: a product's results in registers are the next
// one's operand (tile_token, delta_mfma.h), so the state never leaves them. K, Q and V pass through
// LDS, the next chunk in registers meanwhile; P's row tiles are formed by a wavefront each and
// exchanged.
//
// Products of decays above 1 may leave fp32 where what they scale is small or zero. A segment with a chunk
// whose decays above 1 multiply to more than 2^64 is taken once more, token by token (H <- a H + k v^T,
// o = H^T q, in the same accumulators), when its chunks are through; others have half of fp32's range for
// what decays scale. (A way out of the chunks' loop, or a test within it, cost all prompts 3 to 12 %, as the
// compiler then orders the loop's reads and products less well.)
//
// The state is kept to fp32: K is exact in bf16, and diag(2^{L_64 - L}) V is taken as three bf16
// terms (2^-25 left). What only the output sees may be rounded harder: S in two terms, P in one (half
// a step of bf16 of each pair weight, once, before an output that is rounded to bf16 itself). With
// fp32 factors K, Q, V, P and S are three terms each.
//
// Measured, 32 heads of 128 x 64 states, bf16: eight prompts of up to 2048 tokens (9412 in all) 116 us
// (31 the first kernel, 10 the second, 71 the third; 2.2 TB/s of what the call cannot do without), one
// prompt of 32768 tokens and 8 key heads 248 us (73, 8 and 163 to 171; 1.7 TB/s). In fp32 eight of up to
// 1000 tokens take 155 us (38, 10 and 102), one workgroup a CU, as K, Q and V are three terms each in LDS.
// What bounds the third is issue: a wavefront's chunk is some 510 vector instructions, about 200 of them
// the splits of S and of the weighed V, and 102 matrix ones, three workgroups a CU, and the one kind
// hardly runs beside the other. With registers for two workgroups and the next chunk's loads earlier it
// took 208 us for the long prompt, with three and no rows ahead 171, when it took 161 as it is.
#include "delta_mfma.h"
#include "linear_device.h"
#include "launch.h"

namespace bole {

// Launch shape: tokens a segment (a multiple of 64), slots (segments of all sequences, spare ones
// among them), groups of columns.
struct LinearPlan {
    int seg, slots, groups;
};

// Workspace (space_slot, linear_device.h), [slot][head]: the state in the order of the accumulators,
// then its decay.
struct LinearSpace {
    f32x4 *s;      // [slot][H][column tile][row tile][64]
    float *decay;  // [slot][H]: its log2
};

// A workgroup's slot, head and column group. Of each slot's heads and groups every XCD (workgroups are
// dealt to the eight in turn) has an eighth, neighbours, as those that share keys read the same lines;
// the spare slots, the last ones, are spread over all.
__device__ __forceinline__ void unit_of(const LinearPlan &p, int H, int &slot, int &h, int &cg) {
    const int each = H * p.groups;  // units of a slot
    int unit = blockIdx.x;
    slot = unit / each;
    unit -= slot * each;
    if (each % 8 == 0) unit = (unit % 8) * (each / 8) + unit / 8;
    h = unit / p.groups;
    cg = unit - h * p.groups;
}

// Product of the values above 1 of a wavefront.
template <int CTRL, int ROWS>
__device__ __forceinline__ float times_dpp(float x) {
    return x * __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(1.f), __float_as_int(x), CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ float product_above(float x) {
    x = x > 1.f ? x : 1.f;
    x = times_dpp<0x111, 0xf>(x);  // as scan_f64
    x = times_dpp<0x112, 0xf>(x);
    x = times_dpp<0x114, 0xf>(x);
    x = times_dpp<0x118, 0xf>(x);
    x = times_dpp<0x142, 0xa>(x);
    x = times_dpp<0x143, 0xc>(x);
    return readlane_f(x, 63);
}

template <int DK>
__device__ __forceinline__ int row_at(int row, int c) {  // as delta_prefill.hip's K
    return row * DK + 8 * (c ^ (DK == 128 ? ((row & 3) << 2 | ((row >> 2) & 3))
                                          : (((row >> 1) & 1) << 2 | ((row >> 3) & 3))));
}

__device__ __forceinline__ int lower_piece(int m, int s) { return s == 0 ? m : 2 + m; }

// LOCAL: a segment's own contribution to the state, from nothing, and its decay; no outputs.
// WHOLE: d_k = DK and the columns fill the groups. Otherwise d_k and d_v are multiples of 8; parts of
// rows from d_k on and of columns from d_v on count as zero.
template <typename TF, int DK, int CT, bool WHOLE, bool LOCAL>
__global__ __launch_bounds__(256, sizeof(TF) == 4 ? 1 : CT == 2 ? 2 : LOCAL ? 4 : 3) void linear_chunk_kernel(
    const LinearArgs a, const LinearPlan p, const LinearSpace w) {
    typedef TF tf4 __attribute__((ext_vector_type(4)));
    constexpr int NK = Terms<TF>::K, NS = Terms<TF>::S;
    constexpr int KS = DK / 32, TILES = DK / 16, CH = DK / 8, PER = kChunk * CH / 256;
    constexpr int VC = 64 * CT, VP = CT == 1 ? 96 : 160, VPER = kChunk * VC / 8 / 256;
    __shared__ __align__(16) __bf16 s_k[NK][kChunk * DK];
    __shared__ __align__(16) __bf16 s_q[LOCAL ? 1 : NK][LOCAL ? 8 : kChunk * DK];
    __shared__ __align__(16) __bf16 s_v[NK][kChunk * VP];
    __shared__ __align__(16) __bf16 s_p[LOCAL ? 1 : NK][6][64][8];
    __shared__ __align__(16) float s_w[2][4][kChunk];  // L in two terms, 2^L, 2^{L_64 - L}
    __shared__ int s_grows;                            // whether some chunk's decays are too large for that
    const DeltaShape &s = a.s;
    int slot, h, cg;
    unit_of(p, s.H, slot, h, cg);
    const int hk = h / (s.H / s.HK);
    const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, g = lane >> 4;
    const Located l = locate(a.offsets, s.B, s.T, p.seg, slot);
    if (!LOCAL && h == 0 && cg == 0 && a.status) {
        if (!l.ordered) {
            if (slot == 0)
                for (int b = tid; b < s.B; b += 256) a.status[b] = BOLE_TREE_BAD_SIZE;
        } else if (l.found && slot == l.slot0 && tid == 0) {
            a.status[l.b] = BOLE_TREE_OK;
        }
    }
    if (!l.found) return;
    const int t0 = (slot - l.slot0) * p.seg;
    if (t0 >= l.n || (LOCAL && t0 + p.seg >= l.n)) return;
    const bool last_seg = t0 + p.seg >= l.n;
    const int n = min(p.seg, l.n - t0), chunks = (n + kChunk - 1) / kChunk;
    const int dk = WHOLE ? DK : s.DK;
    const size_t sk = (size_t)s.HK * dk, sv = (size_t)s.H * s.DV, row0 = (size_t)l.lo + t0;
    const TF *kb = static_cast<const TF *>(a.k) + row0 * sk + (size_t)hk * dk;
    const TF *qb = static_cast<const TF *>(a.q) + row0 * sk + (size_t)hk * dk;
    const TF *vb = static_cast<const TF *>(a.v) + row0 * sv + (size_t)h * s.DV + cg * VC;
    const float *gb = a.gate + row0 * s.H + h;
    const int left = s.DV - cg * VC;  // columns from the group's first on

    // ---- the state: element e of row tile j is row tile_token(j, 4 g + e), column 16 (wave CT + ct) + col
    const int c0 = 16 * wave * CT;
    float *Hu = a.H0 + ((size_t)l.b * s.H + h) * dk * s.DV + cg * VC + c0 + col;
    auto state_has = [&](int ct, int j, int e) {
        return WHOLE || (tile_token(j, 4 * g + e) < dk && c0 + 16 * ct + col < left);
    };
    const size_t at_ws = space_slot(l.lo, p.seg, slot - l.slot0) * s.H + h;
    f32x4 *sw = w.s + (at_ws * p.groups * 4 * CT + (cg * 4 + wave) * CT) * TILES * 64 + lane;
    f32x4 st[CT][TILES];
    // ---- loads: rows past the last token repeat it (they do not decay, and their 2^{L_64 - L} is 0).
    // Addresses are a chunk's (scalar) plus a lane's 32-bit offset in bytes.
    constexpr int SZ = sizeof(TF), ROWS = 256 / CH, VROWS = 256 / (VC / 8);
    const uint32_t skb = (uint32_t)(sk * SZ), svb = (uint32_t)(sv * SZ);
    const int kc = WHOLE || 8 * (tid % CH) < dk ? tid % CH : 0, vc = WHOLE || 8 * (tid % (VC / 8)) < left ? tid % (VC / 8) : 0;
    const uint32_t krow = (uint32_t)(tid / CH) * skb, vrow = (uint32_t)(tid / (VC / 8)) * svb;
    RowPart<TF> kr[PER], qr[LOCAL ? 1 : PER], vr[VPER];
    auto fetch = [&](int chunk) {
        const int first = chunk * kChunk;
        const uint32_t most = min(n - 1 - first, kChunk - 1);
        const char *k0 = reinterpret_cast<const char *>(kb) + (size_t)first * skb;
        const char *q0 = reinterpret_cast<const char *>(qb) + (size_t)first * skb;
        const char *v0 = reinterpret_cast<const char *>(vb) + (size_t)first * svb;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const uint32_t off = min(krow + ROWS * j * skb, most * skb) + 8 * SZ * kc;
            kr[j].load(reinterpret_cast<const TF *>(k0 + off));
            if constexpr (!LOCAL) qr[j].load(reinterpret_cast<const TF *>(q0 + off));
        }
#pragma unroll
        for (int j = 0; j < VPER; ++j) {
            const uint32_t off = min(vrow + VROWS * j * svb, most * svb) + 8 * SZ * vc;
            vr[j].load(reinterpret_cast<const TF *>(v0 + off));
        }
        if (!WHOLE) {
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (8 * (tid % CH) >= dk) {
                    kr[j].clear();
                    if constexpr (!LOCAL) qr[j].clear();
                }
#pragma unroll
            for (int j = 0; j < VPER; ++j)
                if (8 * (tid % (VC / 8)) >= left) vr[j].clear();
        }
    };
    // Places of operand pieces in s_k and s_q: part 4 ks + g of row tile_token(m, col), and rows
    // 32 sb + 8 g + 4 half .. + 3 of a transposing read's part of row tile j. What is added to a row in
    // multiples of 32 leaves its permutation, and a step of ks flips bits of the place: two places each,
    // as all sixteen would take registers that prefetched rows need.
    int opnd[2], trans[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        opnd[x] = row_at<DK>(tile_token(x, col), g);
        trans[x] = row_at<DK>(8 * g + (col >> 2) + 4 * x, col & 3);
    }
    auto operand = [&](const __bf16 *from, int m, int ks) { return load16(from + (opnd[m & 1] ^ 32 * ks) + 32 * (m >> 1) * DK); };
    auto stage = [&]() {
        bf16x8 y[NK];
        static_assert(ROWS % 16 == 0, "rows that keep their permutation");
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int at = row_at<DK>(tid / CH, tid % CH) + ROWS * j * DK;
            kr[j].terms(y);
#pragma unroll
            for (int i = 0; i < NK; ++i) *reinterpret_cast<bf16x8 *>(&s_k[i][at]) = y[i];
            if constexpr (!LOCAL) {
                qr[j].terms(y);
#pragma unroll
                for (int i = 0; i < NK; ++i) *reinterpret_cast<bf16x8 *>(&s_q[i][at]) = y[i];
            }
        }
#pragma unroll
        for (int j = 0; j < VPER; ++j) {
            const int e = tid + 256 * j;
            vr[j].terms(y);
#pragma unroll
            for (int i = 0; i < NK; ++i)
                *reinterpret_cast<bf16x8 *>(&s_v[i][e / (VC / 8) * VP + 8 * (e % (VC / 8))]) = y[i];
        }
    };
    // decays of a chunk's tokens, by one wavefront: a token a lane
    auto fetch_gate = [&](int chunk) {
        const int t = chunk * kChunk + lane;
        return t < n ? gb[(size_t)t * s.H] : 1.f;
    };
    double total = 0.0;
    auto weigh = [&](int chunk, float gate) {
        const double L = scan_f64((double)log2_decay(gate)), all = shfl_f64(L, 63);
        float(*to)[kChunk] = s_w[chunk & 1];
        to[0][lane] = (float)L;
        to[1][lane] = (float)(L - (double)(float)L);
        to[2][lane] = __builtin_amdgcn_exp2f((float)L);
        to[3][lane] = chunk * kChunk + lane < n ? __builtin_amdgcn_exp2f((float)(all - L)) : 0.f;
        if (__any(gate > 1.f) && product_above(gate) > 0x1p64f) s_grows = 1;
        total += all;
    };

    auto first_state = [&]() {
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int j = 0; j < TILES; ++j) {
                st[ct][j] = (f32x4)0.f;
                if (LOCAL) continue;
                if (l.n > p.seg) {
                    st[ct][j] = sw[(ct * TILES + j) * 64];
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (state_has(ct, j, e)) st[ct][j][e] = Hu[(size_t)tile_token(j, 4 * g + e) * s.DV + 16 * ct];
                }
            }
    };
    fetch(0);
    first_state();
    float gate_next = 1.f;
    if (wave == 0) {
        const float gate = fetch_gate(0);
        gate_next = fetch_gate(1);
        s_grows = 0;
        weigh(0, gate);
    }
    stage();
    lds_barrier();
    char *ob = reinterpret_cast<char *>(static_cast<TF *>(a.out) + row0 * sv + (size_t)h * s.DV + cg * VC);
    const uint32_t ooff = (uint32_t)tile_token(0, col) * svb + (c0 + 4 * g) * SZ;
    int chunk = 0;
    do {
#pragma unroll
        for (int x = 0; x < 2; ++x) asm volatile("" : "+v"(opnd[x]), "+v"(trans[x]));  // (worked out anew in each turn)
        const float(*wt)[kChunk] = s_w[chunk & 1];
        f32x4 o[CT][4];
        if constexpr (!LOCAL) {
            // ---- P: the wavefront's row tile, as operand pieces
            const int i = tile_token(wave, col), above = i - 8 * g;  // j <= i in each lane's own numbers
            const float li = wt[0][i], lr = wt[1][i];
            f32x4 pair[4];
            bf16x8 own_q[KS][NK];
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int t = 0; t < NK; ++t) own_q[ks][t] = load16(s_q[t] + ((wave & 1 ? opnd[1] : opnd[0]) ^ 32 * ks) + 32 * (wave >> 1) * DK);
#pragma unroll
            for (int jt = 0; jt < 4; ++jt) {
                pair[jt] = (f32x4)0.f;
                if (jt >> 1 > wave >> 1) continue;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    bf16x8 x[NK];
#pragma unroll
                    for (int t = 0; t < NK; ++t) x[t] = operand(s_k[t], jt, ks);
                    pair[jt] = mfma_terms(x, own_q[ks], pair[jt]);
                }
                const int j0 = tile_token(jt, 4 * g);
                const f32x4 lj = *reinterpret_cast<const f32x4 *>(&wt[0][j0]);
                const f32x4 ljr = *reinterpret_cast<const f32x4 *>(&wt[1][j0]);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    pair[jt][r] *= tile_token(jt, 0) + r <= above ? __builtin_amdgcn_exp2f((li - lj[r]) + (lr - ljr[r])) : 0.f;
            }
#pragma unroll
            for (int sb = 0; sb < 2; ++sb) {
                if (sb > wave >> 1) continue;
                bf16x8 y[NK];
                split_terms8<NK>(pair[2 * sb], pair[2 * sb + 1], y);
#pragma unroll
                for (int t = 0; t < NK; ++t)
                    *reinterpret_cast<bf16x8 *>(&s_p[t][lower_piece(wave, sb)][lane][0]) = y[t];
            }
            // ---- O^T = S^T Q^T diag(2^L): a lane has four columns of one token's row
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int m = 0; m < 4; ++m) o[ct][m] = (f32x4)0.f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                bf16x8 sb[CT][NS];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) split_terms8<NS>(st[ct][2 * ks], st[ct][2 * ks + 1], sb[ct]);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    bf16x8 y[NK];
#pragma unroll
                    for (int t = 0; t < NK; ++t) y[t] = operand(s_q[t], m, ks);
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                        for (int x = NS - 1; x >= 0; --x)
#pragma unroll
                            for (int t = 0; t < NK && x + t < NS; ++t) o[ct][m] = mfma16_bf16(sb[ct][x], y[t], o[ct][m]);
                }
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float start = wt[2][tile_token(m, col)];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) o[ct][m] *= start;
            }
            lds_barrier();
        }
        // ---- V's operand pieces: tokens 32 sb + 8 g .. + 7 of the lane's column
        const float decay = wt[2][kChunk - 1];
        bf16x8 v[CT][2][NK], ev[CT][2][3];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int sb = 0; sb < 2; ++sb)
#pragma unroll
                for (int t = 0; t < NK; ++t) {
                    const __bf16 *vp = &s_v[t][(32 * sb + 8 * g + (col >> 2)) * VP + c0 + 16 * ct + 4 * (col & 3)];
                    v[ct][sb][t] = join(read_transposed(vp), read_transposed(vp + 4 * VP));
                }
        if constexpr (!LOCAL) {
            // ---- O^T += V^T P^T
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int sb = 0; sb <= m >> 1; ++sb) {
                    bf16x8 y[NK];
#pragma unroll
                    for (int t = 0; t < NK; ++t) y[t] = load16(&s_p[t][lower_piece(m, sb)][lane][0]);
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) o[ct][m] = mfma_terms(v[ct][sb], y, o[ct][m]);
                }
            char *o0 = ob + (size_t)(chunk * kChunk) * svb;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int token = 32 * (m >> 1) + 4 * (m & 1);  // of the lane's first one
                if (tile_token(0, col) + token >= n - chunk * kChunk) continue;
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
                    if (WHOLE || c0 + 16 * ct + 4 * g < left)
                        *reinterpret_cast<tf4 *>(o0 + (size_t)token * svb + (ooff + 16 * SZ * ct)) =
                            __builtin_convertvector(o[ct][m], tf4);
            }
        }
        fetch(min(chunk + 1, chunks - 1));
        __builtin_amdgcn_sched_barrier(0);  // (they would sink to behind the products)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int sb = 0; sb < 2; ++sb) {
                f32x4 x[2];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e >> 2][e & 3] = (float)v[ct][sb][0][e];
#pragma unroll
                    for (int t = 1; t < NK; ++t) x[e >> 2][e & 3] += (float)v[ct][sb][t][e];
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) x[e] *= *reinterpret_cast<const f32x4 *>(&wt[3][32 * sb + 8 * g + 4 * e]);
                split_terms8<3>(x[0], x[1], ev[ct][sb]);
            }
        // ---- S <- 2^{L_64} S + K^T (diag V)
#pragma unroll
        for (int j = 0; j < TILES; ++j) {
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) st[ct][j] *= decay;
#pragma unroll
            for (int sb = 0; sb < 2; ++sb) {
                bf16x8 x[NK];
#pragma unroll
                for (int t = 0; t < NK; ++t)
                    x[t] = join(read_transposed(s_k[t] + (trans[0] ^ 32 * (j >> 1)) + 32 * sb * DK + 4 * (j & 1)),
                                read_transposed(s_k[t] + (trans[1] ^ 32 * (j >> 1)) + 32 * sb * DK + 4 * (j & 1)));
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) st[ct][j] = mfma_terms(x, ev[ct][sb], st[ct][j]);
            }
        }
        if (wave == 0 && chunk + 1 < chunks) {
            weigh(chunk + 1, gate_next);
            gate_next = fetch_gate(chunk + 2);
        }
        lds_barrier();
        if (chunk + 1 < chunks) {
            stage();
            lds_barrier();
        }
    } while (++chunk < chunks);

    if (__builtin_amdgcn_readfirstlane(s_grows)) {  // ---- once more, token by token
        first_state();
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the outputs written above come before these
#pragma unroll 1
        for (int t = 0; t < n; ++t) {
            const float decay = gb[(size_t)t * s.H];
            const TF *k = kb + (size_t)t * sk, *q = qb + (size_t)t * sk;
            float v[CT], z[CT];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                const int c = c0 + 16 * ct + col;
                v[ct] = WHOLE || c < left ? to_f32(vb[(size_t)t * sv + c]) : 0.f;
                z[ct] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < TILES; ++j) {
                asm volatile("" ::: "memory");  // (all rows' loads at once would take more registers than the loop above)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int row = tile_token(j, 4 * g + e);
                    const bool in = WHOLE || row < dk;
                    const float kr = in ? to_f32(k[row]) : 0.f, qr = !LOCAL && in ? to_f32(q[row]) : 0.f;
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) {
                        st[ct][j][e] = fmaf(kr, v[ct], decay * st[ct][j][e]);
                        z[ct] = fmaf(st[ct][j][e], qr, z[ct]);
                    }
                }
            }
            if constexpr (!LOCAL) {
                TF *o = static_cast<TF *>(a.out) + (row0 + t) * sv + (size_t)h * s.DV + cg * VC + c0 + col;
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    const float y = sum32(sum16(z[ct]));
                    if (g == 0 && (WHOLE || c0 + 16 * ct + col < left)) o[16 * ct] = (TF)y;
                }
            }
        }
    }

    if (LOCAL) {
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int j = 0; j < TILES; ++j) sw[(ct * TILES + j) * 64] = st[ct][j];
        if (tid == 0 && cg == 0) w.decay[at_ws] = (float)total;
    } else if (last_seg) {
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int j = 0; j < TILES; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (state_has(ct, j, e)) Hu[(size_t)tile_token(j, 4 * g + e) * s.DV + 16 * ct] = st[ct][j][e];
    }
}

// Over a sequence's segments: each one's contribution gives way to the state that it starts from. A
// thread has four elements of a state, and eight segments' loads in flight.
__global__ __launch_bounds__(256) void linear_carry_kernel(const LinearArgs a, const LinearPlan p,
                                                           const LinearSpace w, int tiles, int row_tiles) {
    const DeltaShape &s = a.s;
    const int unit = blockIdx.x;  // (a state has a multiple of four tiles of 64 pieces)
    const int piece = blockIdx.y * 256 + threadIdx.x, lane = piece & 63, tile = piece >> 6;
    const int b = unit / s.H, h = unit - b * s.H;
    if (!offsets_ordered(a.offsets, s.B, s.T)) return;
    const int lo = a.offsets[b], n = a.offsets[b + 1] - lo;
    if (n <= p.seg) return;
    const int count = (n + p.seg - 1) / p.seg;
    const int ct = tile / row_tiles, j = tile - ct * row_tiles, col = 16 * ct + (lane & 15);
    const float *Hu = a.H0 + (size_t)unit * s.DK * s.DV;
    f32x4 S;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int row = tile_token(j, 4 * (lane >> 4) + e);
        S[e] = row < s.DK && col < s.DV ? Hu[(size_t)row * s.DV + col] : 0.f;
    }
    const size_t first = space_slot(lo, p.seg, 0) * s.H + h, step = (size_t)s.H * tiles * 64;
    f32x4 *x = w.s + first * tiles * 64 + piece;
    const float *d = w.decay + first;
    for (int i = 0; i < count; i += 8) {
        f32x4 own[8];
        float decay[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int at = min(i + k, count - 2);  // (the last segment's is not needed, and not there)
            own[k] = x[at * step];
            decay[k] = d[(size_t)at * s.H];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (i + k >= count) break;
            x[(i + k) * step] = S;
            // (past fp32's range as two roots, and no infinity, so that what is zero stays zero)
            const bool far = fabsf(decay[k]) > 126.f;
            const float by = __builtin_amdgcn_exp2f(far ? fminf(0.5f * decay[k], 127.9f) : decay[k]);
            if (far) S *= by;
            S = S * by + own[k];
        }
    }
}

// ---- host

static DeltaShape shape(const bole_linear_dims_t &d) {
    return {d.batch, d.heads, d.key_heads, d.d_k, d.d_v, d.total_tokens};
}

static bool chunked(const bole_linear_dims_t &d) {
    // row offsets within a chunk are 32-bit
    const int64_t row = (int64_t)d.heads * (d.d_v > d.d_k ? d.d_v : d.d_k) * (d.factor_dtype == BOLE_DTYPE_F32 ? 4 : 2);
    return !(d.flags & BOLE_FLAG_FORCE_GENERIC) && d.gate_kind == BOLE_GATE_SCALAR && d.d_k <= 128 &&
           d.d_k % 8 == 0 && d.d_v % 8 == 0 && d.batch > 0 && row * kChunk <= 0x7fffffffLL;
}

// Column tiles a wavefront: two, in bf16 from 65 columns on, where the call is cut into segments anyway
// and has four chunks for each of 512 such workgroups: K's and Q's reads from LDS, and P, serve both then
// (32 heads of 128 x 128: one 32768-token prompt 389 us, 454 with one tile; four of up to 2048 106 and
// 121). One otherwise, for twice the workgroups and three of them a CU in place of two (eight of up to
// 2048 142, 173 with two; 16 of them 190 and 239; one of 300 tokens 32 and 40).
static int column_tiles(const bole_linear_dims_t &d) {
    if (d.factor_dtype != BOLE_DTYPE_BF16 || d.d_v <= 64) return 1;
    const int64_t chunks = ((int64_t)d.total_tokens + kChunk - 1) / kChunk;
    const int64_t one = (int64_t)d.heads * ((d.d_v + 63) / 64), two = (int64_t)d.heads * ((d.d_v + 127) / 128);
    return d.batch * one < 512 && chunks * two >= 4 * 512 ? 2 : 1;
}

// From a call's sizes alone. Segments so that 512 workgroups run, of at least four chunks, since each
// costs a state's way through memory, and K and V are read twice (one 32768-token prompt of 32 heads
// 249 us, with 256 workgroups 359, with 768 238; eight of up to 2048 tokens 116, 132 and 103; two of up
// to 4096 58, 69 and 66). Where the sequences alone give 512, they are cut only from four times their
// average length on (32 of up to 2048 tokens 210 us whole, 291 cut at twice the average).
static LinearPlan plan(const bole_linear_dims_t &d) {
    LinearPlan p;
    const int columns = 64 * column_tiles(d);
    p.groups = (d.d_v + columns - 1) / columns;
    const int64_t chunks = (d.total_tokens + kChunk - 1) / kChunk, units = (int64_t)d.heads * p.groups;
    int64_t seg = (chunks * units + 511) / 512;
    if (seg < 4) seg = 4;
    if (d.batch * units >= 512) {
        const int64_t most = 4 * ((chunks + d.batch - 1) / d.batch);
        if (seg < most) seg = most;
    }
    if (seg * kChunk >= d.total_tokens) seg = chunks > 0 ? chunks : 1;
    p.seg = (int)(seg * kChunk);
    p.slots = d.total_tokens / p.seg + d.batch;
    return p;
}

static int row_width(const bole_linear_dims_t &d) { return d.d_k <= 64 ? 64 : 128; }

size_t linear_prefill_workspace(const bole_linear_dims_t &d) {
    const size_t walk = linear_walk_workspace(d);  // (of rows that are not on 16-byte addresses too)
    if (!chunked(d)) return walk;
    const LinearPlan p = plan(d);
    const size_t state = (size_t)p.groups * 64 * column_tiles(d) * row_width(d) + 4;  // (and its decay)
    const size_t need = space_slots(d.total_tokens, p.seg) * d.heads * state * sizeof(float);
    return need > walk ? need : walk;
}

template <typename TF, int DK, int CT, bool WHOLE>
static hipError_t launch_shape(const LinearArgs &a, const LinearPlan &p, const LinearSpace &w, bool cut,
                               hipStream_t stream) {
    const int64_t units = (int64_t)p.slots * a.s.H * p.groups;
    const dim3 grid((unsigned)units), block(256);
    if (cut) {
        linear_chunk_kernel<TF, DK, CT, WHOLE, true><<<grid, block, 0, stream>>>(a, p, w);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        const int tiles = p.groups * 4 * CT * DK / 16;
        linear_carry_kernel<<<dim3((unsigned)(a.s.B * a.s.H), (unsigned)(tiles / 4)), block, 0, stream>>>(a, p, w, tiles,
                                                                                                     DK / 16);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    linear_chunk_kernel<TF, DK, CT, WHOLE, false><<<grid, block, 0, stream>>>(a, p, w);
    return hipGetLastError();
}

template <typename TF, int CT>
static hipError_t launch_width(const LinearArgs &a, const LinearPlan &p, const LinearSpace &w, bool cut,
                               hipStream_t stream) {
    const bool columns = a.s.DV % (64 * CT) == 0;
    if (a.s.DK == 128 && columns) return launch_shape<TF, 128, CT, true>(a, p, w, cut, stream);
    if (a.s.DK == 64 && columns) return launch_shape<TF, 64, CT, true>(a, p, w, cut, stream);
    return a.s.DK <= 64 ? launch_shape<TF, 64, CT, false>(a, p, w, cut, stream)
                        : launch_shape<TF, 128, CT, false>(a, p, w, cut, stream);
}

hipError_t launch_linear_prefill(float *H0, const void *q, const void *k, const void *v,
                                 const float *gate, const int32_t *seq_offsets, void *out,
                                 void *workspace, const bole_linear_dims_t &d, int32_t *seq_status,
                                 hipStream_t stream) {
    const LinearArgs a = {H0, q, k, v, gate, seq_offsets, out, seq_status, shape(d)};
    const uintptr_t rows = reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) |
                           reinterpret_cast<uintptr_t>(v) | reinterpret_cast<uintptr_t>(out);
    if (!chunked(d) || rows % 16 != 0) return launch_linear_walk(a, d, workspace, stream);
    const LinearPlan p = plan(d);
    const size_t n = space_slots(d.total_tokens, p.seg) * d.heads;
    const LinearSpace w = {static_cast<f32x4 *>(workspace),
                           static_cast<float *>(workspace) + n * p.groups * 64 * column_tiles(d) * row_width(d)};
    if (d.factor_dtype == BOLE_DTYPE_F32) return launch_width<float, 1>(a, p, w, n > 0, stream);
    return column_tiles(d) == 2 ? launch_width<__bf16, 2>(a, p, w, n > 0, stream)
                                : launch_width<__bf16, 1>(a, p, w, n > 0, stream);
}

hipError_t launch_linear_step(float *H0, const void *q, const void *k, const void *v,
                              const float *gate, void *out, const bole_linear_dims_t &d,
                              hipStream_t stream) {
    const LinearArgs a = {H0, q, k, v, gate, nullptr, out, nullptr, shape(d)};
    return launch_linear_step_walk(a, d, stream);
}

}  // namespace bole
