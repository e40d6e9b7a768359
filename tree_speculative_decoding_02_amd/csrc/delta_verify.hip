// delta_verify.hip - tree verification for the gated delta rule.
//
// With L_i the sum of log2-decays on the root-to-i path, the updates and outputs of a tree
// (nodes in topological order, j above i meaning a strict ancestor) are
//     u_i = b_i (v_i - 2^{L_i} H0^T k_i - sum_{j above i} 2^{L_i - L_j} (k_i . k_j) u_j),
//     o_i = 2^{L_i} H0^T q_i + sum_{j on path(i)} 2^{L_i - L_j} (q_i . k_j) u_j:
// a unit lower triangular system in the updates, the same for every column of the state.
#include <type_traits>

#include "delta_mfma.h"
#include "launch.h"

namespace bole {

// Any width up to 256 and either factor type: one 256-thread workgroup per (sequence, value
// head, 64 state columns). Pair weights in LDS; the H0 terms of all rows in parallel; then one
// wavefront, a column a lane, solves the triangular system row by row. Sums over d_k and over
// ancestors run in fp64 for fp32 factors (their products are exact there), in fp32 for bf16.
template <typename TF>
__global__ __launch_bounds__(256) void delta_verify_generic_kernel(
    const float *__restrict__ H0, const TF *__restrict__ q, const TF *__restrict__ k,
    const TF *__restrict__ v, const float *__restrict__ gate, const float *__restrict__ beta,
    const int32_t *__restrict__ parent, const int32_t *__restrict__ node_offsets,
    TF *__restrict__ out, int32_t *__restrict__ tree_status, const DeltaShape s) {
    typedef typename std::conditional<std::is_same<TF, float>::value, double, float>::type A;
    __shared__ uint64_t s_mask[kMaxTree];
    __shared__ double s_L[kMaxTree];
    __shared__ float s_beta[kMaxTree];
    __shared__ float s_A[kMaxTree][kMaxTree + 1], s_P[kMaxTree][kMaxTree + 1];
    __shared__ float s_u[kMaxTree][64];
    __shared__ int s_bad;
    const int unit = blockIdx.x, c0 = blockIdx.y * 64, tid = threadIdx.x;
    const int b = unit / s.H, h = unit - b * s.H, hk = h / (s.H / s.HK);
    const bool first = h == 0 && c0 == 0 && tid == 0 && tree_status;
    const TreeRange tr = tree_range(node_offsets, b, s.T);
    if (tr.status != BOLE_TREE_OK) {
        if (first) tree_status[b] = tr.status;
        return;
    }
    const int lo = tr.lo, n = tr.n, cols = min(64, s.DV - c0);
    if (tid < 64) {
        const bool in = tid < n;
        const float lg = in ? log2_decay(gate[(size_t)(lo + tid) * s.H + h]) : 0.f;
        const WaveTopoD t = wave_topology_cumlog_f64(in ? parent[lo + tid] : -1, lg, n);
        s_mask[tid] = t.mask;
        s_L[tid] = t.L;
        s_beta[tid] = in ? beta[(size_t)(lo + tid) * s.H + h] : 0.f;
        if (tid == 0) s_bad = t.bad;
    }
    __syncthreads();
    if (first) tree_status[b] = s_bad;
    const size_t sk = (size_t)s.HK * s.DK, sv = (size_t)s.H * s.DV;
    const TF *kb = k + (size_t)lo * sk + (size_t)hk * s.DK, *qb = q + (size_t)lo * sk + (size_t)hk * s.DK;
    const size_t v0 = (size_t)lo * sv + (size_t)h * s.DV + c0;
    if (s_bad) {
        for (int e = tid; e < n * cols; e += 256)
            out[v0 + (size_t)(e / cols) * sv + e % cols] = (TF)__builtin_nanf("");
        return;
    }
    for (int e = tid; e < n * n; e += 256) {
        const int i = e / n, j = e - i * n;
        float wa = 0.f, wp = 0.f;
        if ((s_mask[i] >> j) & 1ull) {
            A kk = 0, qk = 0;
            for (int r = 0; r < s.DK; ++r) {
                const A x = (A)to_f32(kb[j * sk + r]);
                kk += x * (A)to_f32(kb[i * sk + r]);
                qk += x * (A)to_f32(qb[i * sk + r]);
            }
            const float d = exp2f((float)(s_L[i] - s_L[j]));
            wp = d * (float)qk;
            wa = i == j ? 0.f : s_beta[i] * d * (float)kk;
        }
        s_A[i][j] = wa;
        s_P[i][j] = wp;
    }
    const float *Hu = H0 + (size_t)unit * s.DK * s.DV + c0;
    for (int e = tid; e < n * cols; e += 256) {
        const int i = e / cols, c = e - i * cols;
        A acc = 0;
        for (int r = 0; r < s.DK; ++r) acc += (A)Hu[(size_t)r * s.DV + c] * (A)to_f32(kb[i * sk + r]);
        s_u[i][c] = s_beta[i] * (to_f32(v[v0 + (size_t)i * sv + c]) - exp2f((float)s_L[i]) * (float)acc);
    }
    __syncthreads();
    if (tid < cols) {
        for (int i = 1; i < n; ++i) {
            A acc = (A)s_u[i][tid];
            for (int j = 0; j < i; ++j) acc -= (A)s_A[i][j] * (A)s_u[j][tid];
            s_u[i][tid] = (float)acc;
        }
    }
    __syncthreads();
    for (int e = tid; e < n * cols; e += 256) {
        const int i = e / cols, c = e - i * cols;
        A acc = 0;
        for (int r = 0; r < s.DK; ++r) acc += (A)Hu[(size_t)r * s.DV + c] * (A)to_f32(qb[i * sk + r]);
        acc *= (A)exp2f((float)s_L[i]);
        for (int j = 0; j <= i; ++j) acc += (A)s_P[i][j] * (A)s_u[j][c];
        out[v0 + (size_t)i * sv + c] = (TF)(float)acc;
    }
}

// d_k up to 128 (a multiple of 8), any d_v: one workgroup of four wavefronts per (sequence, value
// head, 64 NT columns). The loads of its state columns are in flight while it forms the tree's
// system (delta_mfma.h); then every wavefront carries its 16 NT columns through
//     R = V - diag(2^L) K H0,   U = X diag(b) R,   O = diag(2^L) Q H0 + P U
// in registers, each product's results being the next one's operand. H0, X, R, P and U are
// taken as two bf16 terms (2^-17 left) for bf16 factors, as three for fp32 ones, so that the
// output's own rounding is the one that counts. Row slots past the last node repeat it: their
// columns of X diag(b) are zero.
//
// Row tile m is nodes 16 m .. 16 m + 15; as a right operand, tiles 2s and 2s + 1 hold in lane
// group g nodes 32 s + 4 g .. + 3 and 32 s + 16 + 4 g .. + 3, and X and P are read to match. The
// wavefronts' own rows of a bf16 K serve all four through LDS, over A, which the system no longer
// needs; Q is read again from the caches. (64 trees of 64 nodes, 32 heads, 128 x 128: 83 us with
// both from the caches, 74 this way; Q through 16 KB more of LDS leaves two workgroups a CU instead
// of three and took 57.4 instead of 54.7 us for trees of up to 64 nodes.)
//
// Measured: 64 trees of up to 64 nodes 48 us (3.5 TB/s: the states' bytes and about as much time
// again for the systems, whose steps wait for each other), 8 trees of 32 nodes and 32 x 128 x 64
// states 10 us (one chain of loads, system and products); fp32, 64 trees of 64 nodes 126 us.
//
// NT = 2 (d_v a multiple of 32): lane c of 16 holds columns 2c and 2c + 1, and a state row's 32
// columns are one 128-byte read.
template <typename TF, int DK, int NT, bool WHOLE>
__global__ __launch_bounds__(256, sizeof(TF) == 2 ? 3 : 2) void delta_verify_kernel(
    const float *__restrict__ H0, const TF *__restrict__ q, const TF *__restrict__ k,
    const TF *__restrict__ v, const float *__restrict__ gate, const float *__restrict__ beta,
    const int32_t *__restrict__ parent, const int32_t *__restrict__ node_offsets,
    TF *__restrict__ out, int32_t *__restrict__ tree_status, const DeltaShape s) {
    typedef float hvec __attribute__((ext_vector_type(NT)));
    typedef TF vvec __attribute__((ext_vector_type(NT)));
    constexpr int KS = DK / 32, NK = Terms<TF>::K, NS = Terms<TF>::S;
    __shared__ DeltaTree t;
    constexpr bool SHARE = SystemRows<TF, DK, WHOLE, true>::kShared;
    static_assert(4 * KS * 512 * 2 <= sizeof(t.A), "K over A");
    const int unit = blockIdx.x, tid = threadIdx.x, lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, g = lane >> 4, dk = WHOLE ? DK : s.DK;
    const int b = unit / s.H, h = unit - b * s.H, hk = h / (s.H / s.HK);
    const bool first = h == 0 && blockIdx.y == 0 && tid == 0 && tree_status;
    const TreeRange tr = tree_range(node_offsets, b, s.T);
    if (tr.status != BOLE_TREE_OK) {
        if (first) tree_status[b] = tr.status;
        return;
    }
    const int lo = tr.lo, n = tr.n;
    const size_t sk = (size_t)s.HK * dk, sv = (size_t)s.H * s.DV;
    const TF *kb = k + (size_t)lo * sk + (size_t)hk * dk, *qb = q + (size_t)lo * sk + (size_t)hk * dk;
    const int c0 = (blockIdx.y * 4 + wave) * 16 * NT;     // the wavefront's columns, then the lane's
    const bool live = c0 < s.DV && n > 0;
    const bool mine = NT == 2 || c0 + col < s.DV;         // lanes past the last column repeat it
    const int c1 = NT == 2 ? c0 + 2 * col : min(c0 + col, s.DV - 1);
    const float *Hu = H0 + (size_t)unit * dk * s.DV + c1;
    hvec hr[KS][8];
    if (live) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int row = 32 * ks + 8 * g + e;
                hr[ks][e] = __builtin_nontemporal_load(
                    reinterpret_cast<const hvec *>(Hu + (size_t)(WHOLE || row < dk ? row : 0) * s.DV));
            }
    }
    SystemRows<TF, DK, WHOLE, true> rows;
    if (n > 0) rows.load(kb, qb, sk, dk, n);
    if (tid < 64) {
        const bool in = tid < n;
        const float lg = in ? log2_decay(gate[(size_t)(lo + tid) * s.H + h]) : 0.f;
        const WaveTopoD w = wave_topology_cumlog_f64(in ? parent[lo + tid] : -1, lg, n);
        t.mask[tid] = w.mask;
        t.L[tid] = (float)w.L;
        t.Lrest[tid] = (float)(w.L - (double)(float)w.L);
        t.start[tid] = __builtin_amdgcn_exp2f((float)w.L);
        t.beta[tid] = in ? beta[(size_t)(lo + tid) * s.H + h] : 0.f;
        if (tid == 0) t.bad = w.bad;
    }
    if (n > 0) rows.share(t.X);
    lds_barrier();
    if (first) tree_status[b] = t.bad;
    const size_t v0 = (size_t)lo * sv + (size_t)h * s.DV;
    if (t.bad) {
        for (int e = tid; e < n * s.DV; e += 256)
            out[v0 + (size_t)(e / s.DV) * sv + e % s.DV] = (TF)__builtin_nanf("");
        return;
    }
    if (n == 0) return;
    f32x4 pair[4];
    pair_products(t, rows, kb, sk, dk, n, pair);
    lds_barrier();
    invert_system(t, n);
    if constexpr (SHARE) {
        rows.share(t.A);
        lds_barrier();
    }
    // row tile m has nodes of the tree
    auto used = [&](int m) { return 16 * m < n; };
    if (!live) return;
    const size_t vc = v0 + c1;
    f32x4 r[4][NT], o[4][NT];
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int c = 0; c < NT; ++c) r[m][c] = o[m][c] = (f32x4)0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        bf16x8 hb[NT][NS];
#pragma unroll
        for (int c = 0; c < NT; ++c) {
            f32x4 x, y;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[e] = hr[ks][e][c];
                y[e] = hr[ks][4 + e][c];
            }
            if (!WHOLE && 32 * ks + 8 * g >= dk) x = y = (f32x4)0.f;
            split_terms8<NS>(x, y, hb[c]);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            if (!used(m)) continue;
            const size_t row = (size_t)min(16 * m + col, n - 1) * sk;
            bf16x8 ka[NK], qa[NK];
            if constexpr (SHARE) {
                ka[0] = *rows.shared(t.A, m, ks);
            } else {
                row_part<WHOLE>(kb + row, 4 * ks + g, dk).terms(ka);
            }
            row_part<WHOLE>(qb + row, 4 * ks + g, dk).terms(qa);
#pragma unroll
            for (int c = 0; c < NT; ++c) {
                r[m][c] = mfma_terms(ka, hb[c], r[m][c]);
                o[m][c] = mfma_terms(qa, hb[c], o[m][c]);
            }
        }
        __builtin_amdgcn_sched_barrier(0);  // rows of one step at a time in registers
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        if (!used(m)) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = 16 * m + 4 * g + e;
            const float d = t.start[i];
            const vvec vv = *reinterpret_cast<const vvec *>(v + vc + (size_t)min(i, n - 1) * sv);
#pragma unroll
            for (int c = 0; c < NT; ++c) {
                r[m][c][e] = (float)vv[c] - d * r[m][c][e];
                o[m][c][e] *= d;
            }
        }
    }
    // U from R, then O, 32 tokens (two row tiles) of the right operand at a time
#pragma unroll
    for (int step = 0; step < 2; ++step) {
        bf16x8 rb[2][NT][NS];
#pragma unroll
        for (int sb = 0; sb < 2; ++sb)
#pragma unroll
            for (int c = 0; c < NT; ++c) split_terms8<NS>(r[2 * sb][c], r[2 * sb + 1][c], rb[sb][c]);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            if (!used(m)) continue;
#pragma unroll
            for (int c = 0; c < NT; ++c)
                if (step == 0) r[m][c] = (f32x4)0.f;
#pragma unroll
            for (int sb = 0; sb <= (m >> 1); ++sb) {
                f32x4 x, y;
                bf16x8 a[NS];
                const int c = 32 * sb + 4 * g;
                if (step == 0) x_piece(t, 16 * m + col, c, c + 16, x, y);
                else p_piece(t, 16 * m + col, c, c + 16, x, y);
                split_terms8<NS>(x, y, a);
#pragma unroll
                for (int c = 0; c < NT; ++c) {
                    if (step == 0) r[m][c] = mfma_terms(a, rb[sb][c], r[m][c]);
                    else o[m][c] = mfma_terms(a, rb[sb][c], o[m][c]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = 16 * m + 4 * g + e;
            vvec y;
#pragma unroll
            for (int c = 0; c < NT; ++c) y[c] = (TF)o[m][c][e];
            if (i < n && mine) *reinterpret_cast<vvec *>(out + vc + (size_t)i * sv) = y;
        }
}

static bool verify_covers(const bole_delta_dims_t &d, const void *q, const void *k) {
    return !(d.flags & BOLE_FLAG_FORCE_GENERIC) && d.d_k <= 128 && d.d_k % 8 == 0 &&
           (reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k)) % 16 == 0;
}

template <typename TF, int DK, bool WHOLE>
static hipError_t launch_mfma(const float *H0, const void *q, const void *k, const void *v,
                              const float *gate, const float *beta, const int32_t *parent,
                              const int32_t *node_offsets, void *out, const bole_delta_dims_t &d,
                              int32_t *tree_status, hipStream_t stream) {
    const DeltaShape s = {d.batch, d.heads, d.key_heads, d.d_k, d.d_v, d.total_tokens};
    const unsigned units = (unsigned)d.batch * (unsigned)d.heads;
    const dim3 block(256);
    const TF *qb = static_cast<const TF *>(q), *kb = static_cast<const TF *>(k), *vb = static_cast<const TF *>(v);
    TF *ob = static_cast<TF *>(out);
    // 32 columns a wavefront (in pairs, so on even addresses) where that still gives each of the
    // four some
    const uintptr_t pairs = reinterpret_cast<uintptr_t>(H0) % 8 |
                            (reinterpret_cast<uintptr_t>(v) | reinterpret_cast<uintptr_t>(out)) % (2 * sizeof(TF));
    if (d.d_v % 32 == 0 && d.d_v > 64 && pairs == 0)
        delta_verify_kernel<TF, DK, 2, WHOLE><<<dim3(units, (d.d_v + 127) / 128), block, 0, stream>>>(
            H0, qb, kb, vb, gate, beta, parent, node_offsets, ob, tree_status, s);
    else
        delta_verify_kernel<TF, DK, 1, WHOLE><<<dim3(units, (d.d_v + 63) / 64), block, 0, stream>>>(
            H0, qb, kb, vb, gate, beta, parent, node_offsets, ob, tree_status, s);
    return hipGetLastError();
}

template <typename TF>
static hipError_t launch_mfma_width(const float *H0, const void *q, const void *k, const void *v,
                                    const float *gate, const float *beta, const int32_t *parent,
                                    const int32_t *node_offsets, void *out, const bole_delta_dims_t &d,
                                    int32_t *tree_status, hipStream_t stream) {
    auto go = [&](auto launch) {
        return launch(H0, q, k, v, gate, beta, parent, node_offsets, out, d, tree_status, stream);
    };
    if (d.d_k <= 64) return d.d_k == 64 ? go(launch_mfma<TF, 64, true>) : go(launch_mfma<TF, 64, false>);
    return d.d_k == 128 ? go(launch_mfma<TF, 128, true>) : go(launch_mfma<TF, 128, false>);
}

template <typename TF>
static hipError_t launch_generic(const float *H0, const void *q, const void *k, const void *v,
                                 const float *gate, const float *beta, const int32_t *parent,
                                 const int32_t *node_offsets, void *out,
                                 const bole_delta_dims_t &d, int32_t *tree_status,
                                 hipStream_t stream) {
    const DeltaShape s = {d.batch, d.heads, d.key_heads, d.d_k, d.d_v, d.total_tokens};
    const dim3 grid((unsigned)d.batch * (unsigned)d.heads, (unsigned)((d.d_v + 63) / 64));
    delta_verify_generic_kernel<TF><<<grid, dim3(256), 0, stream>>>(
        H0, static_cast<const TF *>(q), static_cast<const TF *>(k), static_cast<const TF *>(v), gate,
        beta, parent, node_offsets, static_cast<TF *>(out), tree_status, s);
    return hipGetLastError();
}

hipError_t launch_delta_verify(const float *H0, const void *q, const void *k, const void *v,
                               const float *gate, const float *beta, const int32_t *parent,
                               const int32_t *node_offsets, void *out, const bole_delta_dims_t &d,
                               int32_t *tree_status, hipStream_t stream) {
    if (verify_covers(d, q, k))
        return d.factor_dtype == BOLE_DTYPE_F32
                   ? launch_mfma_width<float>(H0, q, k, v, gate, beta, parent, node_offsets, out, d,
                                              tree_status, stream)
                   : launch_mfma_width<__bf16>(H0, q, k, v, gate, beta, parent, node_offsets, out, d,
                                               tree_status, stream);
    return d.factor_dtype == BOLE_DTYPE_F32
               ? launch_generic<float>(H0, q, k, v, gate, beta, parent, node_offsets, out, d,
                                       tree_status, stream)
               : launch_generic<__bf16>(H0, q, k, v, gate, beta, parent, node_offsets, out, d,
                                        tree_status, stream);
}

}  // namespace bole
