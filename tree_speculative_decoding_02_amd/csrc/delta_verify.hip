// delta_verify.hip - tree verification for the gated delta rule.
//
// With L_i the sum of log2-decays on the root-to-i path, the updates and outputs of a tree
// (nodes in topological order, j above i meaning a strict ancestor) are
//     u_i = b_i (v_i - 2^{L_i} H0^T k_i - sum_{j above i} 2^{L_i - L_j} (k_i . k_j) u_j),
//     o_i = 2^{L_i} H0^T q_i + sum_{j on path(i)} 2^{L_i - L_j} (q_i . k_j) u_j:
// a unit lower triangular system in the updates, the same for every column of the state.
#include <type_traits>

#include "delta_device.h"
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
    return d.factor_dtype == BOLE_DTYPE_F32
               ? launch_generic<float>(H0, q, k, v, gate, beta, parent, node_offsets, out, d,
                                       tree_status, stream)
               : launch_generic<__bf16>(H0, q, k, v, gate, beta, parent, node_offsets, out, d,
                                        tree_status, stream);
}

}  // namespace bole
