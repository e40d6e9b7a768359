// delta_mfma.h - the triangular system of up to 64 tokens (a chunk of a prompt, or a draft
// tree) on the matrix cores, shared by the gated delta rule's chunked prefill and its tree
// verification.
//
// With L_i the cumulative log2-decay on token i's path and j above i a strict ancestor (in a
// chunk: an earlier token),
//     A_ij = b_i 2^{L_i - L_j} (k_i . k_j)   for j above i, else 0,
//     P_ij = 2^{L_i - L_j} (q_i . k_j)       for j on the path of i, else 0,
//     U = X diag(b) (V - diag(2^L) K H0),   X = (I + A)^-1,   O = diag(2^L) Q H0 + P U.
// X is formed once and serves every state column: the four 16 x 16 diagonal blocks by forward
// substitution, the blocks below them by fp32 matrix products
//     X_ij = -X_ii sum_{k=j}^{i-1} A_ik X_kj.
// Products of k and q are bf16 products with fp32 sums, exact but for those sums; decays and
// everything after them are fp32.
#pragma once

#include "delta_device.h"

namespace bole {

constexpr int kChunk = 64;

struct DeltaTokens {           // LDS of one workgroup, 50 KB
    float A[kChunk * kChunk];  // A, X, P: element (i, j) at square_at(i, j)
    float X[kChunk * kChunk];
    float P[kChunk * kChunk];
    double L[kChunk];
    float beta[kChunk], start[kChunk];   // strengths, 2^L
    uint64_t mask[kChunk];
    int bad;
};

// A row's sixteen 16-byte pieces are permuted by its number, so that 16 rows' pieces of one
// column lie in distinct banks.
__device__ __forceinline__ int square_at(int i, int j) {
    return i * kChunk + ((((j >> 2) ^ i) & 15) << 2 | (j & 3));
}

// Token that lane index r (0..15) of row tile m stands for. Tiles 2s and 2s + 1 cover tokens
// 32 s .. 32 s + 31 so that a product's results in registers (rows 4g .. 4g + 3 of lane group
// g, both tiles) are tokens 32 s + 8 g .. + 7: the B operand of the next product.
__device__ __forceinline__ int tile_token(int m, int r) {
    return 32 * (m >> 1) + 8 * (r >> 2) + 4 * (m & 1) + (r & 3);
}

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// fp32 x as bf16 terms of falling size: two leave 2^-17 of it, three 2^-25. In pairs, for the
// packed conversion.
template <int N>
__device__ __forceinline__ void split_terms2(f32x2 x, bf16x2 (&y)[N]) {
#pragma unroll
    for (int t = 0; t < N; ++t) {
        y[t] = __builtin_convertvector(x, bf16x2);
        if (t + 1 < N) x -= __builtin_convertvector(y[t], f32x2);
    }
}

template <int N>
__device__ __forceinline__ void split_terms8(const f32x4 &a, const f32x4 &b, bf16x8 (&y)[N]) {
    bf16x2 p[4][N];
    split_terms2<N>(__builtin_shufflevector(a, a, 0, 1), p[0]);
    split_terms2<N>(__builtin_shufflevector(a, a, 2, 3), p[1]);
    split_terms2<N>(__builtin_shufflevector(b, b, 0, 1), p[2]);
    split_terms2<N>(__builtin_shufflevector(b, b, 2, 3), p[3]);
#pragma unroll
    for (int i = 0; i < N; ++i)
        y[i] = __builtin_shufflevector(__builtin_shufflevector(p[0][i], p[1][i], 0, 1, 2, 3),
                                       __builtin_shufflevector(p[2][i], p[3][i], 0, 1, 2, 3), 0, 1, 2,
                                       3, 4, 5, 6, 7);
}

// c += a b with a and b in N terms each, leaving out the products below the last term.
template <int N>
__device__ __forceinline__ f32x4 mfma_terms(const bf16x8 (&a)[N], const bf16x8 (&b)[N], f32x4 c) {
#pragma unroll
    for (int o = N - 1; o >= 0; --o)  // smallest products first
#pragma unroll
        for (int i = 0; i <= o; ++i) c = mfma16_bf16(a[i], b[o - i], c);
    return c;
}

// Fills t (A, P, X) for the n tokens at rows 0 .. n - 1 of k and q; t.L, t.beta and t.mask are
// set and a barrier passed; n >= 1. Four wavefronts; ends with a barrier. From n on, rows and columns
// are those of the identity (X) and zero (A, P).
template <int DK>
__device__ __forceinline__ void delta_system(DeltaTokens &t, const __bf16 *__restrict__ k,
                                             const __bf16 *__restrict__ q, size_t stride, int n) {
    const int lane = lane_id(), wave = threadIdx.x >> 6, col = lane & 15, g = lane >> 4;
    constexpr int KS = DK / 32;
    // ---- pair products: row tile `wave` (tokens 16 wave ..), column tiles up to it
    auto piece = [&](const __bf16 *p, int row, int ks) {  // rows past the last repeat it
        return load16(p + (size_t)min(row, n - 1) * stride + 32 * ks + 8 * g);
    };
    bf16x8 ka[KS], qa[KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        ka[ks] = piece(k, 16 * wave + col, ks);
        qa[ks] = piece(q, 16 * wave + col, ks);
    }
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) {
        f32x4 kk = (f32x4)0.f, qk = (f32x4)0.f;
        if (jt <= wave && 16 * wave < n) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const bf16x8 b = jt == wave ? ka[ks] : piece(k, 16 * jt + col, ks);
                kk = mfma16_bf16(ka[ks], b, kk);
                qk = mfma16_bf16(qa[ks], b, qk);
            }
        }
        const int j = 16 * jt + col;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 16 * wave + 4 * g + r;
            float av = 0.f, pv = 0.f;
            if (j <= i && i < n && ((t.mask[i] >> j) & 1ull)) {
                const float d = __builtin_amdgcn_exp2f((float)(t.L[i] - t.L[j]));
                pv = d * qk[r];
                if (j < i) av = t.beta[i] * d * kk[r];
            }
            t.A[square_at(i, j)] = av;
            t.P[square_at(i, j)] = pv;
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    // ---- X: diagonal block `wave`, column `col` (every lane group computes the same), from
    // what this wavefront itself wrote
    {
        const int base = 16 * wave;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            f32x4 row[4];
#pragma unroll
            for (int c = 0; c < (i + 3) / 4; ++c)
                row[c] = *reinterpret_cast<const f32x4 *>(&t.A[square_at(base + i, base + 4 * c)]);
            float acc[2] = {i == col ? 1.f : 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < i; ++j) acc[j & 1] = fmaf(-row[j >> 2][j & 3], x[j], acc[j & 1]);
            x[i] = acc[0] + acc[1];
            if (i % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // a few rows of A in registers
        }
        // lane group g writes rows 4 g ..; the blocks right of the diagonal are zero
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if ((i >> 2) == g) t.X[square_at(base + i, base + col)] = x[i];
        for (int jt = wave + 1; jt < 4; ++jt)
#pragma unroll
            for (int r = 0; r < 4; ++r) t.X[square_at(base + 4 * g + r, 16 * jt + col)] = 0.f;
    }
    lds_barrier();
    // ---- column `wave` of the blocks below the diagonal, downwards: each needs the diagonal
    // blocks (above) and the blocks over it, which this wavefront wrote
    const int j = wave;
    for (int i = j + 1; i < 4; ++i) {
        f32x4 y = (f32x4)0.f;
        if (16 * i < n) {
            f32x4 s = (f32x4)0.f;
            for (int b = j; b < i; ++b)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    s = __builtin_amdgcn_mfma_f32_16x16x4f32(
                        t.A[square_at(16 * i + col, 16 * b + 4 * r + g)],
                        t.X[square_at(16 * b + 4 * r + g, 16 * j + col)], s, 0, 0, 0);
#pragma unroll
            for (int r = 0; r < 4; ++r)  // k index 4 g + r on both sides
                y = __builtin_amdgcn_mfma_f32_16x16x4f32(
                    t.X[square_at(16 * i + col, 16 * i + 4 * g + r)], -s[r], y, 0, 0, 0);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) t.X[square_at(16 * i + 4 * g + r, 16 * j + col)] = y[r];
    }
    lds_barrier();
}

// Row `token`, columns 32 s + 8 g .. + 7 of X diag(b).
__device__ __forceinline__ void x_piece(const DeltaTokens &t, int token, int s, int g, f32x4 &a,
                                        f32x4 &b) {
    const int c0 = 32 * s + 8 * g;
    a = *reinterpret_cast<const f32x4 *>(&t.X[square_at(token, c0)]) *
        *reinterpret_cast<const f32x4 *>(&t.beta[c0]);
    b = *reinterpret_cast<const f32x4 *>(&t.X[square_at(token, c0 + 4)]) *
        *reinterpret_cast<const f32x4 *>(&t.beta[c0 + 4]);
}

__device__ __forceinline__ void p_piece(const DeltaTokens &t, int token, int s, int g, f32x4 &a,
                                        f32x4 &b) {
    const int c0 = 32 * s + 8 * g;
    a = *reinterpret_cast<const f32x4 *>(&t.P[square_at(token, c0)]);
    b = *reinterpret_cast<const f32x4 *>(&t.P[square_at(token, c0 + 4)]);
}

}  // namespace bole
