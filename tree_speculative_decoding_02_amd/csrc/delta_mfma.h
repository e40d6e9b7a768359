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
// substitution, what lies below them by fp32 matrix products, first within the two 32 x 32
// diagonal blocks, then between them:   X_ij = -X_ii A_ij X_jj   (blocks of either size).
// Products of bf16 k and q are exact but for their fp32 sums; fp32 ones are taken as three bf16
// terms each. Decays and everything after them are fp32.
//
// Kernels are built for d_k = 64 and 128; WHOLE says that the call's d_k is that. Otherwise it is
// smaller, a multiple of 8, and the 8-element parts of a row from d_k on count as zero.
#pragma once

#include "delta_device.h"

namespace bole {

constexpr int kChunk = 64;

struct DeltaTokens {           // LDS of one workgroup, 33 KB
    float A[kChunk * kChunk];  // A, X: element (i, j) at square_at(i, j)
    float X[kChunk * kChunk];  // (before there is an X: bf16 rows of K, share_rows)
    float L[kChunk], Lrest[kChunk];      // cumulative log2-decay (fp64) as two fp32 terms
    float beta[kChunk];                  // strengths
};

struct DeltaTree : DeltaTokens {         // and of a draft tree, 17 KB more
    float P[kChunk * kChunk];
    float start[kChunk];                 // 2^L
    uint64_t mask[kChunk];
    int bad;
};

// A row's sixteen 16-byte pieces are permuted by its number, so that 16 rows' pieces of one
// column lie in distinct banks.
__device__ __forceinline__ int square_at(int i, int j) {
    return i * kChunk + ((((j >> 2) ^ i) & 15) << 2 | (j & 3));
}

// The same for row 16 ai + 4 x + r, column 16 aj + c, spelt out so that what depends on the lane
// is worked out once: x and c from the lane, ai, aj and r not.
__device__ __forceinline__ int block_at(int ai, int aj, int x, int r, int c) {
    return 1024 * ai + 64 * r + (256 * x + ((aj ^ x) << 4)) + ((((c >> 2) ^ r) << 2) | (c & 3));
}

// Row 16 ai + c, columns 16 aj + 4 x .. + 3.
__device__ __forceinline__ int block_row_at(int ai, int aj, int x, int c) {
    return 1024 * ai + 64 * c + ((aj ^ (c >> 2)) << 4) + ((x ^ (c & 3)) << 2);
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

// c += a b with a in NA and b in NB >= NA terms, leaving out the products below b's last term.
template <int NA, int NB>
__device__ __forceinline__ f32x4 mfma_terms(const bf16x8 (&a)[NA], const bf16x8 (&b)[NB], f32x4 c) {
#pragma unroll
    for (int o = NB - 1; o >= 0; --o)  // smallest products first
#pragma unroll
        for (int i = 0; i <= (o < NA ? o : NA - 1); ++i) c = mfma16_bf16(a[i], b[o - i], c);
    return c;
}

// Terms of a factor (K) and of an fp32 quantity beside it (S) that leave the result's rounding,
// to the factors' type, the one that counts.
template <typename TF> struct Terms;
template <> struct Terms<__bf16> { static constexpr int K = 1, S = 2; };
template <> struct Terms<float> { static constexpr int K = 3, S = 3; };

// Eight consecutive elements of a factor's row, as loaded and as terms.
template <typename TF> struct RowPart;
template <> struct RowPart<__bf16> {
    bf16x8 x;
    __device__ __forceinline__ void load(const __bf16 *p) { x = load16(p); }
    __device__ __forceinline__ void clear() { x = (bf16x8)(__bf16)0.f; }
    __device__ __forceinline__ void terms(bf16x8 (&y)[1]) const { y[0] = x; }
};
template <> struct RowPart<float> {
    f32x4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = *reinterpret_cast<const f32x4 *>(p);
        b = *reinterpret_cast<const f32x4 *>(p + 4);
    }
    __device__ __forceinline__ void clear() { a = b = (f32x4)0.f; }
    __device__ __forceinline__ void terms(bf16x8 (&y)[3]) const { split_terms8<3>(a, b, y); }
};

// Part c (of 8 elements) of the row at p; zero from d_k on.
template <bool WHOLE, typename TF>
__device__ __forceinline__ RowPart<TF> row_part(const TF *p, int c, int dk) {
    RowPart<TF> x;
    if (WHOLE) {
        x.load(p + 8 * c);
    } else {
        x.load(p + (8 * c < dk ? 8 * c : 0));
        if (8 * c >= dk) x.clear();
    }
    return x;
}

// Token of row r of row tile m: in order for trees, whose products all meet in LDS; as operands
// of the next product for chunks.
template <bool TREE>
__device__ __forceinline__ int row_of(int m, int r) { return TREE ? 16 * m + r : tile_token(m, r); }

// A wavefront's own rows of k and q (row tile `wave`) as operands; rows past the last repeat it.
// Loaded early, they are in flight while the decays are summed up.
template <typename TF, int DK, bool WHOLE, bool TREE>
struct SystemRows {
    static constexpr bool kShared = sizeof(TF) == 2;
    RowPart<TF> k[DK / 32], q[DK / 32];
    __device__ __forceinline__ void load(const TF *kp, const TF *qp, size_t stride, int dk, int n) {
        const int row = row_of<TREE>(threadIdx.x >> 6, lane_id() & 15), g = lane_id() >> 4;
        const size_t at = (size_t)min(row, n - 1) * stride;
#pragma unroll
        for (int ks = 0; ks < DK / 32; ++ks) {
            k[ks] = row_part<WHOLE>(kp + at, 4 * ks + g, dk);
            q[ks] = row_part<WHOLE>(qp + at, 4 * ks + g, dk);
        }
    }
    // bf16 rows of K, as operands, to all four wavefronts by way of `to`
    __device__ __forceinline__ void share(void *to) const {
        if constexpr (kShared) {
            const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
#pragma unroll
            for (int ks = 0; ks < DK / 32; ++ks) *shared(to, wave, ks) = k[ks].x;
        }
    }
    static __device__ __forceinline__ bf16x8 *shared(void *to, int m, int ks) {
        return static_cast<bf16x8 *>(to) + (m * (DK / 32) + ks) * 64 + lane_id();
    }
};

// c + A B for 16 x 16 blocks of squares in LDS: block (ai, aj) of a, block (bi, bj) of b.
__device__ __forceinline__ f32x4 block_product(const float *a, int ai, int aj, const float *b, int bi,
                                               int bj, f32x4 c) {
    const int col = lane_id() & 15, g = lane_id() >> 4;
    const f32x4 x = *reinterpret_cast<const f32x4 *>(&a[block_row_at(ai, aj, g, col)]);
#pragma unroll
    for (int r = 0; r < 4; ++r)  // k index 4 g + r on both sides
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[r], b[block_at(bi, bj, g, r, col)], c, 0, 0, 0);
    return c;
}

// c - A B with B in registers as products leave it (row 4 g + r, column col).
__device__ __forceinline__ f32x4 block_product_reg(const float *a, int ai, int aj, const f32x4 &b, f32x4 c) {
    const int col = lane_id() & 15, g = lane_id() >> 4;
    const f32x4 x = *reinterpret_cast<const f32x4 *>(&a[block_row_at(ai, aj, g, col)]);
#pragma unroll
    for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[r], -b[r], c, 0, 0, 0);
    return c;
}

__device__ __forceinline__ void put_block(float *a, int ai, int aj, const f32x4 &v) {
    const int col = lane_id() & 15, g = lane_id() >> 4;
#pragma unroll
    for (int r = 0; r < 4; ++r) a[block_at(ai, aj, g, r, col)] = v[r];
}

// The pair products of the n tokens at rows 0 .. n - 1 of k: A into t, P into t (TREE) or, as the
// wavefront's operand pieces, p. t.L, t.beta and (TREE) t.mask are set for all 64 tokens, those
// from n on with their predecessor's decay and no strength, rows.share(t.X) was called, and a
// barrier passed; n >= 1. Four wavefronts. Each holds K_j's rows on the left and its own on the
// right, so that a lane has four neighbours of one row. P's rows from n on belong to no token;
// what lies right of the 32 x 32 diagonal blocks (TREE: of their tiles) is not written.
template <typename TF, int DK, bool WHOLE, bool TREE, typename Tokens>
__device__ __forceinline__ void pair_products(Tokens &t, const SystemRows<TF, DK, WHOLE, TREE> &rows,
                                              const TF *__restrict__ k, size_t stride, int dk, int n,
                                              f32x4 (&p)[4]) {
    const int lane = lane_id(), col = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    constexpr int KS = DK / 32, NK = Terms<TF>::K;
    const int i = row_of<TREE>(wave, col);
    const float li = t.L[i], lr = t.Lrest[i], bi = t.beta[i];
    uint32_t mask[2];
    if constexpr (TREE) {
        mask[0] = (uint32_t)t.mask[i];
        mask[1] = (uint32_t)(t.mask[i] >> 32);
    }
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) {
        p[jt] = (f32x4)0.f;
        if (TREE ? jt > wave : jt >> 1 > wave >> 1) continue;
        f32x4 kk = (f32x4)0.f, qk = (f32x4)0.f;
        const TF *kj = k + (size_t)min(row_of<TREE>(jt, col), n - 1) * stride;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            bf16x8 x[NK], b[NK];
            if constexpr (SystemRows<TF, DK, WHOLE, TREE>::kShared) x[0] = *rows.shared(t.X, jt, ks);
            else row_part<WHOLE>(kj, 4 * ks + g, dk).terms(x);
            rows.k[ks].terms(b);
            kk = mfma_terms(x, b, kk);
            rows.q[ks].terms(b);
            qk = mfma_terms(x, b, qk);
        }
        const int j0 = row_of<TREE>(jt, 4 * g);
        const f32x4 lj = *reinterpret_cast<const f32x4 *>(&t.L[j0]);
        const f32x4 ljr = *reinterpret_cast<const f32x4 *>(&t.Lrest[j0]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float d = __builtin_amdgcn_exp2f((li - lj[r]) + (lr - ljr[r]));
            bool on = j0 + r <= i;
            if constexpr (TREE) on = (mask[jt >> 1] >> (16 * (jt & 1) + 4 * g + r)) & 1u;
            d = on ? d : 0.f;
            qk[r] *= d;
            kk[r] *= bi * d;  // the diagonal is not read
        }
        p[jt] = qk;
        *reinterpret_cast<f32x4 *>(&t.A[square_at(i, j0)]) = kk;
        if constexpr (TREE) *reinterpret_cast<f32x4 *>(&t.P[square_at(i, j0)]) = qk;
    }
    if constexpr (TREE) {  // the part of the 32 x 32 diagonal blocks that is right of the tiles
        if ((wave & 1) == 0) put_block(t.P, wave, wave + 1, (f32x4)0.f);
    }
}

// X from A, both in t, whose A was written before a barrier; n as above. Ends with a barrier.
// X's columns from n on are those of the identity (times no strength); what lies right of the
// 32 x 32 diagonal blocks is not defined.
__device__ __forceinline__ void invert_system(DeltaTokens &t, int n) {
    const int lane = lane_id(), col = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const f32x4 zero = (f32x4)0.f;
    // ---- X: the diagonal blocks, block g and column `col` of it a lane of one wavefront
    if (wave == 0) {
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            f32x4 row[4];
#pragma unroll
            for (int c = 0; c < (i + 3) / 4; ++c)
                row[c] = *reinterpret_cast<const f32x4 *>(
                    &t.A[1024 * g + 64 * i + ((g ^ (i >> 2)) << 4) + ((c ^ (i & 3)) << 2)]);
            float acc[4] = {i == col ? 1.f : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < i; ++j) acc[j & 3] = fmaf(-row[j >> 2][j & 3], x[j], acc[j & 3]);
            x[i] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
            t.X[1024 * g + 64 * i + ((g ^ (i >> 2)) << 4) + ((((col >> 2) ^ (i & 3)) << 2) | (col & 3))] = x[i];
        }
    } else if (wave & 1) {
        put_block(t.X, wave - 1, wave, zero);
    }
    lds_barrier();
    // ---- within the 32 x 32 blocks
    if (wave < 2) {
        const int i = 2 * wave + 1, j = 2 * wave;
        f32x4 y = zero;
        if (16 * i < n) y = block_product_reg(t.X, i, i, block_product(t.A, i, j, t.X, j, j, zero), zero);
        put_block(t.X, i, j, y);
    }
    lds_barrier();
    // ---- between them: T = A X of the first 32 tokens (left in X's unused upper right), then
    // -X T of the last
    const int i = 2 + (wave >> 1), j = wave & 1;
    f32x4 y = zero;
    if (n > 32) {
        f32x4 s = block_product(t.A, i, 1, t.X, 1, j, zero);
        if (j == 0) s = block_product(t.A, i, 0, t.X, 0, 0, s);
        if (i == 2) put_block(t.X, j, 2, s);
        lds_barrier();
        y = block_product_reg(t.X, i, i, s, zero);
        if (i == 3) y = y - block_product(t.X, 3, 2, t.X, j, 2, zero);
    }
    put_block(t.X, i, j, y);
    lds_barrier();
}

// Row `token` of X diag(b) and of a tree's P, columns c .. c + 3 and d .. d + 3.
__device__ __forceinline__ void x_piece(const DeltaTokens &t, int token, int c, int d, f32x4 &a,
                                        f32x4 &b) {
    a = *reinterpret_cast<const f32x4 *>(&t.X[square_at(token, c)]) *
        *reinterpret_cast<const f32x4 *>(&t.beta[c]);
    b = *reinterpret_cast<const f32x4 *>(&t.X[square_at(token, d)]) *
        *reinterpret_cast<const f32x4 *>(&t.beta[d]);
}

__device__ __forceinline__ void p_piece(const DeltaTree &t, int token, int c, int d, f32x4 &a,
                                        f32x4 &b) {
    a = *reinterpret_cast<const f32x4 *>(&t.P[square_at(token, c)]);
    b = *reinterpret_cast<const f32x4 *>(&t.P[square_at(token, d)]);
}

}  // namespace bole
