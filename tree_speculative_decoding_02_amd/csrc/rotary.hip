// rotary.hip - norm of every head's query and key and its rotation by position, in one pass:
//     y = x / sqrt(mean(x^2) + eps) * weight,
//     (y_a, y_b) <- (y_a cos t - y_b sin t, y_b cos t + y_a sin t),   t = position * inv_freq[j].
//
// A row's angles are the same for all of its heads: they are taken once, in fp64, reduced to one
// turn, and their sines and cosines kept in LDS (an fp32 angle at position 2^20 is off by 2^-5).
// Bound by the rows' way through HBM: 2 bytes read and 2 written an element in bf16.
#include <cmath>

#include "delta_device.h"
#include "launch.h"

namespace bole {

struct RotaryArgs {
    const void *q, *k, *q_weight, *k_weight;
    const float *inv_freq;
    const int32_t *first_position, *parent, *offsets;
    void *q_out, *k_out;
    int32_t *status;
    int B, H, HK, D, R, T;           // R: rotated dimensions
    int64_t q_stride, k_stride;
    float eps;
};

constexpr int kMaxPairs = 128;

// Position of a row: kNoRow for one that is nobody's or must be left, kNanRowAt for one that
// becomes NaN. One wavefront; reports its sequence's status where it is the first row.
constexpr int kNoRow = -1, kNanRowAt = -2;

__device__ __forceinline__ int row_position(const RotaryArgs &a, int row) {
    const RowOwner o = owner_of(a.offsets, a.B, a.T, row);
    const int lane = lane_id();
    if (row == 0 && a.status)  // sequences without rows, and all of them if offsets are unordered
        for (int b = lane; b < a.B; b += 64)
            if (!o.ordered || a.offsets[b + 1] == a.offsets[b])
                a.status[b] = o.ordered ? BOLE_TREE_OK : BOLE_TREE_BAD_SIZE;
    if (!o.found) return kNoRow;
    int st = BOLE_TREE_OK, at = row - o.lo;
    if (a.parent) {
        if (o.n > kMaxTree) {
            st = BOLE_TREE_BAD_SIZE;
        } else {
            const WaveTopo t = wave_topology(a.parent + o.lo, o.n);
            st = t.bad;
            at = __shfl(t.depth, at, 64) - 1;
        }
    }
    const int first = a.first_position[o.b];
    if (st == BOLE_TREE_OK && (first < 0 || (int64_t)first + o.n - 1 > 0x7fffffffLL)) st = BOLE_TREE_BAD_CACHE;
    if (row == o.lo && lane == 0 && a.status) a.status[o.b] = st;
    if (st != BOLE_TREE_OK) return st == BOLE_TREE_BAD_SIZE ? kNoRow : kNanRowAt;
    return first + at;
}

__device__ __forceinline__ float2 turn_of(int position, float inv_freq) {
    double t = (double)position * (double)inv_freq * 0.15915494309189533577;  // in turns
    t -= rint(t);
    float2 y;  // cos, sin
    sincospif((float)(2.0 * t), &y.y, &y.x);
    return y;
}

// Any width and alignment: a workgroup a row, a wavefront a head at a time.
template <typename T>
__global__ __launch_bounds__(256) void rotary_generic_kernel(const RotaryArgs a, bool interleaved) {
    __shared__ float2 s_turn[kMaxPairs];
    __shared__ float s_y[4][256];
    const int row = blockIdx.x, tid = threadIdx.x, lane = lane_id(), wave = tid >> 6, P = a.R / 2;
    const int pos = row_position(a, row);
    if (pos == kNoRow) return;
    if (pos >= 0 && tid < P) s_turn[tid] = turn_of(pos, a.inv_freq[tid]);
    __syncthreads();
    for (int h = wave; h < a.H + a.HK; h += 4) {
        const bool key = h >= a.H;
        const int hh = key ? h - a.H : h;
        const T *x = static_cast<const T *>(key ? a.k : a.q) + (size_t)row * (key ? a.k_stride : a.q_stride) + (size_t)hh * a.D;
        T *y = static_cast<T *>(key ? a.k_out : a.q_out) + ((size_t)row * (key ? a.HK : a.H) + hh) * a.D;
        const T *w = static_cast<const T *>(key ? a.k_weight : a.q_weight);
        float v[4], sum = 0.f;
        for (int j = 0; j < 4; ++j) {
            v[j] = lane + 64 * j < a.D ? to_f32(x[lane + 64 * j]) : 0.f;
            sum = fmaf(v[j], v[j], sum);
        }
        float scale = 1.f;
        if (w) {
            for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d, 64);
            scale = 1.f / sqrtf(sum / a.D + a.eps);
        }
        for (int j = 0; j < 4; ++j)
            if (lane + 64 * j < a.D) {
                v[j] = w ? v[j] * scale * to_f32(w[lane + 64 * j]) : v[j];
                s_y[wave][lane + 64 * j] = v[j];
            }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        for (int j = 0; j < 4; ++j) {
            const int e = lane + 64 * j;
            if (e >= a.D) break;
            float r = v[j];
            if (pos >= 0 && e < a.R) {
                const int p = interleaved ? e >> 1 : e % P;
                const bool second = interleaved ? e & 1 : e >= P;
                const float other = s_y[wave][interleaved ? e ^ 1 : second ? e - P : e + P];
                const float2 t = s_turn[p];
                r = second ? fmaf(other, t.y, v[j] * t.x) : fmaf(-other, t.y, v[j] * t.x);
            }
            y[e] = pos >= 0 ? (T)r : (T)__builtin_nanf("");
        }
        asm volatile("" ::: "memory");
    }
}

// Heads whose lanes hold 8 consecutive elements each: LP lanes a head (8 LP >= d), 256 / LP heads at
// a time, of ROWS neighbouring rows. The other half of a pair (j, j + half) is another lane's.
//
// With ROWS 1 the heads are dealt to gridDim.y workgroups, so that a row is one pass: for few rows,
// where the chain of loads behind a row's position is what takes time.
template <typename T> struct Eight;  // 8 elements as loaded
template <> struct Eight<__bf16> {
    uint4 x;
    __device__ __forceinline__ void load(const __bf16 *p) { x = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ float get(int i) const {
        const uint32_t w = (&x.x)[i >> 1];
        return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
    }
    __device__ __forceinline__ Eight from(int lane) const {
        Eight y;
#pragma unroll
        for (int i = 0; i < 4; ++i) (&y.x.x)[i] = (uint32_t)__shfl((int)(&x.x)[i], lane, 64);
        return y;
    }
    static __device__ __forceinline__ void store(__bf16 *p, const float (&y)[8]) {
        bf16x8 z;
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = (__bf16)y[i];
        *reinterpret_cast<bf16x8 *>(p) = z;
    }
};
template <> struct Eight<float> {
    f32x4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = *reinterpret_cast<const f32x4 *>(p);
        b = *reinterpret_cast<const f32x4 *>(p + 4);
    }
    __device__ __forceinline__ float get(int i) const { return i < 4 ? a[i] : b[i - 4]; }
    __device__ __forceinline__ Eight from(int lane) const {
        Eight y;
#pragma unroll
        for (int i = 0; i < 4; ++i) y.a[i] = __shfl(a[i], lane, 64), y.b[i] = __shfl(b[i], lane, 64);
        return y;
    }
    static __device__ __forceinline__ void store(float *p, const float (&y)[8]) {
        *reinterpret_cast<f32x4 *>(p) = f32x4{y[0], y[1], y[2], y[3]};
        *reinterpret_cast<f32x4 *>(p + 4) = f32x4{y[4], y[5], y[6], y[7]};
    }
};

template <int CTRL>
__device__ __forceinline__ float add_dpp(float x) {
    return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, false));
}

// Sum over LP neighbouring lanes, in all of them.
template <int LP>
__device__ __forceinline__ float sum_lanes(float x) {
    x = add_dpp<0xB1>(x);   // lanes 1, 2, then the mirrored half row and row
    x = add_dpp<0x4E>(x);
    x = add_dpp<0x141>(x);
    if constexpr (LP >= 16) x = add_dpp<0x140>(x);
    if constexpr (LP >= 32) x = sum16(x);
    return x;
}

template <typename T, int LP, bool INTER, int ROWS>
__global__ __launch_bounds__(256) void rotary_kernel(const RotaryArgs a) {
    __shared__ __align__(16) float s_cos[ROWS][kMaxPairs], s_sin[ROWS][kMaxPairs];
    __shared__ int s_pos[ROWS];
    const int tid = threadIdx.x, wave = tid >> 6, row0 = blockIdx.x * ROWS, P = a.R / 2;
    const int heads = a.H + a.HK, rows = min(ROWS, a.T - row0), items = rows * heads;
    const int c = tid % LP, part = 8 * c;               // the lane's elements of its head
    const bool in = part < a.D, turned = part < a.R;
    const int half = P / 8;                             // pairs (j, j + half): the other's lane
    const bool second = c >= half;
    const int other = (tid & 63) + (second ? -half : half);
    struct Item {
        int r, h;
        bool key, live;
        Eight<T> x;
    };
    auto fetch = [&](int first) {
        Item t;
        const int i = min(first + tid / LP, items - 1);
        t.live = in && first + tid / LP < items;
        t.r = ROWS == 1 ? 0 : i / heads;
        t.h = i - t.r * heads;
        t.key = t.h >= a.H;
        t.h -= t.key ? a.H : 0;
        const T *x = static_cast<const T *>(t.key ? a.k : a.q) +
                     (size_t)(row0 + t.r) * (t.key ? a.k_stride : a.q_stride) + t.h * a.D + (in ? part : 0);
        t.x.load(x);
        return t;
    };
    constexpr int STEP = 256 / LP;
    int first = blockIdx.y * STEP;
    if (a.T == 0 || first >= items) {
        if (a.T == 0 && wave == 0) row_position(a, 0);  // reports sequences without rows
        return;
    }
    Item t = fetch(first);
    // every wavefront (ROWS 1), or wavefront w for row w
    int pos = kNoRow;
    if (ROWS == 1 || wave < rows) {
        pos = row_position(a, row0 + (ROWS == 1 ? 0 : wave));
        if (ROWS > 1 && lane_id() == 0) s_pos[wave] = pos;
    }
    if constexpr (ROWS > 1) __syncthreads();
    for (int i = tid; i < rows * P; i += 256) {
        const int r = ROWS == 1 ? 0 : i / P, j = i - r * P;
        const int at = ROWS == 1 ? pos : s_pos[r];
        if (at < 0) continue;
        const float2 y = turn_of(at, a.inv_freq[j]);
        s_cos[r][j] = y.x, s_sin[r][j] = y.y;
    }
    __syncthreads();
    for (; first < items; first += STEP * gridDim.y) {
        Item next = t;
        if (first + STEP * (int)gridDim.y < items) next = fetch(first + STEP * gridDim.y);
        const T *w = static_cast<const T *>(t.key ? a.k_weight : a.q_weight);
        float v[8], u[8], sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[e] = t.x.get(e);
            sum = fmaf(in ? v[e] : 0.f, v[e], sum);
        }
        sum = sum_lanes<LP>(in ? sum : 0.f);
        Eight<T> x2 = t.x, w1, w2;
        if (!INTER && P > 0) x2 = t.x.from(other);
        const int at = ROWS == 1 ? pos : s_pos[t.r];
        if (w) {
            const float scale = 1.f / sqrtf(sum / a.D + a.eps);
            w1.load(w + (in ? part : 0));
            w2 = w1;
            if (!INTER && turned) w2.load(w + part + (second ? -P : P));
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] = v[e] * scale * w1.get(e);
                u[e] = x2.get(e) * scale * w2.get(e);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = x2.get(e);
        }
        if (turned && at >= 0) {
            if constexpr (INTER) {
                const f32x4 co = *reinterpret_cast<const f32x4 *>(&s_cos[t.r][part / 2]);
                const f32x4 si = *reinterpret_cast<const f32x4 *>(&s_sin[t.r][part / 2]);
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float x = v[e], y = v[e + 1];
                    v[e] = fmaf(-y, si[e / 2], x * co[e / 2]);
                    v[e + 1] = fmaf(x, si[e / 2], y * co[e / 2]);
                }
            } else {
                const int j = second ? part - P : part;
                const f32x4 *co = reinterpret_cast<const f32x4 *>(&s_cos[t.r][j]), *si = reinterpret_cast<const f32x4 *>(&s_sin[t.r][j]);
                const f32x4 cs[2] = {co[0], co[1]}, sn[2] = {si[0], si[1]};
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = fmaf(second ? u[e] : -u[e], sn[e >> 2][e & 3], v[e] * cs[e >> 2][e & 3]);
            }
        }
        if (at == kNanRowAt) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __builtin_nanf("");
        }
        if (t.live && at != kNoRow)
            Eight<T>::store(static_cast<T *>(t.key ? a.k_out : a.q_out) +
                            ((size_t)(row0 + t.r) * (t.key ? a.HK : a.H) + t.h) * a.D + part, v);
        t = next;
    }
}

// ---- host

template <typename T, int LP, bool INTER>
static hipError_t launch_lanes(const RotaryArgs &a, hipStream_t stream) {
    // four rows a workgroup once that leaves every CU two of them
    if (a.T >= 2048) {
        rotary_kernel<T, LP, INTER, 4><<<dim3((unsigned)((a.T + 3) / 4)), dim3(256), 0, stream>>>(a);
    } else {
        const int passes = ((a.H + a.HK) * LP + 255) / 256;
        rotary_kernel<T, LP, INTER, 1><<<dim3((unsigned)(a.T > 0 ? a.T : 1), (unsigned)passes), dim3(256), 0, stream>>>(a);
    }
    return hipGetLastError();
}

template <typename T, bool INTER>
static hipError_t launch_pairs(const RotaryArgs &a, hipStream_t stream) {
    if (a.D <= 64) return launch_lanes<T, 8, INTER>(a, stream);
    if (a.D <= 128) return launch_lanes<T, 16, INTER>(a, stream);
    return launch_lanes<T, 32, INTER>(a, stream);
}

template <typename T>
static hipError_t launch_typed(const RotaryArgs &a, bool interleaved, bool generic, hipStream_t stream) {
    uintptr_t bits = (uintptr_t)(a.q_stride * sizeof(T)) | (uintptr_t)(a.k_stride * sizeof(T));
    for (const void *p : {a.q, a.k, a.q_weight, a.k_weight, static_cast<const void *>(a.q_out), static_cast<const void *>(a.k_out)})
        bits |= reinterpret_cast<uintptr_t>(p);
    if (generic || bits % 16 != 0 || a.D % 8 != 0 || a.R % (interleaved ? 8 : 16) != 0) {
        rotary_generic_kernel<T><<<dim3((unsigned)(a.T > 0 ? a.T : 1)), dim3(256), 0, stream>>>(a, interleaved);
        return hipGetLastError();
    }
    return interleaved ? launch_pairs<T, true>(a, stream) : launch_pairs<T, false>(a, stream);
}

hipError_t launch_rotary(const void *q, const void *k, const void *q_weight, const void *k_weight,
                         const float *inv_freq, const int32_t *first_position, const int32_t *parent,
                         const int32_t *node_offsets, void *q_out, void *k_out,
                         const bole_rotary_dims_t &d, int32_t *seq_status, hipStream_t stream) {
    const RotaryArgs a = {q, k, q_weight, k_weight, inv_freq, first_position, parent, node_offsets,
                          q_out, k_out, seq_status, d.batch, d.heads, d.kv_heads, d.head_dim,
                          d.rotary_dim, d.total_rows, d.q_stride, d.k_stride, d.eps};
    const bool inter = d.flags & BOLE_FLAG_INTERLEAVED, generic = d.flags & BOLE_FLAG_FORCE_GENERIC;
    return d.dtype == BOLE_DTYPE_F32 ? launch_typed<float>(a, inter, generic, stream)
                                     : launch_typed<__bf16>(a, inter, generic, stream);
}

}  // namespace bole

extern "C" {

bole_status_t bole_rotary_check_dims(const bole_rotary_dims_t *d) {
    if (d == nullptr) return BOLE_ERR_INVALID_VALUE;
    if (d->batch < 0 || d->heads < 1 || d->kv_heads < 1 || d->head_dim < 1 || d->total_rows < 0 ||
        d->rotary_dim < 0 || d->rotary_dim % 2 != 0 || d->rotary_dim > d->head_dim)
        return BOLE_ERR_INVALID_VALUE;
    if (d->dtype != BOLE_DTYPE_BF16 && d->dtype != BOLE_DTYPE_F32) return BOLE_ERR_INVALID_VALUE;
    if (d->flags & ~(BOLE_FLAG_FORCE_GENERIC | BOLE_FLAG_INTERLEAVED)) return BOLE_ERR_INVALID_VALUE;
    if (!std::isfinite(d->eps) || d->eps < 0.f) return BOLE_ERR_INVALID_VALUE;
    if (d->q_stride < (int64_t)d->heads * d->head_dim || d->k_stride < (int64_t)d->kv_heads * d->head_dim)
        return BOLE_ERR_INVALID_VALUE;
    // a launch has fewer than 2^32 threads, 256 a row
    if (d->head_dim > 256 || d->heads > 65535 || d->kv_heads > 65535 || d->total_rows >= 1 << 24)
        return BOLE_ERR_UNSUPPORTED;
    return BOLE_OK;
}

bole_status_t bole_qk_norm_rotary(const void *q, const void *k, const void *q_weight,
                                  const void *k_weight, const float *inv_freq,
                                  const int32_t *first_position, const int32_t *parent,
                                  const int32_t *node_offsets, void *q_out, void *k_out,
                                  const bole_rotary_dims_t *dims, int32_t *seq_status,
                                  bole_stream_t stream) {
    const bole_status_t st = bole_rotary_check_dims(dims);
    if (st != BOLE_OK) return st;
    const bole_rotary_dims_t &d = *dims;
    if (d.batch == 0) return BOLE_OK;
    if (first_position == nullptr || node_offsets == nullptr || (d.rotary_dim > 0 && inv_freq == nullptr))
        return BOLE_ERR_INVALID_VALUE;
    if (d.total_rows > 0 && (q == nullptr || k == nullptr || q_out == nullptr || k_out == nullptr))
        return BOLE_ERR_INVALID_VALUE;
    const hipError_t e = bole::launch_rotary(q, k, q_weight, k_weight, inv_freq, first_position, parent,
                                             node_offsets, q_out, k_out, d, seq_status,
                                             reinterpret_cast<hipStream_t>(stream));
    return e == hipSuccess ? BOLE_OK : BOLE_ERR_HIP;
}

}  // extern "C"
