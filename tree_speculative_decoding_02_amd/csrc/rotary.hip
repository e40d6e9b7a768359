// rotary.hip - norm of every head's query and key and its rotation by position, in one pass:
//     y = x / sqrt(mean(x^2) + eps) * weight,
//     (y_a, y_b) <- (y_a cos t - y_b sin t, y_b cos t + y_a sin t),   t = position * inv_freq[j].
//
// A row's angles are the same for all of its heads: they are taken once, in fp64, reduced to one
// turn, and their sines and cosines kept in LDS (an fp32 angle at position 2^20 is off by 2^-5).
// Bound by the rows' way through HBM, 2 bytes read and 2 written an element in bf16: two prompts of 8192
// tokens, 32 query and 8 key heads of 128, 71 us (4.7 TB/s); 64 single tokens 4.8 us, launch and chain.
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
// With ROWS 1 the heads of few rows are dealt to gridDim.y workgroups: what takes time there is the
// chain of loads behind a row's position.
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

// What multiplies an element and its pair's other one, for each row: weight times cosine and, with
// its sign, the other's weight times sine. So a head costs three operations an element (with both
// weights and the angle apart it was bound by the vector units: two prompts of 8192 tokens 84 us).
// Element 8 c + i of a head at [i / 4][c][i % 4], so that neighbouring lanes read 16-byte neighbours.
template <int LP, int ROWS>
struct RotaryTables {
    float own[ROWS][2][8 * LP], other[ROWS][2][8 * LP];  // [row][query or key]
    int pos[ROWS];
    static __device__ __forceinline__ int at(int e) { return ((e >> 2) & 1) * 4 * LP + (e >> 3) * 4 + (e & 3); }
};

template <typename T, int LP, bool INTER, int ROWS>
__global__ __launch_bounds__(256) void rotary_kernel(const RotaryArgs a) {
    __shared__ __align__(16) RotaryTables<LP, ROWS> t;
    const int tid = threadIdx.x, wave = tid >> 6, row0 = blockIdx.x * ROWS, P = a.R / 2;
    const int rows = min(ROWS, a.T - row0);
    const int c = tid % LP, part = 8 * c;               // the lane's elements of its head
    const bool in = part < a.D;
    const int half = P / 8;                             // pairs (j, j + half): the other's lane
    const int from = (tid & 63) + (c >= half ? -half : half);
    constexpr int STEP = 256 / LP;
    // a pass takes STEP heads of the rows' queries, then of their keys
    const int q_passes = (rows * a.H + STEP - 1) / STEP, passes = q_passes + (rows * a.HK + STEP - 1) / STEP;
    int pass = blockIdx.y;
    if (a.T == 0 || pass >= passes) {
        if (a.T == 0 && wave == 0) row_position(a, 0);  // reports sequences without rows
        return;
    }
    struct Item {
        int r, h;
        bool live;
        Eight<T> x;
    };
    auto fetch = [&](int p) {
        const bool key = p >= q_passes;
        const int heads = key ? a.HK : a.H, i = (key ? p - q_passes : p) * STEP + tid / LP;
        const T *x = static_cast<const T *>(key ? a.k : a.q);
        const int64_t stride = key ? a.k_stride : a.q_stride;
        Item y;
        y.live = in && i < rows * heads;
        // (exact: below 2^19 halves and whole numbers lie apart in fp32 by more than the product's error)
        y.r = ROWS == 1 ? 0 : min((int)(((float)i + 0.5f) * (1.f / (float)heads)), rows - 1);
        y.h = min(i - y.r * heads, heads - 1);
        y.x.load(x + (size_t)row0 * stride + (size_t)y.r * stride + (uint32_t)(y.h * a.D + (in ? part : 0)));
        return y;
    };
    Item y = fetch(pass);
    // every wavefront (ROWS 1), or wavefront w for row w
    int pos = kNoRow;
    if (ROWS == 1 || wave < rows) {
        pos = row_position(a, row0 + (ROWS == 1 ? 0 : wave));
        if (ROWS > 1 && lane_id() == 0) t.pos[wave] = pos;
    }
    if constexpr (ROWS > 1) __syncthreads();
    for (int k = tid; k < rows * (a.D - P); k += 256) {  // pairs, then elements that are not turned
        const int r = ROWS == 1 ? 0 : k / (a.D - P), j = k - r * (a.D - P);
        const int at = ROWS == 1 ? pos : t.pos[r];
        if (at == kNoRow) continue;
        const bool pair = j < P;
        const int ea = !pair ? j + P : INTER ? 2 * j : j, eb = INTER ? 2 * j + 1 : j + P;
        const float2 turn = pair && at >= 0 ? turn_of(at, a.inv_freq[j]) : float2{1.f, 0.f};
        const float bad = at == kNanRowAt ? __builtin_nanf("") : 1.f;
#pragma unroll
        for (int key = 0; key < 2; ++key) {
            const T *w = static_cast<const T *>(key ? a.k_weight : a.q_weight);
            const float wa = w ? to_f32(w[ea]) : 1.f, wb = w && pair ? to_f32(w[eb]) : 1.f;
            t.own[r][key][t.at(ea)] = bad * wa * turn.x;
            t.other[r][key][t.at(ea)] = -wb * turn.y;
            if (pair) {
                t.own[r][key][t.at(eb)] = bad * wb * turn.x;
                t.other[r][key][t.at(eb)] = wa * turn.y;
            }
        }
    }
    __syncthreads();
    const float inv_d = 1.f / (float)a.D;
    for (; pass < passes; pass += gridDim.y) {
        Item next = y;
        if (pass + (int)gridDim.y < passes) next = fetch(pass + gridDim.y);
        const bool key = pass >= q_passes;
        float v[8], u[8], sum = 0.f, scale = 1.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = y.x.get(e);
        if (key ? a.k_weight != nullptr : a.q_weight != nullptr) {
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fmaf(v[e], v[e], sum);
            const float mean = fmaf(sum_lanes<LP>(in ? sum : 0.f), inv_d, a.eps);
            const bool tiny = mean < 0x1p-100f;  // (the instruction takes no denormals)
            scale = __builtin_amdgcn_rsqf(tiny ? mean * 0x1p64f : mean) * (tiny ? 0x1p32f : 1.f);
        }
        if constexpr (INTER) {
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = part < a.R ? v[e ^ 1] : 0.f;
        } else {
            Eight<T> z = y.x;
            if (P > 0) z = y.x.from(from);
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = part < a.R ? z.get(e) : 0.f;
        }
        const f32x4 *own = reinterpret_cast<const f32x4 *>(t.own[y.r][key]) + c;
        const f32x4 *other = reinterpret_cast<const f32x4 *>(t.other[y.r][key]) + c;
        const f32x4 ow[2] = {own[0], own[LP]}, ot[2] = {other[0], other[LP]};
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fmaf(u[e], ot[e >> 2][e & 3], v[e] * ow[e >> 2][e & 3]) * scale;
        if (y.live && (ROWS == 1 ? pos : t.pos[y.r]) != kNoRow)
            Eight<T>::store(static_cast<T *>(key ? a.k_out : a.q_out) +
                            ((size_t)(row0 + y.r) * (key ? a.HK : a.H) + y.h) * a.D + part, v);
        y = next;
    }
}

// ---- host

template <typename T, int LP, bool INTER>
static hipError_t launch_lanes(const RotaryArgs &a, hipStream_t stream) {
    // Four rows a workgroup from 4096 rows on (40 heads of 128: 16384 rows 71 us, 77 with one row each, 4096
    // 19.9 and 19.8, 2048 13.9 and 11.0), one from 512 on, and two passes of one below (500 rows 6.4 us, one
    // pass 7.2, whole rows 6.7).
    if (a.T >= 4096) {
        rotary_kernel<T, LP, INTER, 4><<<dim3((unsigned)((a.T + 3) / 4)), dim3(256), 0, stream>>>(a);
    } else {
        const int passes = (a.H * LP + 255) / 256 + (a.HK * LP + 255) / 256;
        const dim3 grid((unsigned)(a.T > 0 ? a.T : 1), a.T >= 512 ? 1u : (unsigned)(passes + 1) / 2);
        rotary_kernel<T, LP, INTER, 1><<<grid, dim3(256), 0, stream>>>(a);
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
