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

hipError_t launch_rotary(const void *q, const void *k, const void *q_weight, const void *k_weight,
                         const float *inv_freq, const int32_t *first_position, const int32_t *parent,
                         const int32_t *node_offsets, void *q_out, void *k_out,
                         const bole_rotary_dims_t &d, int32_t *seq_status, hipStream_t stream) {
    const RotaryArgs a = {q, k, q_weight, k_weight, inv_freq, first_position, parent, node_offsets,
                          q_out, k_out, seq_status, d.batch, d.heads, d.kv_heads, d.head_dim,
                          d.rotary_dim, d.total_rows, d.q_stride, d.k_stride, d.eps};
    const bool inter = d.flags & BOLE_FLAG_INTERLEAVED;
    const dim3 grid((unsigned)(d.total_rows > 0 ? d.total_rows : 1)), block(256);
    if (d.dtype == BOLE_DTYPE_F32)
        rotary_generic_kernel<float><<<grid, block, 0, stream>>>(a, inter);
    else
        rotary_generic_kernel<__bf16><<<grid, block, 0, stream>>>(a, inter);
    return hipGetLastError();
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
