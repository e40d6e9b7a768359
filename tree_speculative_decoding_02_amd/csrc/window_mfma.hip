// window_mfma.hip - windowed attention on the matrix cores, bf16, head widths 64, 96 and 128.
//
// A sequence's rows and the G = H / H_kv query heads that share a key head are packed as
// rows R = i G + g, so one pass over the keys serves all of them. With the transposed score
// tile S^T = K Q^T (keys down, queries across), a lane holds one query: its running maximum
// and sum are lane-local up to a last exchange between the lanes that share the query, and
// the exponentials, rounded to bf16, already lie as the B operand of O^T = V^T P^T (a
// permutation of the keys within a product, the same for both operands). V^T comes from
// row-major LDS through the transposing read.
//
// The keys a tile of rows can see are one virtual list: the cached first tokens and the cached
// window behind the tile's first row, then, on a key tile's edge, the call's own first tokens and
// own rows. Tiles of 64 keys that every row sees are taken without tests; the others test each
// key. Slots past the end of either part repeat its last key, so nothing that no row of the
// sequence sees is read, and no load depends on a branch.
//
// Two shapes of workgroup:
//  - rows: 128 rows, 32 a wavefront, keys and values staged in LDS for all four wavefronts
//    (two buffers, one barrier a tile). For prompts and draft trees.
//  - tokens: 16 rows, the key tiles dealt to the four wavefronts, each with its own softmax
//    state, merged at the end; keys go straight to registers. For single tokens, where the
//    cache's bytes set the time.
// With few rows in the whole call the key list is also split over workgroups; a second kernel
// merges the parts.
//
// Measured, 32 query heads over 8 key heads of 128, a window of 4096 (prompts: 1024) and 4 first
// tokens: 64 single tokens 162 us (5.7 TB/s), 64 draft trees of up to 32 nodes 171 us (5.4 TB/s),
// both bound by the cache's bytes; one single token 11 us, its two kernels' chains of loads; two
// prompts of 8192 tokens 363 us (761 TFLOP/s). Of those the matrix instructions alone take 177,
// with LDS reads and exponentials 266; the rest is keys on their way through registers to LDS.
#include "window_rows.h"
#include "launch.h"

namespace bole {

// ---- host

static bool covers(const bole_window_dims_t &d) {
    return !(d.flags & BOLE_FLAG_FORCE_GENERIC) &&
           (d.head_dim == 64 || d.head_dim == 96 || d.head_dim == 128) && d.batch > 0;
}

// From a call's sizes alone. The tokens form (bf16) for up to one of its tiles a sequence on
// average: with 8 rows 189 us against 193 in the rows form (64 sequences), 29 against 33 (8); from
// 20 rows on 238 against 192, 35 against 35. Parts so that 512 workgroups (two a CU) run, but no more
// than one for each 256 keys begun (so that each has more than 128): of 8 single tokens 29 us, with
// 256 or 768 workgroups 35 and 32; one token in parts of 128 or 512 keys 15 and 14 us against 11.
// The keys are those that the cache can show a row, and the row's own: lengths are not known here,
// and a prompt's own rows are not counted, so one behind a short cache runs in one part.
static WindowPlan plan(const bole_window_dims_t &d) {
    WindowPlan p;
    const int64_t G = d.heads / d.kv_heads, rows = d.total_rows * G;
    p.f32 = d.dtype == BOLE_DTYPE_F32;
    p.tokens = !p.f32 && rows <= 16LL * d.batch;
    p.tile = p.f32 ? 64 : p.tokens ? kTokenTile : kRowTile;
    p.slots = (int)(rows / p.tile + d.batch);
    const int64_t cached = (int64_t)d.max_pages * d.page_size;
    const int64_t seen = (cached < (int64_t)d.window + d.sinks ? cached : (int64_t)d.window + d.sinks) + 1;
    const int64_t base = (int64_t)p.slots * d.kv_heads;
    int64_t n = (512 + base - 1) / base;
    if (n > (seen + 255) / 256) n = (seen + 255) / 256;
    p.parts = (int)(n > 64 ? 64 : n < 1 ? 1 : n);
    return p;
}

size_t window_workspace(const bole_window_dims_t &d) {
    if (!covers(d)) return 0;
    const WindowPlan p = plan(d);
    if (p.parts == 1) return 0;
    return (size_t)p.parts * p.slots * d.kv_heads * p.tile * (d.head_dim + 2) * sizeof(float);
}

bool window_mfma_applies(const bole_window_dims_t &d, const WindowArgs &a) {
    uintptr_t bits = 0;
    for (const void *p : {a.q, a.k, a.v, a.k_cache, a.v_cache, static_cast<const void *>(a.out)})
        bits |= reinterpret_cast<uintptr_t>(p);
    return covers(d) && bits % 16 == 0;
}

template <int D>
__global__ __launch_bounds__(256, 2) void window_rows_kernel(const WindowArgs a, const WindowParts parts,
                                                             int slots) {
    __shared__ __align__(16) char s_mem[kRowsLds<D>];
    rows_body<D>(WindowKeys{a}, parts, slots, blockIdx.x, blockIdx.y, s_mem);
}

template <int D>
__global__ __launch_bounds__(256, 2) void window_tokens_kernel(const WindowArgs a, const WindowParts parts,
                                                               int slots) {
    __shared__ __align__(16) char s_mem[kTokensLds<D>];
    tokens_body<D>(WindowKeys{a}, parts, slots, blockIdx.x, blockIdx.y, s_mem);
}

template <int D>
static hipError_t launch_width(const WindowArgs &a, const bole_window_dims_t &d, const WindowPlan &p,
                               const WindowParts &parts, hipStream_t stream) {
    const dim3 grid((unsigned)(p.slots * d.kv_heads), (unsigned)p.parts), block(256);
    if (p.tokens)
        window_tokens_kernel<D><<<grid, block, 0, stream>>>(a, parts, p.slots);
    else
        window_rows_kernel<D><<<grid, block, 0, stream>>>(a, parts, p.slots);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && p.parts > 1) {
        if (p.tokens)
            window_join_kernel<__bf16, D, kTokenTile><<<dim3(grid.x, kTokenTile), block, 0, stream>>>(a, parts, p.slots);
        else
            window_join_kernel<__bf16, D, kRowTile><<<dim3(grid.x, kRowTile), block, 0, stream>>>(a, parts, p.slots);
        e = hipGetLastError();
    }
    return e;
}

hipError_t launch_window_mfma(const WindowArgs &a, const bole_window_dims_t &d, void *workspace,
                              hipStream_t stream) {
    const WindowPlan p = plan(d);
    WindowParts parts = {static_cast<float *>(workspace), nullptr, p.parts};
    if (p.parts > 1)
        parts.ml = parts.o + (size_t)p.parts * p.slots * d.kv_heads * p.tile * d.head_dim;
    if (p.f32) return launch_window_f32(a, p, parts, stream);
    switch (d.head_dim) {
        case 64: return launch_width<64>(a, d, p, parts, stream);
        case 96: return launch_width<96>(a, d, p, parts, stream);
        default: return launch_width<128>(a, d, p, parts, stream);
    }
}

}  // namespace bole
