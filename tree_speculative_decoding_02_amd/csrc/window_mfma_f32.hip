// window_mfma_f32.hip - windowed attention on the fp32 matrix instructions, head widths 64, 96
// and 128. The same shape as the bf16 rows form (window_mfma.hip): S^T = K Q^T, a query a lane
// group of 16 lanes' column, and the exponentials in registers are the right operand of
// O^T = V^T P^T as they are: of v_mfma_f32_16x16x4_f32's results lane group g holds rows
// 4 g .. 4 g + 3, and with step r of a product taking keys {4 g + r} from every group, register
// r is that step's operand.
//
// One workgroup: 64 rows, 16 a wavefront, keys and values staged in LDS 64 at a time, the next
// 64 in registers meanwhile. The fp32 matrix rate (a sixteenth of bf16's) bounds prompts and
// trees, the cache's bytes single tokens: 32 heads over 8 of 128, a window of 4096, 64 single
// tokens 442 us (4.2 TB/s), 64 trees of up to 32 nodes 1077 us (45 TFLOP/s, the matrix instructions
// at work half of the time); two prompts of 2048 tokens, window 1024, 679 us (102 TFLOP/s).
#include "window_rows_f32.h"
#include "launch.h"

namespace bole {

template <int D>
__global__ __launch_bounds__(256, 2) void window_f32_kernel(const WindowArgs a, const WindowParts parts,
                                                            int slots) {
    __shared__ __align__(16) char s_mem[kF32Lds<D>];
    f32_body<D>(WindowKeys{a}, parts, slots, blockIdx.x, blockIdx.y, s_mem);
}

template <int D>
static hipError_t launch_width(const WindowArgs &a, const WindowPlan &p, const WindowParts &parts,
                               hipStream_t stream) {
    const unsigned tiles = (unsigned)(p.slots * a.s.HK);
    window_f32_kernel<D><<<dim3(tiles, (unsigned)p.parts), dim3(256), 0, stream>>>(a, parts, p.slots);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && p.parts > 1) {
        window_join_kernel<float, D, kF32Tile><<<dim3(tiles, kF32Tile), dim3(256), 0, stream>>>(a, parts, p.slots);
        e = hipGetLastError();
    }
    return e;
}

hipError_t launch_window_f32(const WindowArgs &a, const WindowPlan &p, const WindowParts &parts,
                             hipStream_t stream) {
    switch (a.s.D) {
        case 64: return launch_width<64>(a, p, parts, stream);
        case 96: return launch_width<96>(a, p, parts, stream);
        default: return launch_width<128>(a, p, parts, stream);
    }
}

}  // namespace bole
