// gfx950 kernel of dropout: y = x under a mask drawn from a counter [+ add].
// 8 columns a lane, one generator block each (ten rounds of two 32 x 32 -> 64 bit
// products).  HBM bound: 16384 x 4096 bf16 51 us, 5.2 TB/s, as a copy; 777 x 1001
// float32 4.2 us, a launch.

#include "blocknorm_device.hpp"

namespace muon {
namespace {

// A workgroup takes rpb rows of `slots` 8-column runs each.
template <class T>
__global__ __launch_bounds__(256) void dropout_kernel(DropoutArgs a, int rpb, int slots) {
    constexpr int V = sizeof(T) == 2 ? 8 : 4, R = 8 / V;
    const Philox m(a.drop);
    const int64_t r0 = int64_t(blockIdx.x) * rpb;
    for (int i = threadIdx.x; i < rpb * slots; i += 256) {
        const int rl = i / slots, c = (i - rl * slots) * 8;
        const int64_t row = r0 + rl;
        if (row >= a.rows) return;
        const int n = a.cols - c;
        float v[8];
        const GMEM T* x = gm(static_cast<const T*>(a.x)) + row * a.ld_x + c;
#pragma unroll
        for (int h = 0; h < R; ++h) run_decode<T, V>(run_get<T, V, false>(x + h * V, n - h * V), v + h * V);
        if (m.cut) {
            const u32x4_t w = m.words(uint32_t(a.row0 + row), uint32_t(c >> 3));
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = m.keep(v[k], w[k >> 1], k & 1);
        }
        if (a.add) {
            const GMEM T* p = gm(static_cast<const T*>(a.add)) + row * a.ld_add + c;
            float b[8];
#pragma unroll
            for (int h = 0; h < R; ++h) run_decode<T, V>(run_get<T, V, false>(p + h * V, n - h * V), b + h * V);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] += b[k];
        }
        GMEM T* y = gm(static_cast<T*>(a.y)) + row * a.ld_y + c;
#pragma unroll
        for (int h = 0; h < R; ++h) run_put<T, V, false>(y + h * V, n - h * V, run_encode<T, V>(v + h * V));
    }
}

}  // namespace

// One launch, or more past 2^31 threads, each of whole workgroups' rows.
hipError_t launch_dropout(const DropoutArgs& a, hipStream_t s) {
    const int slots = (a.cols + 7) / 8;
    // four runs a thread, fewer where that leaves fewer than 8 workgroups a CU (777 x
    // 1001 float32, one run: 6.3 us; four: 6.9)
    const int64_t runs = a.rows * slots / (256 * 2048), most = (runs < 1 ? 1 : runs > 4 ? 4 : runs) * 256;
    const int rpb = slots >= most ? 1 : int(most / slots);
    const int64_t slice = (kSliceThreads + 255) / 256 * rpb, es = a.dt == 0 ? 2 : 4;
    for (int64_t r0 = 0; r0 < a.rows; r0 += slice) {
        DropoutArgs b = a;
        b.rows = a.rows - r0 < slice ? a.rows - r0 : slice;
        b.row0 = r0;
        b.x = static_cast<const char*>(a.x) + r0 * a.ld_x * es;
        b.y = static_cast<char*>(a.y) + r0 * a.ld_y * es;
        if (a.add) b.add = static_cast<const char*>(a.add) + r0 * a.ld_add * es;
        const dim3 grid(unsigned((b.rows + rpb - 1) / rpb)), block(256);
        if (a.dt == 0) hipLaunchKernelGGL((dropout_kernel<uint16_t>), grid, block, 0, s, b, rpb, slots);
        else hipLaunchKernelGGL((dropout_kernel<float>), grid, block, 0, s, b, rpb, slots);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace muon
