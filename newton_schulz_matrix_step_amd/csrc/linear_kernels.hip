// gfx950 kernels of the linear layer's three products:
//
//   forward          y  = act(x W + b) + residual           (z = x W + b kept, also in 8 bits)
//   input gradient   dx = (dy W^T) act'(z) + add            (act(z) written beside it)
//   weight gradient  dW = x^T dy, db = column sums of dy    (x also from its 8-bit checkpoint)
//
// Each is one product C = A B over k with its own operand layouts and epilogue;
// products run on the matrix cores (v_mfma_f32_16x16x32_bf16, or
// v_mfma_f32_16x16x4_f32 for float32 tensors) with float32 sums, and every
// result is rounded once, at its store.

#include "linear_device.hpp"

namespace muon {
namespace {

// ---------------------------------------------------------------------------
// The splits' sums, added in order, through the epilogue: 8 elements a lane.
// The workgroups past the output's join the column sums.  HBM bound for large
// outputs (four splits of 1024 x 4096: 76 MB in 11.9 us), else a launch (4.5 us).
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void linear_join_kernel(LinArgs a, int64_t out_blocks) {
    if (int64_t(blockIdx.x) >= out_blocks) {
        const int64_t n = (int64_t(blockIdx.x) - out_blocks) * 256 + threadIdx.x;
        if (n >= a.N) return;
        float v = 0.f;
        for (int s = 0; s < a.splits; ++s) v += gm(a.db_partial)[int64_t(s) * a.N + n];
        if (a.accumulate) v += load1(a.db, n, a.db_dt);
        store1(a.db, n, a.db_dt, v);
        return;
    }
    const OutShape o = out_shape(a);
    const int64_t rpr = o.ldp / 8;                       // runs per row, a multiple of 4
    const int64_t idx = int64_t(blockIdx.x) * 256 + threadIdx.x;
    const int64_t r = idx / rpr, c = (idx % rpr) * 8;
    int64_t n = o.cols - c;
    n = r < o.rows ? (n > 8 ? 8 : n) : 0;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.f;
    if (n > 0) {
        const GMEM float* p = gm(a.partial) + r * o.ldp + c;
        for (int s = 0; s < a.splits; ++s, p += o.rows * o.ldp) {
            const f32x4_t x = *reinterpret_cast<const GMEM f32x4_t*>(p);
            const f32x4_t y = *reinterpret_cast<const GMEM f32x4_t*>(p + 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[k] += x[k];
                v[4 + k] += y[k];
            }
        }
    }
    epilogue_any(a, r, c, n > 0 ? int(n) : 0, v);
}

// An operand with rows that are not whole aligned 16-byte chunks, copied into
// the workspace with such rows (their ends zero): 16 bytes a lane.
template <class T>
__global__ __launch_bounds__(256) void linear_pack_kernel(const T* src, int64_t ld, T* dst, int64_t ldd, int64_t rows,
                                                          int64_t cols) {
    constexpr int E = Num<T>::EPC;
    const int64_t cpr = ldd / E, i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    const int64_t r = i / cpr, c = (i - r * cpr) * E;
    if (r >= rows) return;
    const GMEM T* p = gm(src) + r * ld + c;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (c + e < cols) {
            if constexpr (Num<T>::dt == 0) w[e / 2] |= uint32_t(p[e]) << (16 * (e & 1));
            else w[e] = __float_as_uint(p[e]);
        }
    *reinterpret_cast<GMEM u32x4_t*>(gm(dst) + r * ldd + c) = u32x4_t{w[0], w[1], w[2], w[3]};
}
template <class T>
hipError_t launch_pack_typed(const T* src, int64_t ld, T* dst, int64_t ldd, int64_t rows, int64_t cols, hipStream_t s) {
    const int64_t cpr = ldd / Num<T>::EPC, slice = (kSliceThreads + cpr - 1) / cpr;   // rows of a launch
    for (int64_t r0 = 0; r0 < rows; r0 += slice) {
        const int64_t nr = rows - r0 < slice ? rows - r0 : slice;
        hipLaunchKernelGGL((linear_pack_kernel<T>), dim3(unsigned((nr * cpr + 255) / 256)), dim3(256), 0, s, src + r0 * ld,
                           ld, dst + r0 * ldd, ldd, nr, cols);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}
}  // namespace

hipError_t launch_pack(const void* src, int64_t ld, void* dst, int64_t ldd, int64_t rows, int64_t cols, int dt,
                       hipStream_t s) {
    return dt == 0 ? launch_pack_typed(static_cast<const uint16_t*>(src), ld, static_cast<uint16_t*>(dst), ldd, rows, cols, s)
                   : launch_pack_typed(static_cast<const float*>(src), ld, static_cast<float*>(dst), ldd, rows, cols, s);
}

namespace {

template <class T, bool AKC, bool BKC, int ASRC, int BSRC, int KIND, bool TR>
hipError_t launch_tile(const LinArgs& a, hipStream_t s) {
    const int64_t nm = (a.M + a.tile - 1) / a.tile, nn = (a.N + a.tile - 1) / a.tile, all = nm * nn * a.splits;
    const dim3 grid(unsigned((all + 7) / 8 * 8)), block(256);
    constexpr bool dma = ASRC == S_DMA && BSRC == S_DMA;
    if (a.tile == 64) {
        if constexpr (dma) {
            if (a.deep) {
                hipLaunchKernelGGL((linear_tile_kernel<T, AKC, BKC, ASRC, BSRC, KIND, TR, 64, 8>), grid, block, 0, s, a);
                return hipGetLastError();
            }
        }
        hipLaunchKernelGGL((linear_tile_kernel<T, AKC, BKC, ASRC, BSRC, KIND, TR, 64, dma ? 4 : 2>), grid, block, 0, s, a);
    } else {
        if constexpr (dma) {
            if (a.deep) {
                hipLaunchKernelGGL((linear_tile_kernel<T, AKC, BKC, ASRC, BSRC, KIND, TR, 128, 4>), grid, block, 0, s, a);
                return hipGetLastError();
            }
        }
        hipLaunchKernelGGL((linear_tile_kernel<T, AKC, BKC, ASRC, BSRC, KIND, TR, 128, 2>), grid, block, 0, s, a);
    }
    return hipGetLastError();
}
template <bool AKC, bool BKC, int KIND, bool TR>
hipError_t launch_pp(const LinArgs& a, hipStream_t s) {
    const int64_t nm = (a.M + 255) / 256, nn = (a.N + 255) / 256, all = nm * nn * a.splits;
    hipLaunchKernelGGL((linear_pp_kernel<AKC, BKC, KIND, TR>), dim3(unsigned((all + 7) / 8 * 8)), dim3(kPpThreads), 0, s,
                       a);
    return hipGetLastError();
}

hipError_t launch_256(const LinArgs& a, hipStream_t s) {
    if (a.kind == LIN_FWD)
        return a.b_kc ? launch_pp<true, true, LIN_FWD, false>(a, s) : launch_pp<true, false, LIN_FWD, false>(a, s);
    if (a.kind == LIN_DX)
        return a.b_kc ? launch_pp<true, true, LIN_DX, false>(a, s) : launch_pp<true, false, LIN_DX, false>(a, s);
    return a.out_trans ? launch_pp<false, false, LIN_DW, true>(a, s) : launch_pp<false, false, LIN_DW, false>(a, s);
}

// x W or dy W^T: B by rows (KC) or by columns of k; element-wise loads for both
// operands where either needs them.
template <class T, bool BKC>
hipError_t launch_rows(const LinArgs& a, hipStream_t s) {
    if (!a.a_dma || !a.b_dma) return launch_tile<T, true, BKC, S_ANY, S_ANY, -1, false>(a, s);
    return a.kind == LIN_FWD ? launch_tile<T, true, BKC, S_DMA, S_DMA, LIN_FWD, false>(a, s)
                             : launch_tile<T, true, BKC, S_DMA, S_DMA, LIN_DX, false>(a, s);
}
template <class T, bool TR>
hipError_t launch_dw(const LinArgs& a, hipStream_t s) {
    if (a.a_exps)
        return a.b_dma ? launch_tile<T, false, false, S_ACT8, S_DMA, LIN_DW, TR>(a, s)
                       : launch_tile<T, false, false, S_ACT8, S_ANY, -1, TR>(a, s);
    return a.a_dma && a.b_dma ? launch_tile<T, false, false, S_DMA, S_DMA, LIN_DW, TR>(a, s)
                              : launch_tile<T, false, false, S_ANY, S_ANY, -1, TR>(a, s);
}

template <class T>
hipError_t launch_typed(const LinArgs& a, hipStream_t s) {
    if (a.kind == LIN_DW) return a.out_trans ? launch_dw<T, true>(a, s) : launch_dw<T, false>(a, s);
    return a.b_kc ? launch_rows<T, true>(a, s) : launch_rows<T, false>(a, s);
}

}  // namespace

// Tile edge and split of a product: the cheapest by a model of its time in us,
// fitted to graph replays on one MI355X.  A tile takes a fixed time (launch,
// first loads, epilogue) and a time per k block of 128 bytes a row, which grows
// with the workgroups that share a CU:
//
//   edge  fixed  per k block: bf16 (weight gradient)  float32
//     64   3.5     0.25 (0.40)                          0.45
//    128   5.5     0.50 (0.75), 0.58 shared             1.75
//    256   11      1.42, 1.30 both row-contiguous (1.50)
//
// No product is faster than its operands' bytes at 5 TB/s.  A split adds the
// joining kernel (4 us and its sums' bytes).  Both sides, measured: 1024 x 1024
// -> 1024 8.5 us on 64-wide tiles, 13 on 128-wide ones, 14 split in two; 2048 x
// 2048 -> 1408 26, 23 and 52 us on 64, 128 and 256; 4096 x 4096 -> 4096 150 us on
// 128, 106 on 256.
// An 8-bit operand is decoded by the product itself, which doubles its time per
// k block, or by a pass of its own into the workspace (1024 x 1000, 500 tokens:
// 9.8 us by itself, 13 in two passes; 4000 tokens: 34 and 32).  Operands without
// whole aligned chunks are read element by element by the product, about nine
// times slower per k block, or copied first to rows that have them (4000 x 3001
// -> 2047: 480 and 89 us; 1 x 2001 -> 999: 14 and 17).
// MUON_LINEAR_EDGE fixes the edge where that tile can serve the call (a host
// build for bounds checking runs each kernel on small sizes); 0: by the model.
#ifndef MUON_LINEAR_EDGE
#define MUON_LINEAR_EDGE 0
#endif
struct TileCost {
    int edge;
    double fixed, block, block_dw, block_f32;
};
constexpr TileCost kTileCosts[] = {{64, 3.5, 0.25, 0.40, 0.45}, {128, 5.5, 0.50, 0.75, 1.75}, {256, 11, 1.42, 1.50, 0}};

LinPlan plan_linear(const LinArgs& a) {
    LinPlan best;
    double best_us = 1e30;
    const OutShape o = out_shape(a);
    const int64_t bk = a.dt == 0 ? 64 : 32, nkb = (a.K + bk - 1) / bk;
    const double es = a.dt == 0 ? 2 : 4;
    const double bytes_us = (double(a.M) * double(a.K) + double(a.K) * double(a.N)) * es / 5e6;
    // rows and columns of the operands as stored, and their re-laid leading dimensions
    const int64_t ar = a.a_kc ? a.M : a.K, ac = a.a_kc ? a.K : a.M, br = a.b_kc ? a.N : a.K, bc = a.b_kc ? a.K : a.N;
    const int64_t chunk = a.dt == 0 ? 8 : 4, lda = (ac + chunk - 1) / chunk * chunk, ldb = (bc + chunk - 1) / chunk * chunk;
    // operands taken as they are (0), or those that need it re-laid first (1): an
    // 8-bit one decoded, a ragged or misaligned one packed
    const bool plain = a.a_dma && a.b_dma;
    for (int relay = 0; relay <= (plain ? 0 : 1); ++relay) {
        const bool fused8 = a.a_exps && !relay, dma = relay || plain;
        double relay_us = 0;
        if (relay && !a.a_dma) relay_us += 4 + double(ar) * double(ac) * es * (a.a_exps ? 1.5 : 2) / 4.5e6;
        if (relay && !a.b_dma) relay_us += 4 + double(br) * double(bc) * es * 2 / 4.5e6;
        for (const TileCost& tc : kTileCosts) {
            if (tc.edge == 256 && (a.dt != 0 || !dma)) continue;
            const int64_t tiles = ((a.M + tc.edge - 1) / tc.edge) * ((a.N + tc.edge - 1) / tc.edge);
            double block = a.dt != 0 ? tc.block_f32 : a.kind == LIN_DW ? tc.block_dw : tc.block;
            if (tc.edge == 256 && a.a_kc && a.b_kc) block = 1.30;
            if (!dma) block *= fused8 && a.b_dma ? 2.0 : 9.0;
            // a split keeps at least 2 k blocks and at most fills two workgroups a CU
            const int64_t most = std::min<int64_t>(std::min<int64_t>(nkb / 2, 512 / tiles), 64);
            for (int64_t s = 1; s <= std::max<int64_t>(most, 1); ++s) {
                const int64_t per = (nkb + s - 1) / s;
                if (s > 1 && (nkb + per - 1) / per != s) continue;   // it would leave a split empty
                if ((tiles * s + 7) / 8 * 8 * (tc.edge == 256 ? 512 : 256) >= kGridThreads) continue;
                const double w = double(tiles * s) / 256;            // workgroups a CU
                double us;
                if (tc.edge == 256) us = 3 + std::ceil(w) * (tc.fixed + block * double(per));
                else if (tc.edge == 64 || w <= 1) us = tc.fixed + block * std::max(w, 1.0) * double(per);
                else us = tc.fixed + 1.16 * block * 2 * std::ceil(w / 2) * double(per);
                us = std::max(us, bytes_us);
                if (s > 1) us += 4 + double(s) * double(o.rows) * double(o.ldp) * 8 / 5e6;
                us += relay_us;
                if (MUON_LINEAR_EDGE && tc.edge != MUON_LINEAR_EDGE) us += 1e9;
                if (us < best_us) {
                    best_us = us;
                    best.tile = tc.edge;
                    best.splits = int(s);
                    best.deep = tiles * s <= 256;
                    best.a_ld = relay && !a.a_dma ? lda : 0;
                    best.b_ld = relay && !a.b_dma ? ldb : 0;
                }
            }
        }
    }
    best.a_bytes = size_t(best.a_ld) * size_t(ar) * size_t(es);
    best.b_bytes = size_t(best.b_ld) * size_t(br) * size_t(es);
    if (best.splits > 1) {
        best.partial_bytes = size_t(best.splits) * size_t(o.rows) * size_t(o.ldp) * 4;
        best.db_bytes = a.db ? size_t(best.splits) * size_t(a.N) * 4 : 0;
    }
    return best;
}

hipError_t launch_linear(const LinArgs& args, hipStream_t s) {
    LinArgs a = args;
    if (a.M <= 0 || a.N <= 0) return hipSuccess;
    if (a.a_ld) {        // re-lay A in the workspace
        const int64_t rows = a.a_kc ? a.M : a.K, cols = a.a_kc ? a.K : a.M;
        hipError_t d;
        if (a.a_exps) {
            Act8Args q;
            q.x = nullptr;
            q.y = a.a_ws;
            q.q = Act8View{static_cast<int8_t*>(const_cast<void*>(a.a)), const_cast<uint8_t*>(a.a_exps), a.lda,
                           a.lda_exps, a.a8_vec};
            q.rows = rows;
            q.ld = a.a_ld;
            q.cols = int32_t(cols);
            q.dt = a.dt;
            q.vec = a.a8_vec;
            d = launch_act8_decode(q, s);
        } else {
            d = launch_pack(a.a, a.lda, a.a_ws, a.a_ld, rows, cols, a.dt, s);
        }
        if (d != hipSuccess) return d;
        a.a = a.a_ws;
        a.lda = a.a_ld;
        a.a_exps = nullptr;
        a.a_dma = 1;
    }
    if (a.b_ld) {
        const hipError_t d =
            launch_pack(a.b, a.ldb, a.b_ws, a.b_ld, a.b_kc ? a.N : a.K, a.b_kc ? a.K : a.N, a.dt, s);
        if (d != hipSuccess) return d;
        a.b = a.b_ws;
        a.ldb = a.b_ld;
        a.b_dma = 1;
    }
    hipError_t e = a.tile == 256 ? launch_256(a, s)
                                 : (a.dt == 0 ? launch_typed<uint16_t>(a, s) : launch_typed<float>(a, s));
    if (e != hipSuccess || a.splits <= 1) return e;
    const OutShape o = out_shape(a);
    const int64_t ob = (o.rows * (o.ldp / 8) + 255) / 256, db = a.db ? (a.N + 255) / 256 : 0;
    hipLaunchKernelGGL(linear_join_kernel, dim3(unsigned(ob + db)), dim3(256), 0, s, a, ob);
    return hipGetLastError();
}

}  // namespace muon
