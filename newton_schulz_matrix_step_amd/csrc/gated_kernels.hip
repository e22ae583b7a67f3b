// gfx950 kernels of the gated feed-forward's products:
//
//   forward          zg = x Wg + bg, zu = x Wu + bu, h = act(zg) zu   (zg, zu kept, also in 8 bits)
//   hidden gradient  dh = dy Wd^T, dzg = dh zu act'(zg), dzu = dh act(zg)   (h written beside them)
//   input gradient   dx = dzg Wg^T + dzu Wu^T + add
//   weight gradient  dWg = x^T dzg, dWu = x^T dzu, column sums dbg, dbu
//
// Each is one launch of the tile kernels of linear_device.hpp: the forward's
// tiles hold the same columns of both projections, so that a lane has both
// sums of its elements; the input gradient is one sum over twice the k; the
// weight gradient's tiles are both outputs'.  Sums are float32, every result is
// rounded once.
//
// Measured, bf16 (MI355X; HBM copies 4.7-5.1 TB/s): forward of 1 token 4096 -> 14336
// 45-52 us on several cards, both weights, out x in, at 4.5-5.2 TB/s (in x out 69: a
// tile's row of k is 64 bytes of each); of 4096 tokens 714-758 us, 1.27-1.35 PFLOP/s,
// matrix pipes busy 69 %.  Smaller products are bound by one or two rounds of tiles
// and their epilogues: hidden gradient of 4001 x 2816 <- 1024 with 8-bit
// pre-activations 55-61 us, with full ones 57 (29 with a k of 64: half is prologue and
// epilogue, with 92 MB through 176 workgroups, one a CU), input gradient of 8192 x 1024 <- 2816 90-95
// (the join of two splits 14), both weight gradients of 8192 x 2048 -> 1408 117-122
// (352 tiles; decoding x 11).

#include "linear_device.hpp"

namespace muon {
namespace {

// The splits' sums, added in order, through the epilogue: 8 elements a lane.
// blockIdx.y is the output of a PAIR_OUT call; the workgroups past the output's
// join the column sums.
__device__ __forceinline__ void add_partial(const GMEM float* p, int64_t step, int splits, float (&v)[8]) {
    for (int s = 0; s < splits; ++s, p += step) {
        const f32x4_t x = *reinterpret_cast<const GMEM f32x4_t*>(p);
        const f32x4_t y = *reinterpret_cast<const GMEM f32x4_t*>(p + 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[k] += x[k];
            v[4 + k] += y[k];
        }
    }
}
__global__ __launch_bounds__(256) void gated_join_kernel(GatedArgs a, int64_t out_blocks) {
    const OutShape o = out_shape(a);
    const int64_t one = o.rows * o.ldp;                  // elements of a split's sums
    if (blockIdx.y) {
        a.out = a.out2;
        a.db = a.db2;
        a.partial += a.splits * one;
        if (a.db_partial) a.db_partial += a.splits * a.N;
    }
    if (int64_t(blockIdx.x) >= out_blocks) {
        const int64_t n = (int64_t(blockIdx.x) - out_blocks) * 256 + threadIdx.x;
        if (n >= a.N || !a.db) return;
        float v = 0.f;
        for (int s = 0; s < a.splits; ++s) v += gm(a.db_partial)[int64_t(s) * a.N + n];
        if (a.accumulate) v += load1(a.db, n, a.db_dt);
        store1(a.db, n, a.db_dt, v);
        return;
    }
    const int64_t rpr = o.ldp / 8;                       // runs per row, a multiple of 4
    const int64_t idx = int64_t(blockIdx.x) * 256 + threadIdx.x;
    const int64_t r = idx / rpr, c = (idx % rpr) * 8;
    int64_t n = o.cols - c;
    n = r < o.rows ? (n > 8 ? 8 : n) : 0;
    const int nv = n > 0 ? int(n) : 0;
    float v[8], u[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = u[k] = 0.f;
    const GMEM float* p = gm(a.partial) + r * o.ldp + c;
    if (a.pair == PAIR_COLS) {
        if (nv) {
            add_partial(p, 2 * one, a.splits, v);
            add_partial(p + one, 2 * one, a.splits, u);
        }
        gated_any(a, r, c, nv, v, u);
    } else {
        if (nv) add_partial(p, one, a.splits, v);
        run_any(a, r, c, nv, v);
    }
}

int64_t tiles_of(const GatedArgs& a, int edge) {
    const int64_t ce = a.pair == PAIR_COLS ? edge / 2 : edge;
    return ((a.M + edge - 1) / edge) * ((a.N + ce - 1) / ce) * (a.pair == PAIR_OUT ? 2 : 1);
}

template <class T, bool AKC, bool BKC, int KIND, bool TR, int PAIR>
hipError_t launch_tile(const GatedArgs& a, hipStream_t s) {
    const dim3 grid(unsigned((tiles_of(a, a.tile) * a.splits + 7) / 8 * 8)), block(256);
    if (a.tile == 64 && a.deep)
        hipLaunchKernelGGL((linear_tile_kernel<T, AKC, BKC, S_DMA, S_DMA, KIND, TR, 64, 8, PAIR>), grid, block, 0, s, a);
    else if (a.tile == 64)
        hipLaunchKernelGGL((linear_tile_kernel<T, AKC, BKC, S_DMA, S_DMA, KIND, TR, 64, 4, PAIR>), grid, block, 0, s, a);
    else if (a.deep)
        hipLaunchKernelGGL((linear_tile_kernel<T, AKC, BKC, S_DMA, S_DMA, KIND, TR, 128, 4, PAIR>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((linear_tile_kernel<T, AKC, BKC, S_DMA, S_DMA, KIND, TR, 128, 2, PAIR>), grid, block, 0, s, a);
    return hipGetLastError();
}
template <bool AKC, bool BKC, int KIND, bool TR, int PAIR>
hipError_t launch_kernel(const GatedArgs& a, hipStream_t s) {
    if (a.tile == 256) {
        const dim3 grid(unsigned((tiles_of(a, 256) * a.splits + 7) / 8 * 8));
        hipLaunchKernelGGL((linear_pp_kernel<AKC, BKC, KIND, TR, PAIR>), grid, dim3(kPpThreads), 0, s, a);
        return hipGetLastError();
    }
    return a.dt == 0 ? launch_tile<uint16_t, AKC, BKC, KIND, TR, PAIR>(a, s)
                     : launch_tile<float, AKC, BKC, KIND, TR, PAIR>(a, s);
}

}  // namespace

int64_t gated_tiles128(const GatedArgs& a) { return tiles_of(a, 128); }

// Tile edge and split: the cheapest by a model of the product's time in us, fitted
// to the four products at ten sizes each in both weight layouts, bf16, on one
// MI355X (float32: at six).  With w workgroups a CU and `per` k blocks of 128
// bytes a row in each:
//
//   edge 64    fixed + (block per + tile) max(w, 1)
//   edge 128   one + block1 per                           w <= 1 (four LDS stages)
//              fixed + (block per + tile) w               else
//   edge 256   ceil(w) (fixed + block per)                `block` grows with the CUs at work (clocks fall)
//
// `tile` and `fixed` hold the epilogue, which is what the hidden gradient spends
// most on: five tensors of its size pass through it.  Both sides, measured:
// 1024 x 1024 -> 1408 hidden, forward 18.5, 14.8 and 28.1 us on edges 64, 128 and
// 256; 4096 x 1024 -> 2816, weight gradient 57.9 on 128, 70.9 on 256; 4096 x 4096
// -> 14336, forward 1004 and 735; 4096 x 1024 -> 1408, hidden gradient 28.5 and
// 53.5.  A split adds the joining kernel (4 us and its sums' bytes, which the
// caches hold: 14 us for two splits of 8192 x 1024).
// Operands without whole aligned chunks are always copied first to rows that have
// them, 8-bit ones decoded: the pairs' kernels have no other source.  It costs most
// where the weights' bytes bound the call (1 token 4096 -> 14335, in x out: 220 us,
// aligned 69; 4095 -> 14335, out x in: 199, aligned 46).  The model leaves it out, as
// it falls on every tile and split alike.
// MUON_LINEAR_EDGE fixes the edge where that tile can serve the call (a host
// build for bounds checking runs each kernel on small sizes); 0: by the model.
#ifndef MUON_LINEAR_EDGE
#define MUON_LINEAR_EDGE 0
#endif
struct GatedCost {
    double fixed64, block64, tile64;
    double one128, block1_128, fixed128, block128, tile128;
    double fixed256, block256, grow256;   // a k block's time at half the CUs or fewer, and how it grows to all
};
//                                       64               128                        256
constexpr GatedCost kForwardCost = {4, 0.19, 1.4, 6.5, 0.50, 8, 0.49, 0.55, 14.5, 0.85, 0.7};
constexpr GatedCost kHiddenCost = {5, 0.20, 2.6, 12, 0.55, 8, 0.55, 9.0, 38, 0.95, 0.9};
constexpr GatedCost kInputCost = {4, 0.21, 0.8, 4, 0.56, 8, 0.45, 0.5, 13, 0.95, 0.9};
constexpr GatedCost kWeightCost = {4, 0.24, 1.0, 5, 0.60, 8, 0.55, 0.5, 17, 1.5, 0};

double gated_us(const GatedArgs& a, int edge, double w, double per) {
    // float32: bound by the matrix pipes, a CU's workgroups one after the other (309 x
    // 5472 -> 2952 forward: 1.8 workgroups a CU of edge 64 171 us, 1.1 of edge 128 331)
    if (a.dt != 0) {
        const bool dh = a.kind == LIN_GATED_DH;
        const double block = w <= 1 ? 0.66 : a.kind == LIN_GATED ? 0.50 : a.kind == LIN_DW ? 0.57 : 0.53;
        if (edge == 64) return 4 + (block * per + (dh ? 2.6 : 1)) * std::ceil(w);
        return 6 + (w <= 1 ? 1.9 * per : 1.85 * per + 2) * std::ceil(w) + (dh ? 16 * std::ceil(w) : 0);
    }
    const GatedCost& c = a.kind == LIN_GATED ? kForwardCost : a.kind == LIN_GATED_DH ? kHiddenCost
                                               : a.kind == LIN_DX                   ? kInputCost
                                                                                    : kWeightCost;
    if (edge == 64) return c.fixed64 + (c.block64 * per + c.tile64) * std::max(w, 1.0);
    if (edge == 128) return w <= 1 ? c.one128 + c.block1_128 * per : c.fixed128 + (c.block128 * per + c.tile128) * w;
    double block = c.block256 + c.grow256 * std::max(w / std::ceil(w) - 0.5, 0.0);
    if (a.a_kc && a.b_kc) block *= 0.93;
    return std::ceil(w) * (c.fixed256 + block * per);
}

GatedPlan plan_gated(GatedArgs& a) {
    const OutShape o = out_shape(a);
    const int64_t bk = a.dt == 0 ? 64 : 32, nkb = (a.K + bk - 1) / bk * (a.pair == PAIR_K ? 2 : 1);
    const double outs = a.pair == PAIR_COLS || a.pair == PAIR_OUT ? 2 : 1, ins = a.pair == PAIR_K ? 2 : 1;
    const double sum_bytes = outs * double(o.rows) * double(o.ldp) * 8;
    const double bytes_us = (ins * double(a.M) * double(a.K) + (a.pair == PAIR_NONE ? 1 : 2) * double(a.K) * double(a.N)) *
                            (a.dt == 0 ? 2 : 4) / 5e6;
    double best = 1e30;
    a.tile = 64;
    a.splits = 1;
    for (int edge = 64; edge <= (a.dt == 0 ? 256 : 128); edge *= 2) {
        const int64_t tiles = tiles_of(a, edge), most = std::min<int64_t>(std::min<int64_t>(nkb / 2, 512 / tiles), 64);
        for (int64_t s = 1; s <= std::max<int64_t>(most, 1); ++s) {
            const int64_t per = (nkb + s - 1) / s;
            if (s > 1 && (nkb + per - 1) / per != s) continue;   // it would leave a split empty
            if ((tiles * s + 7) / 8 * 8 * (edge == 256 ? 512 : 256) >= kGridThreads) continue;
            double us = std::max(gated_us(a, edge, double(tiles * s) / 256, double(per)), bytes_us);
            if (s > 1) us += (a.dt == 0 ? 4 : 8) + double(s) * sum_bytes / 1.2e7;
            if (MUON_LINEAR_EDGE && edge != MUON_LINEAR_EDGE) us += 1e9;
            if (us < best) {
                best = us;
                a.tile = edge;
                a.splits = int(s);
            }
        }
    }
    a.deep = tiles_of(a, a.tile) * a.splits <= 256;
    const int64_t chunk = a.dt == 0 ? 8 : 4, es = a.dt == 0 ? 2 : 4;
    const int64_t ar = a.a_kc ? a.M : a.K, ac = a.a_kc ? a.K : a.M, br = a.b_kc ? a.N : a.K, bc = a.b_kc ? a.K : a.N;
    a.a_ld = a.a_dma ? 0 : (ac + chunk - 1) / chunk * chunk;
    a.b_ld = a.b_dma ? 0 : (bc + chunk - 1) / chunk * chunk;
    GatedPlan g;
    g.a_bytes = size_t(a.a_ld) * size_t(ar) * size_t(es);
    g.b_bytes = size_t(a.b_ld) * size_t(br) * size_t(es);
    if (a.splits > 1) {
        g.partial_bytes = size_t(outs) * size_t(a.splits) * size_t(o.rows) * size_t(o.ldp) * 4;
        g.db_bytes = a.db || a.db2 ? size_t(outs) * size_t(a.splits) * size_t(a.N) * 4 : 0;
    }
    return g;
}

hipError_t launch_gated(const GatedArgs& args, hipStream_t s) {
    GatedArgs a = args;
    if (a.M <= 0 || a.N <= 0) return hipSuccess;
    const int64_t ar = a.a_kc ? a.M : a.K, ac = a.a_kc ? a.K : a.M, br = a.b_kc ? a.N : a.K, bc = a.b_kc ? a.K : a.N;
    hipError_t e = hipSuccess;
    if (a.a_ld) {        // operands with rows of whole aligned chunks, in the workspace
        if (a.a_exps) {
            Act8Args q;
            q.x = nullptr;
            q.y = a.a_ws;
            q.q = Act8View{static_cast<int8_t*>(const_cast<void*>(a.a)), const_cast<uint8_t*>(a.a_exps), a.lda,
                           a.lda_exps, a.a8_vec};
            q.rows = ar;
            q.ld = a.a_ld;
            q.cols = int32_t(ac);
            q.dt = a.dt;
            q.vec = a.a8_vec;
            e = launch_act8_decode(q, s);
        } else {
            e = launch_pack(a.a, a.lda, a.a_ws, a.a_ld, ar, ac, a.dt, s);
            if (e == hipSuccess && a.pair == PAIR_K) e = launch_pack(a.a2, a.lda, a.a2_ws, a.a_ld, ar, ac, a.dt, s);
        }
        if (e != hipSuccess) return e;
        a.a = a.a_ws;
        a.a2 = a.a2_ws;
        a.lda = a.a_ld;
    }
    if (a.b_ld) {
        e = launch_pack(a.b, a.ldb, a.b_ws, a.b_ld, br, bc, a.dt, s);
        if (e == hipSuccess && a.pair != PAIR_NONE) e = launch_pack(a.b2, a.ldb, a.b2_ws, a.b_ld, br, bc, a.dt, s);
        if (e != hipSuccess) return e;
        a.b = a.b_ws;
        a.b2 = a.b2_ws;
        a.ldb = a.b_ld;
    }
    if (a.pair == PAIR_COLS)
        e = a.b_kc ? launch_kernel<true, true, LIN_GATED, false, PAIR_COLS>(a, s)
                   : launch_kernel<true, false, LIN_GATED, false, PAIR_COLS>(a, s);
    else if (a.pair == PAIR_K)
        e = a.b_kc ? launch_kernel<true, true, LIN_DX, false, PAIR_K>(a, s)
                   : launch_kernel<true, false, LIN_DX, false, PAIR_K>(a, s);
    else if (a.pair == PAIR_OUT)
        e = a.out_trans ? launch_kernel<false, false, LIN_DW, true, PAIR_OUT>(a, s)
                        : launch_kernel<false, false, LIN_DW, false, PAIR_OUT>(a, s);
    else
        e = a.b_kc ? launch_kernel<true, true, LIN_GATED_DH, false, PAIR_NONE>(a, s)
                   : launch_kernel<true, false, LIN_GATED_DH, false, PAIR_NONE>(a, s);
    if (e != hipSuccess || a.splits <= 1) return e;
    const OutShape o = out_shape(a);
    const int64_t ob = (o.rows * (o.ldp / 8) + 255) / 256, db = a.db || a.db2 ? (a.N + 255) / 256 : 0;
    hipLaunchKernelGGL(gated_join_kernel, dim3(unsigned(ob + db), a.pair == PAIR_OUT ? 2u : 1u), dim3(256), 0, s, a, ob);
    return hipGetLastError();
}

}  // namespace muon
