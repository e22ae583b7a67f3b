// gfx950 kernels of the junction between two blocks, backward:
//
//   g  = ds + r (a - [mean a] - xh mean(a xh)),  a = dy gain, xh = (s - mu) r      (norm_pre)
//   dx = alpha g,  e = drop(g),  b = beta e gate gain,  oh = (branch - mu') r'
//   dbranch = r' (b - [mean b] - oh mean(b oh))                                    (norm_post)
//
// ([..]: layer norm only) and over the rows P = sum dy xh, Q = sum dy, S = sum e oh
// and D = sum e, from which dpre_gain = P, dpre_bias = Q, dpost_gain = beta gate S,
// dpost_bias = beta gate D, dgate = beta (gain S + bias D).
//
// One pass over the rows, HBM bound; a workgroup keeps the column sums of its
// rows in registers and a second kernel adds the workgroups' in a fixed order.
// Measured: 8192 x 4096 bf16 RMS 88 us, layer norms 95-99 (the bytes 78.5 at a copy's
// rate); with a float32 stream 122 and 128-130 (118); 4096 x 8192 with one and layer
// norms 189-202: sixteen waves spill.

#include "blocknorm_device.hpp"

namespace muon {
namespace {

// LAYER: means, and the sums Q and D.
template <class ST, class BT, int NW, bool LAYER>
__global__ __launch_bounds__(block_waves(NW) * 64, LAYER && sizeof(ST) == 4 && NW < 16 ? 2 : 4) void blocknorm_grad_kernel(BlockNormGradArgs a) {
    constexpr int E = kRowElems, RB = block_waves(NW) / NW, NT = block_waves(NW) * 64;
    using G = BlockRow<run_width<ST, BT>(), NW, E>;
    __shared__ float red[2][2][block_waves(NW)];
    __shared__ float cs[RB > 1 ? NT * E : 1];       // [row group][element][lane]
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6)), rg = wave / NW;   // (rows are scalar)
    const int lane = wave % NW * 64 + int(threadIdx.x & 63);
    const Philox m(a.drop);
    const bool has_b = a.dbranch != nullptr, has_o = a.branch != nullptr;
    float sum[LAYER ? 4 : 2][E];                     // P, S (, Q, D)
#pragma unroll
    for (int q = 0; q < (LAYER ? 4 : 2); ++q)
#pragma unroll
        for (int i = 0; i < E; ++i) sum[q][i] = 0.f;
    const float inv_n = 1.f / float(a.cols);
    const int64_t step = int64_t(gridDim.x) * RB;
    typename G::template Raw<BT> ry, ro;
    typename G::template Raw<ST> rs, rd;
    auto load = [&](int64_t row) {
        const bool in = row < a.rows;
        if (a.pre) {
            G::template load<BT, true>(a.dy, row * a.ld_dy, a.cols, lane, in, ry);
            G::template load<ST, true>(a.s, row * a.ld_s, a.cols, lane, in, rs);
        }
        if (a.ds) G::template load<ST, true>(a.ds, row * a.ld_ds, a.cols, lane, in, rd);
        if (has_o) G::template load<BT, true>(a.branch, row * a.ld_branch, a.cols, lane, in, ro);
    };
    int64_t r0 = int64_t(blockIdx.x) * RB;
    if (r0 < a.rows) load(r0 + rg);
    // the factors of both norms' gradients wait in LDS: a lane's 8 of each would
    // cost registers for a third row in flight
    __shared__ __align__(16) float par[2][E / 4][G::LANES][4];
    if (rg == 0) {
        float w[E];
        if (has_b) {
            G::param(a.post_gain, a.pdt, a.cols, lane, 1.f, w);
            if (a.gate) {
                float g[E];
                G::param(a.gate, a.pdt, a.cols, lane, 1.f, g);
#pragma unroll
                for (int i = 0; i < E; ++i) w[i] *= g[i];
            }
#pragma unroll
            for (int i = 0; i < E; ++i) par[1][i / 4][lane][i % 4] = w[i] * a.beta;
        }
        G::param(a.pre_gain, a.pdt, a.cols, lane, 1.f, w);
#pragma unroll
        for (int i = 0; i < E; ++i) par[0][i / 4][lane][i % 4] = w[i];
    }
    __syncthreads();
    auto factors = [&](int which, float (&w)[E]) {
#pragma unroll
        for (int q = 0; q < E / 4; ++q) {
            const f32x4_t t = *reinterpret_cast<const f32x4_t*>(par[which][q][lane]);
#pragma unroll
            for (int k = 0; k < 4; ++k) w[4 * q + k] = t[k];
        }
    };
    RowSums<NW> sums{red, wave};
    for (; r0 < a.rows; r0 += step) {
        const int64_t row = r0 + rg;
        const bool on = row < a.rows;
        float g[E], h[E], o[E];
        float mu = 0.f, r = 0.f, pm = 0.f, pr = 1.f;
        if (a.pre && on) {
            r = gm(a.pre_rstd)[row];
            if (LAYER && a.pre == NORM_LAYER) mu = gm(a.pre_mean)[row];
        }
        if (a.post && on) {
            pr = gm(a.post_rstd)[row];
            if (LAYER && a.post == NORM_LAYER) pm = gm(a.post_mean)[row];
        }
        if (a.pre) {
            G::decode(ry, a.cols, lane, g);
            G::decode(rs, a.cols, lane, h);
        }
        if (a.ds) {
            float t[E];
            G::decode(rd, a.cols, lane, t);
#pragma unroll
            for (int i = 0; i < E; ++i) o[i] = t[i];
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) o[i] = 0.f;
        }
        if (a.pre) {
            float s[2] = {0.f, 0.f}, w[E];
            factors(0, w);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                // past the last column dy and the gain are 0, so xh there adds nothing
                h[i] = (h[i] - mu) * r;
                sum[0][i] = fmaf(g[i], h[i], sum[0][i]);
                if constexpr (LAYER) sum[2][i] += g[i];
                g[i] *= w[i];
                if constexpr (LAYER) s[0] += g[i];
                s[1] = fmaf(g[i], h[i], s[1]);
            }
            sums(s);
            const float c1 = LAYER && a.pre == NORM_LAYER ? s[0] * inv_n : 0.f, c2 = s[1] * inv_n;
#pragma unroll
            for (int i = 0; i < E; ++i) g[i] = fmaf(r, g[i] - c1 - h[i] * c2, o[i]);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) g[i] = o[i];
        }
        if (has_o) G::decode(ro, a.cols, lane, o);
        // (ds may be dx: another row's, not yet written)
        load(row + step);
        typename G::template Raw<ST> out;
#pragma unroll
        for (int i = 0; i < E; ++i) h[i] = a.alpha * g[i];
        G::encode(h, out);
        if (on) G::template store<ST, false>(a.dx, row * a.ld_dx, a.cols, lane, out);
        if (!has_b) continue;
        // what is dropped adds nothing, whatever it was (a norm's row is NaN with it)
        if (m.cut) G::mask(m, uint32_t(row), lane, g, o, !a.post);
        float w[E];
        factors(1, w);
        if (has_o) {
            float s[2] = {0.f, 0.f};
#pragma unroll
            for (int j = 0; j < G::C; ++j)
#pragma unroll
                for (int k = 0; k < G::V; ++k) {
                    const int i = j * G::V + k;
                    // past the last column g is not 0 under a layer norm: the sums leave it out by the gain there
                    o[i] = (o[i] - pm) * pr;
                    sum[1][i] = fmaf(g[i], o[i], sum[1][i]);
                    if constexpr (LAYER) sum[3][i] += g[i];
                    g[i] *= w[i];
                    if constexpr (LAYER) s[0] += g[i];
                    s[1] = fmaf(g[i], o[i], s[1]);
                }
            if (a.post) {
                sums(s);
                const float c1 = LAYER && a.post == NORM_LAYER ? s[0] * inv_n : 0.f, c2 = s[1] * inv_n;
#pragma unroll
                for (int i = 0; i < E; ++i) g[i] = pr * (g[i] - c1 - o[i] * c2);
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) g[i] *= w[i];
        }
        typename G::template Raw<BT> ob;
        G::encode(g, ob);
        if (on) G::template store<BT, false>(a.dbranch, row * a.ld_dbranch, a.cols, lane, ob);
    }
    // the column sums, one kind at a time: of a workgroup's row groups through LDS
#pragma unroll
    for (int q = 0; q < (LAYER ? 4 : 2); ++q) {
        const int at = a.at[q == 0 ? 0 : q == 1 ? 2 : q == 2 ? 1 : 3];
        if (at < 0) continue;
        GMEM float* p = gm(a.partial) + (int64_t(at) * a.parts + blockIdx.x) * a.cols;
        if constexpr (RB > 1) {
            constexpr int kOne = G::LANES * E;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < E; ++i) cs[(rg * E + i) * G::LANES + lane] = sum[q][i];
            __syncthreads();
            for (int w = threadIdx.x; w < kOne; w += NT) {
                const int i = w / G::LANES, l = w % G::LANES;
                float v = 0.f;
#pragma unroll
                for (int x = 0; x < RB; ++x) v += cs[x * kOne + w];
                const int c = G::col(i / G::V, l) + i % G::V;
                if (c < a.cols) p[c] = v;
            }
        } else {
            G::store_f32(p, a.cols, lane, sum[q]);
        }
    }
}

// Rows longer than the registers hold, or shorter than a run: a workgroup walks rows, 8 columns a lane
// at a time, three passes over each; a lane adds to its own columns' sums in the
// workgroup's row of partial sums.  Far from its bytes (4096 x 12288 bf16, RMS 1220 us,
// layer norms 1490, where the bytes take 118): single elements, and the partial sums
// read and written for every row.
__global__ __launch_bounds__(kNT) void blocknorm_grad_long_kernel(BlockNormGradArgs a) {
    __shared__ float red[kWaves];
    const Philox m(a.drop);
    const float n = float(a.cols);
    const bool has_b = a.dbranch != nullptr, has_o = a.branch != nullptr;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const bool first = row == blockIdx.x;
        const float r = a.pre ? gm(a.pre_rstd)[row] : 0.f, mu = a.pre == NORM_LAYER ? gm(a.pre_mean)[row] : 0.f;
        const float pr = a.post ? gm(a.post_rstd)[row] : 1.f, pm = a.post == NORM_LAYER ? gm(a.post_mean)[row] : 0.f;
        float c1 = 0.f, c2 = 0.f;
        // dy, xh and a of 8 columns
        auto pre8 = [&](int c, float(&y)[8], float(&x)[8], float(&t)[8]) {
            const int nv = a.cols - c;
            get8(a.dy, row * a.ld_dy + c, a.dt, nv, y);
            get8(a.s, row * a.ld_s + c, a.sdt, nv, x);
            par8(a.pre_gain, c, a.pdt, nv, 1.f, t);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                x[k] = k < nv ? (x[k] - mu) * r : 0.f;
                t[k] *= y[k];
            }
        };
        if (a.pre) {
            float s0 = 0.f, s1 = 0.f;
            for (int c = threadIdx.x * 8; c < a.cols; c += kNT * 8) {
                float y[8], x[8], t[8];
                pre8(c, y, x, t);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    s0 += t[k];
                    s1 = fmaf(t[k], x[k], s1);
                }
            }
            s0 = block_add(s0, red);
            s1 = block_add(s1, red);
            c1 = a.pre == NORM_LAYER ? s0 / n : 0.f;
            c2 = s1 / n;
        }
        // g of 8 columns (and, with sums, what dy adds to them)
        auto put = [&](int which, int c, const float(&v)[8]) {
            if (a.at[which] < 0) return;
            GMEM float* p = gm(a.partial) + (int64_t(a.at[which]) * a.parts + blockIdx.x) * a.cols + c;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (c + k < a.cols) p[k] = first ? v[k] : p[k] + v[k];
        };
        auto g8 = [&](int c, bool sums, float(&g)[8]) {
            const int nv = a.cols - c;
            if (a.ds) get8(a.ds, row * a.ld_ds + c, a.sdt, nv, g);
            else
#pragma unroll
                for (int k = 0; k < 8; ++k) g[k] = 0.f;
            if (!a.pre) return;
            float y[8], x[8], t[8];
            pre8(c, y, x, t);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                g[k] = fmaf(r, t[k] - c1 - x[k] * c2, g[k]);
                x[k] *= y[k];
            }
            if (sums) {
                put(0, c, x);
                put(1, c, y);
            }
        };
        // b and oh of 8 columns from g
        auto post8 = [&](int c, bool sums, float(&g)[8], float(&o)[8]) {
            const int nv = a.cols - c;
            float w[8], f[8];
            par8(a.post_gain, c, a.pdt, nv, 1.f, w);
            par8(a.gate, c, a.pdt, nv, 1.f, f);
            get8(a.branch, row * a.ld_branch + c, a.dt, has_o ? nv : 0, o);
            if (m.cut) m.run<8>(uint32_t(row), uint32_t(c), g, o, !a.post);   // (dropped: nothing)
            float e[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                o[k] = has_o && k < nv ? (o[k] - pm) * pr : 0.f;
                e[k] = g[k] * o[k];
            }
            if (sums) {
                put(2, c, e);
                put(3, c, g);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) g[k] *= w[k] * f[k] * a.beta;
        };
        float d1 = 0.f, d2 = 0.f;
        if (a.post) {
            float s0 = 0.f, s1 = 0.f;
            for (int c = threadIdx.x * 8; c < a.cols; c += kNT * 8) {
                float g[8], o[8];
                g8(c, false, g);
                post8(c, false, g, o);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (c + k < a.cols) {
                        s0 += g[k];
                        s1 = fmaf(g[k], o[k], s1);
                    }
            }
            s0 = block_add(s0, red);
            s1 = block_add(s1, red);
            d1 = a.post == NORM_LAYER ? s0 / n : 0.f;
            d2 = s1 / n;
        }
        for (int c = threadIdx.x * 8; c < a.cols; c += kNT * 8) {   // (a lane reads ds before it writes dx there)
            float g[8], v[8];
            g8(c, true, g);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = a.alpha * g[k];
            store8(a.dx, row * a.ld_dx + c, a.sdt, false, a.cols - c, v);
            if (!has_b) continue;
            post8(c, true, g, v);
            if (a.post)
#pragma unroll
                for (int k = 0; k < 8; ++k) g[k] = pr * (g[k] - d1 - v[k] * d2);
            store8(a.dbranch, row * a.ld_dbranch + c, a.dt, false, a.cols - c, g);
        }
    }
}

// The parameters' gradients from the partial rows' sums: 64 columns a workgroup,
// 4 a lane, 32 rows at once, joined in LDS (blockIdx.y 0: P and Q, 1: S and D).
constexpr int kJoinCols = 64;
constexpr int kJoinRows = kNT / (kJoinCols / 4);
__global__ __launch_bounds__(kNT) void blocknorm_join_kernel(BlockNormGradArgs a) {
    __shared__ __align__(16) float acc[2][kJoinRows][kJoinCols];
    const int cl = threadIdx.x % (kJoinCols / 4) * 4, pl = threadIdx.x / (kJoinCols / 4), y = blockIdx.y;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        const int at = a.at[2 * y + w], n = a.cols - int(blockIdx.x) * kJoinCols - cl;
        if (n > 0 && at >= 0) {
            const GMEM float* q = gm(a.partial) + int64_t(at) * a.parts * a.cols + blockIdx.x * kJoinCols + cl;
#pragma unroll 8
            for (int p = pl; p < a.parts; p += kJoinRows) {
                float t[4];
                run_decode<float, 4>(run_get<float, 4, false>(q + int64_t(p) * a.cols, n), t);
#pragma unroll
                for (int k = 0; k < 4; ++k) s[k] += t[k];
            }
        }
        *reinterpret_cast<f32x4_t*>(&acc[w][pl][cl]) = f32x4_t{s[0], s[1], s[2], s[3]};
    }
    __syncthreads();
    const int c = blockIdx.x * kJoinCols + threadIdx.x;
    if (threadIdx.x >= kJoinCols || c >= a.cols) return;
    float s = 0.f, d = 0.f;
#pragma unroll 8
    for (int p = 0; p < kJoinRows; ++p) {
        s += acc[0][p][threadIdx.x];
        d += acc[1][p][threadIdx.x];
    }
    auto put = [&](void* o, float v) {
        if (!o) return;
        if (a.accumulate) v += load1(o, c, a.pdt);
        store1(o, c, a.pdt, v);
    };
    if (y == 0) {
        put(a.dpre_gain, s);
        put(a.dpre_bias, d);
    } else {
        const float gate = a.gate ? load1(a.gate, c, a.pdt) : 1.f;
        if (a.dpost_gain) put(a.dpost_gain, a.beta * gate * s);
        if (a.dpost_bias) put(a.dpost_bias, a.beta * gate * d);
        if (a.dgate) {
            const float gain = a.post_gain ? load1(a.post_gain, c, a.pdt) : 1.f;
            put(a.dgate, a.beta * (a.post_bias ? fmaf(gain, s, load1(a.post_bias, c, a.pdt) * d) : gain * s));
        }
    }
}

// Two workgroups a CU, each a row of partial sums (8192 x 4096 bf16, RMS 88 us, layer
// norms 98; one 94 and 107; three 91 and 113); one where a float32 stream's layer norms take the registers of two.
constexpr int kMaxParts = 512;

bool layer_sums(const BlockNormGradArgs& a) {   // means, or sums that only layer norms have
    return a.post == NORM_LAYER || a.pre == NORM_LAYER || a.at[1] >= 0 || a.at[3] >= 0;
}

}  // namespace

int blocknorm_parts(const BlockNormGradArgs& a) {
    const int w = block_row_waves(a.cols);
    const int64_t rb = !block_row_fits(a.cols) ? 1 : block_waves(w) / w, n = (a.rows + rb - 1) / rb;
    const int most = a.sdt == 1 && layer_sums(a) ? kMaxParts / 2 : kMaxParts;
    return int(n < most ? n : most);
}

hipError_t launch_blocknorm_grad(const BlockNormGradArgs& a, hipStream_t s) {
    if (a.parts > 0) {
        const dim3 grid{unsigned(a.parts)}, block(kNT);
        const bool layer = layer_sums(a);
        if (!block_row_fits(a.cols)) {
            hipLaunchKernelGGL(blocknorm_grad_long_kernel, grid, block, 0, s, a);
        } else {
            pick_types(a.sdt, a.dt, [&](auto st, auto bt) {
                using ST = decltype(st);
                using BT = decltype(bt);
                pick_block_row(a.cols, [&](auto nw) {
                    constexpr int NW = decltype(nw)::value;
                    const dim3 block(block_waves(NW) * 64);
                    if (layer) hipLaunchKernelGGL((blocknorm_grad_kernel<ST, BT, NW, true>), grid, block, 0, s, a);
                    else hipLaunchKernelGGL((blocknorm_grad_kernel<ST, BT, NW, false>), grid, block, 0, s, a);
                });
            });
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const bool post = a.at[2] >= 0 || a.at[3] >= 0;
    if (a.sums == 0) return hipSuccess;
    hipLaunchKernelGGL(blocknorm_join_kernel, dim3(unsigned((a.cols + kJoinCols - 1) / kJoinCols), post ? 2u : 1u), dim3(kNT), 0,
                       s, a);
    return hipGetLastError();
}

}  // namespace muon
