// gfx950 kernels of layer norm (forward, backward, the reduction of the gain's
// and bias' gradients) and of the 8-bit activation checkpoints.
//
//   forward   mu = mean x, r = 1 / sqrt(mean (x - mu)^2 + eps), y = (x - mu) r g + b
//   backward  xh = (x - mu) r, a = dy g,
//             dx = r (a - mean a - xh mean(a xh)) [+ add]
//             dg = sum over rows of dy xh,  db = sum over rows of dy
//
// All of them stream rows once: HBM bound.  A row lies in the registers of NW
// waves (E elements a lane, in 16-byte runs), so both passes over it (mean,
// then centred squares; the two row sums, then dx) read it from memory once.
// That holds to 8192 columns.  With 32 elements a lane (to 16384) the backward
// kernel spills 283-566 VGPRs to scratch, the forward one without 16-byte
// vectors 80: 4096 x 12288 bf16 backward with an added gradient 182 us where its
// bytes take 78, 4096 x 8192 67 where they take 52.
// Statistics and sums are float32.

#include "norm_device.hpp"

namespace muon {
namespace {

template <class T, bool VEC, int NW, int E, bool STREAM>
__global__ __launch_bounds__(kNT) void norm_kernel(NormArgs a) {
    using G = RowGeom<T, VEC, NW, E>;
    constexpr int RB = kWaves / NW;      // rows a workgroup works on at once
    __shared__ float red[2][kWaves][2];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x % G::LANES, rg = wave / NW;
    float g[E], b[E];
    param_load<T, VEC, NW, E>(a.gain, a.pdt, a.pvec, a.cols, lane, g);
    if (a.bias) param_load<T, VEC, NW, E>(a.bias, a.pdt, a.pvec, a.cols, lane, b);
    const float n = float(a.cols);   // divided by: the mean of equal values is exact
    const int64_t step = int64_t(gridDim.x) * RB;
    RowRaw<T, VEC, NW, E> raw;
    int64_t r0 = int64_t(blockIdx.x) * RB;
    if (r0 < a.rows) row_load<T, VEC, NW, E>(a.x, (r0 + rg) * a.ld_x, a.cols, lane, r0 + rg < a.rows, raw);
    for (; r0 < a.rows; r0 += step) {
        const int64_t row = r0 + rg;
        const bool on = row < a.rows;
        float v[E];
        row_decode<T, VEC, NW, E>(raw, v);
        const int64_t nr = row + step;   // the next row's loads run under this one's arithmetic
        row_load<T, VEC, NW, E>(a.x, nr * a.ld_x, a.cols, lane, nr < a.rows, raw);
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < E; ++i) s[0] += v[i];
        row_sum<NW, 1>(s, red[0], wave);
        const float mu = s[0] / n;
        float q[1] = {0.f};
#pragma unroll
        for (int j = 0; j < G::C; ++j) {
            const bool in = G::col(j, lane) < a.cols;
#pragma unroll
            for (int k = 0; k < G::V; ++k) {
                float& t = v[j * G::V + k];
                t = in ? t - mu : 0.f;
                q[0] = fmaf(t, t, q[0]);
            }
        }
        row_sum<NW, 1>(q, red[1], wave);
        const float r = 1.f / __builtin_sqrtf(q[0] / n + a.eps);
        if (on && lane == 0) {
            if (a.mean) gm(a.mean)[row] = mu;
            if (a.rstd) gm(a.rstd)[row] = r;
        }
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = a.bias ? fmaf(v[i] * r, g[i], b[i]) : v[i] * r * g[i];
        if (on) row_store<T, VEC, NW, E, STREAM>(a.y, row * a.ld_y, a.cols, lane, v);
        if (a.y8.codes) row_store_act8<T, VEC, NW, E>(a.y8, row, a.cols, lane, on, v);
    }
}

// Rows longer than the registers hold: one workgroup per row, three passes
// over it (the second and third read it from the caches).
__global__ __launch_bounds__(kNT) void norm_long_kernel(NormArgs a) {
    __shared__ float red[kWaves];
    const int64_t row = blockIdx.x;
    const float n = float(a.cols);   // divided by: the mean of equal values is exact
    float s = 0.f;
    for (int c = threadIdx.x; c < a.cols; c += kNT) s += load1(a.x, row * a.ld_x + c, a.dt);
    const float mu = block_add(s, red) / n;
    float q = 0.f;
    for (int c = threadIdx.x; c < a.cols; c += kNT) {
        const float t = load1(a.x, row * a.ld_x + c, a.dt) - mu;
        q = fmaf(t, t, q);
    }
    const float r = 1.f / __builtin_sqrtf(block_add(q, red) / n + a.eps);
    if (threadIdx.x == 0) {
        if (a.mean) gm(a.mean)[row] = mu;
        if (a.rstd) gm(a.rstd)[row] = r;
    }
    for (int c0 = 0; c0 < a.cols; c0 += kNT) {   // every lane runs every step: groups of 32 lanes agree below
        const int c = c0 + threadIdx.x;
        const bool in = c < a.cols;
        float y = 0.f;
        if (in) {
            y = (load1(a.x, row * a.ld_x + c, a.dt) - mu) * r * load1(a.gain, c, a.pdt);
            if (a.bias) y += load1(a.bias, c, a.pdt);
            store1(a.y, row * a.ld_y + c, a.dt, y);
        }
        if (a.y8.codes) {
            float m = max_mag(y, 0.f);
#pragma unroll
            for (int d = 1; d < kAct8Group; d *= 2) m = max_mag(m, __shfl_xor(m, d, 64));
            if (in) {
                const uint32_t e = act8_exp(m);
                gm(a.y8.codes)[row * a.y8.ld + c] = int8_t(act8_code(y, e));
                if (c % kAct8Group == 0) gm(a.y8.exps)[row * a.y8.lde + c / kAct8Group] = uint8_t(e);
            }
        }
    }
}

// Backward.  A workgroup walks rows with a stride of the grid and keeps, per
// lane, the running sums of dy xh and dy of its columns; at the end it adds the
// sums of its row groups in LDS and writes one row of partial sums.  A second
// kernel adds the partial rows in a fixed order.  Few workgroups (one a CU): each
// costs a row of partial sums written and read again.
template <class T, bool VEC, int NW, int E>
__global__ __launch_bounds__(kNT) void norm_grad_kernel(NormGradArgs a) {
    using G = RowGeom<T, VEC, NW, E>;
    constexpr int RB = kWaves / NW;
    __shared__ float red[2][kWaves][2];
    __shared__ float cs[RB > 1 ? 2 * kNT * E : 1];   // [row group][sum][element][lane]
    const int wave = threadIdx.x >> 6, lane = threadIdx.x % G::LANES, rg = wave / NW;
    float g[E], dg[E], db[E];
    param_load<T, VEC, NW, E>(a.gain, a.pdt, a.pvec, a.cols, lane, g);
#pragma unroll
    for (int i = 0; i < E; ++i) dg[i] = db[i] = 0.f;
    const float n = float(a.cols);   // divided by: the mean of equal values is exact
    const int64_t step = int64_t(gridDim.x) * RB;
    RowRaw<T, VEC, NW, E> rx, ry, ra;
    int64_t r0 = int64_t(blockIdx.x) * RB;
    if (r0 < a.rows) {
        row_load<T, VEC, NW, E, true>(a.x, (r0 + rg) * a.ld_x, a.cols, lane, r0 + rg < a.rows, rx);
        row_load<T, VEC, NW, E, true>(a.dy, (r0 + rg) * a.ld_dy, a.cols, lane, r0 + rg < a.rows, ry);
        if (a.add) row_load<T, VEC, NW, E, true>(a.add, (r0 + rg) * a.ld_add, a.cols, lane, r0 + rg < a.rows, ra);
    }
    int half = 0;
    for (; r0 < a.rows; r0 += step, half ^= 1) {
        const int64_t row = r0 + rg;
        const bool on = row < a.rows;
        const float mu = on ? gm(a.mean)[row] : 0.f, r = on ? gm(a.rstd)[row] : 0.f;
        float xh[E], y[E];
        row_decode<T, VEC, NW, E>(rx, xh);
        row_decode<T, VEC, NW, E>(ry, y);
        const int64_t nr = row + step;
        row_load<T, VEC, NW, E, true>(a.x, nr * a.ld_x, a.cols, lane, nr < a.rows, rx);
        row_load<T, VEC, NW, E, true>(a.dy, nr * a.ld_dy, a.cols, lane, nr < a.rows, ry);
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < E; ++i) {
            // past the last column dy, g are 0, so xh there adds nothing
            xh[i] = (xh[i] - mu) * r;
            dg[i] = fmaf(y[i], xh[i], dg[i]);
            db[i] += y[i];
            y[i] *= g[i];
            s[0] += y[i];
            s[1] = fmaf(y[i], xh[i], s[1]);
        }
        row_sum<NW, 2>(s, red[half], wave);
        const float c1 = s[0] / n, c2 = s[1] / n;
#pragma unroll
        for (int i = 0; i < E; ++i) y[i] = r * (y[i] - c1 - xh[i] * c2);
        if (a.add) {
            row_decode<T, VEC, NW, E>(ra, xh);
#pragma unroll
            for (int i = 0; i < E; ++i) y[i] += xh[i];
            // (add may be dx: another row's, not yet written)
            row_load<T, VEC, NW, E, true>(a.add, nr * a.ld_add, a.cols, lane, nr < a.rows, ra);
        }
        if (on) row_store<T, VEC, NW, E>(a.dx, row * a.ld_dx, a.cols, lane, y);
    }
    GMEM float* pg = gm(a.partial) + int64_t(blockIdx.x) * a.cols;
    GMEM float* pb = pg + int64_t(a.parts) * a.cols;
    if constexpr (RB > 1) {
        // every row group's sums through LDS, each thread adding its share of the columns
        constexpr int kOne = G::LANES * E;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            cs[(rg * 2 * E + i) * G::LANES + lane] = dg[i];
            cs[((rg * 2 + 1) * E + i) * G::LANES + lane] = db[i];
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < 2 * kOne / kNT; ++q) {
            const int at = q * kNT + threadIdx.x, w = at / kOne, i = at % kOne / G::LANES, l = at % G::LANES;
            float v = 0.f;
#pragma unroll
            for (int r = 0; r < RB; ++r) v += cs[r * 2 * kOne + at];
            const int c = G::col(i / G::V, l) + i % G::V;
            if (c < a.cols) (w ? pb : pg)[c] = v;
        }
    } else {
#pragma unroll
        for (int j = 0; j < G::C; ++j) {
            const int c = G::col(j, lane);
            if (c >= a.cols) continue;
            if constexpr (VEC) {         // cols is a multiple of V: 16-byte aligned rows
#pragma unroll
                for (int k = 0; k < G::V; k += 4) {
                    const float* x = dg + j * G::V + k;
                    const float* y = db + j * G::V + k;
                    *reinterpret_cast<GMEM f32x4_t*>(pg + c + k) = f32x4_t{x[0], x[1], x[2], x[3]};
                    *reinterpret_cast<GMEM f32x4_t*>(pb + c + k) = f32x4_t{y[0], y[1], y[2], y[3]};
                }
            } else {
                pg[c] = dg[j];
                pb[c] = db[j];
            }
        }
    }
}

// Long rows: dx row by row, the column sums in a kernel of their own.
__global__ __launch_bounds__(kNT) void norm_grad_long_kernel(NormGradArgs a) {
    __shared__ float red[kWaves];
    const int64_t row = blockIdx.x;
    const float n = float(a.cols), mu = gm(a.mean)[row], r = gm(a.rstd)[row];
    float s0 = 0.f, s1 = 0.f;
    for (int c = threadIdx.x; c < a.cols; c += kNT) {
        const float t = load1(a.dy, row * a.ld_dy + c, a.dt) * load1(a.gain, c, a.pdt);
        s0 += t;
        s1 = fmaf(t, (load1(a.x, row * a.ld_x + c, a.dt) - mu) * r, s1);
    }
    const float c1 = block_add(s0, red) / n, c2 = block_add(s1, red) / n;
    for (int c = threadIdx.x; c < a.cols; c += kNT) {
        const float t = load1(a.dy, row * a.ld_dy + c, a.dt) * load1(a.gain, c, a.pdt);
        const float xh = (load1(a.x, row * a.ld_x + c, a.dt) - mu) * r;
        float d = r * (t - c1 - xh * c2);
        if (a.add) d += load1(a.add, row * a.ld_add + c, a.dt);
        store1(a.dx, row * a.ld_dx + c, a.dt, d);
    }
}
__global__ __launch_bounds__(kNT) void norm_grad_cols_kernel(NormGradArgs a, int col_blocks) {
    const int part = blockIdx.x / col_blocks, c = (blockIdx.x % col_blocks) * kNT + threadIdx.x;
    if (c >= a.cols) return;
    float dg = 0.f, db = 0.f;
    for (int64_t r = part; r < a.rows; r += a.parts) {
        const float y = load1(a.dy, r * a.ld_dy + c, a.dt);
        dg = fmaf(y, (load1(a.x, r * a.ld_x + c, a.dt) - gm(a.mean)[r]) * gm(a.rstd)[r], dg);
        db += y;
    }
    gm(a.partial)[int64_t(part) * a.cols + c] = dg;
    gm(a.partial)[(int64_t(a.parts) + part) * a.cols + c] = db;
}

// dgain / dbias = the partial rows' sums: 16 columns a workgroup, 32 rows at
// once, joined in LDS (blockIdx.y: gain, bias).
constexpr int kRedCols = 16;
__global__ __launch_bounds__(kNT) void norm_grad_join_kernel(NormGradArgs a) {
    __shared__ float acc[kNT];
    const int cl = threadIdx.x % kRedCols, pl = threadIdx.x / kRedCols;
    const int c = blockIdx.x * kRedCols + cl;
    const int which = blockIdx.y;
    float s = 0.f;
    if (c < a.cols) {
        const GMEM float* q = gm(a.partial) + int64_t(which) * a.parts * a.cols + c;
#pragma unroll 8
        for (int p = pl; p < a.parts; p += kNT / kRedCols) s += q[int64_t(p) * a.cols];
    }
    acc[threadIdx.x] = s;
    __syncthreads();
    if (pl != 0 || c >= a.cols) return;
    s = 0.f;
    for (int p = 0; p < kNT / kRedCols; ++p) s += acc[p * kRedCols + cl];
    void* o = which ? a.dbias : a.dgain;
    if (!o) return;
    if (a.accumulate) s += load1(o, c, a.pdt);
    store1(o, c, a.pdt, s);
}

// ---- 8-bit checkpoints: 8 elements a lane, 4 lanes a group ----
// A workgroup takes RPB rows of `slots` 8-element runs each (padded to whole
// groups).  HBM bound: 16384 x 4096 bf16 encoded and decoded in 81 us, 406 MB at
// 5.0 TB/s.
__global__ __launch_bounds__(256) void act8_encode_kernel(Act8Args a, int rpb, int slots) {
    const int64_t r0 = int64_t(blockIdx.x) * rpb;
    const int n = rpb * slots;           // multiple of 4; every lane of a group runs the same steps
    for (int i = threadIdx.x; i < n; i += 256) {
        const int rl = i / slots, c = (i - rl * slots) * 8;
        const int64_t row = r0 + rl;
        const int nv = row < a.rows ? a.cols - c : 0;
        float v[8];
        load8(a.x, row * a.ld + c, a.dt, a.vec, nv, v);
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) m = max_mag(m, v[k]);
        m = max_mag(m, __shfl_xor(m, 1, 64));
        m = max_mag(m, __shfl_xor(m, 2, 64));
        if (nv <= 0) continue;
        const uint32_t e = act8_exp(m);
        GMEM int8_t* p = gm(a.q.codes) + row * a.q.ld + c;
        if (a.vec && nv >= 8) {
            u32x2_t w = {0u, 0u};
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k >> 2] |= act8_code(v[k], e) << (8 * (k & 3));
            *reinterpret_cast<GMEM u32x2_t*>(p) = w;
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < nv) p[k] = int8_t(act8_code(v[k], e));
        }
        if (c % kAct8Group == 0) gm(a.q.exps)[row * a.q.lde + c / kAct8Group] = uint8_t(e);
    }
}

__global__ __launch_bounds__(256) void act8_decode_kernel(Act8Args a, int rpb, int slots) {
    const int64_t r0 = int64_t(blockIdx.x) * rpb;
    const int n = rpb * slots;
    for (int i = threadIdx.x; i < n; i += 256) {
        const int rl = i / slots, c = (i - rl * slots) * 8;
        const int64_t row = r0 + rl;
        const int nv = a.cols - c;
        if (row >= a.rows || nv <= 0) continue;
        const float step = act8_step(gm(a.q.exps)[row * a.q.lde + c / kAct8Group]);
        const GMEM int8_t* p = gm(a.q.codes) + row * a.q.ld + c;
        float v[8];
        if (a.vec && nv >= 8) {
            const u32x2_t w = *reinterpret_cast<const GMEM u32x2_t*>(p);
            act8_dec4(w[0], step, v);
            act8_dec4(w[1], step, v + 4);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = k < nv ? float(p[k]) * step : 0.f;
        }
        store8(a.y, row * a.ld + c, a.dt, a.vec, nv, v);
    }
}

// The widest row each variant holds: NW waves x 64 lanes x E elements.
template <class F>
bool pick_row(int cols, F&& f) {
    if (cols <= 512) f(std::integral_constant<int, 1>{}, std::integral_constant<int, 8>{});
    else if (cols <= 1024) f(std::integral_constant<int, 1>{}, std::integral_constant<int, 16>{});
    else if (cols <= 2048) f(std::integral_constant<int, 2>{}, std::integral_constant<int, 16>{});
    else if (cols <= 4096) f(std::integral_constant<int, 4>{}, std::integral_constant<int, 16>{});
    else if (cols <= 8192) f(std::integral_constant<int, 8>{}, std::integral_constant<int, 16>{});
    else if (cols <= 16384) f(std::integral_constant<int, 8>{}, std::integral_constant<int, 32>{});
    else return false;
    return true;
}
int row_waves(int cols) { return cols <= 1024 ? 1 : cols <= 2048 ? 2 : cols <= 4096 ? 4 : 8; }

// Forward: two workgroups a CU (8192 x 4096 bf16 27.5 us, kept stores; four a CU 29.4).
// Backward: one (45.8 us; half as many 64.5, half as many again 58).
constexpr int kMaxFwdBlocks = 512;
constexpr int kMaxGradParts = 256;

}  // namespace

int norm_grad_parts(int64_t rows, int cols) {
    if (cols > 16384) return int(rows < 64 ? rows : 64);
    const int64_t rb = kWaves / row_waves(cols);
    const int64_t n = (rows + rb - 1) / rb;
    return int(n < kMaxGradParts ? n : kMaxGradParts);
}

// The looping kernels of rows past 16384 columns take one workgroup a row (so
// many would be more than 275 GB).
bool norm_rows_fit(int64_t rows, int64_t cols) { return cols <= 16384 || rows < kGridThreads / kNT; }

hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
    if (a.rows <= 0) return hipSuccess;
    // y is stored past the caches where the L2s (32 MiB) cannot hold it for its
    // reader anyway; it need then not be written back at the kernel's end: 8191 x
    // 2048 float32 27.2 -> 25.1 us, 8192 x 4096 bf16 26.5 -> 25.6, and with the
    // product that reads it (4096 -> 4096) 227 both ways.  Under that the product
    // finds y in the caches, which is worth more than the norm itself gains: 2048 x
    // 768 with 768 -> 768 13.6 us kept and 14.3 streamed (the norm alone 4.9, 4.8),
    // 4096 x 1024 with 1024 -> 4096 40.7 and 41.3 (6.7, 6.0).
    const bool stream = a.rows * a.cols * (a.dt == 0 ? 2 : 4) > (32ll << 20);
    const bool reg = pick_row(a.cols, [&](auto nw, auto e) {
        constexpr int NW = decltype(nw)::value, E = decltype(e)::value;
        constexpr int RB = kWaves / NW;
        const int64_t nb = (a.rows + RB - 1) / RB;
        const dim3 grid(unsigned(nb < kMaxFwdBlocks ? nb : kMaxFwdBlocks)), block(kNT);
        auto go = [&](auto zero) {
            using T = decltype(zero);
            if (!a.vec) hipLaunchKernelGGL((norm_kernel<T, false, NW, E, false>), grid, block, 0, s, a);
            else if (stream) hipLaunchKernelGGL((norm_kernel<T, true, NW, E, true>), grid, block, 0, s, a);
            else hipLaunchKernelGGL((norm_kernel<T, true, NW, E, false>), grid, block, 0, s, a);
        };
        if (a.dt == 0) go(uint16_t{});
        else go(float{});
    });
    if (!reg) hipLaunchKernelGGL(norm_long_kernel, dim3(unsigned(a.rows)), dim3(kNT), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t s) {
    if (a.parts > 0) {
        const bool reg = pick_row(a.cols, [&](auto nw, auto e) {
            constexpr int NW = decltype(nw)::value, E = decltype(e)::value;
            const dim3 grid{unsigned(a.parts)}, block(kNT);
            if (a.dt == 0) {
                if (a.vec) hipLaunchKernelGGL((norm_grad_kernel<uint16_t, true, NW, E>), grid, block, 0, s, a);
                else hipLaunchKernelGGL((norm_grad_kernel<uint16_t, false, NW, E>), grid, block, 0, s, a);
            } else {
                if (a.vec) hipLaunchKernelGGL((norm_grad_kernel<float, true, NW, E>), grid, block, 0, s, a);
                else hipLaunchKernelGGL((norm_grad_kernel<float, false, NW, E>), grid, block, 0, s, a);
            }
        });
        if (!reg) {
            // the sums first: dx may lie where add does, and neither is read by them
            const int cb = (a.cols + kNT - 1) / kNT;
            hipLaunchKernelGGL(norm_grad_cols_kernel, dim3(unsigned(cb) * unsigned(a.parts)), dim3(kNT), 0, s, a, cb);
            hipLaunchKernelGGL(norm_grad_long_kernel, dim3(unsigned(a.rows)), dim3(kNT), 0, s, a);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(norm_grad_join_kernel, dim3(unsigned((a.cols + kRedCols - 1) / kRedCols), a.dbias ? 2u : 1u),
                       dim3(kNT), 0, s, a);
    return hipGetLastError();
}

namespace {

// One launch, or more past 2^31 threads, each of whole workgroups' rows.
template <class K>
hipError_t launch_act8(const Act8Args& a, K* kernel, hipStream_t s) {
    const int slots = (a.cols + kAct8Group - 1) / kAct8Group * (kAct8Group / 8);
    const int rpb = slots >= 1024 ? 1 : 1024 / slots;
    const int64_t slice = (kSliceThreads + 255) / 256 * rpb, es = a.dt == 0 ? 2 : 4;
    for (int64_t r0 = 0; r0 < a.rows; r0 += slice) {
        Act8Args b = a;
        b.rows = a.rows - r0 < slice ? a.rows - r0 : slice;
        if (a.x) b.x = static_cast<const char*>(a.x) + r0 * a.ld * es;
        if (a.y) b.y = static_cast<char*>(a.y) + r0 * a.ld * es;
        b.q.codes += r0 * a.q.ld;
        b.q.exps += r0 * a.q.lde;
        hipLaunchKernelGGL(kernel, dim3(unsigned((b.rows + rpb - 1) / rpb)), dim3(256), 0, s, b, rpb, slots);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_act8_encode(const Act8Args& a, hipStream_t s) { return launch_act8(a, act8_encode_kernel, s); }
hipError_t launch_act8_decode(const Act8Args& a, hipStream_t s) { return launch_act8(a, act8_decode_kernel, s); }

}  // namespace muon
