// gfx950 kernels of the junction between two blocks, forward:
//
//   t = norm_post(branch) gain + bias           RMS or layer norm, or the branch itself
//   s = alpha x + beta gate drop(t)             rounded to the stream's type
//   y = norm_pre(s) gain + bias                 of s as rounded
//
// One pass over the rows, HBM bound: a row lies in the registers of NW waves, 8
// elements of every operand a lane.  Statistics and sums are float32.  Measured:
// 8191 x 2048, float32 stream, bf16 branch and y, RMS 40 us, 5.06 TB/s (a copy 5.1);
// 8192 x 4096 bf16 RMS 55, layer norms 75-76 (two exact passes over the registers: the
// instructions of a row are what bounds it).

#include "blocknorm_device.hpp"

namespace muon {
namespace {

// 8-bit copy of the lane's share of y: the lanes that hold a group of 32 columns
// agree on its magnitude.
template <class G, int E>
__device__ __forceinline__ void store_act8(const Act8View& q, int64_t row, int cols, int lane, bool on,
                                           const float (&v)[E]) {
    constexpr int V = G::V, GL = kAct8Group / V;
#pragma unroll
    for (int j = 0; j < G::C; ++j) {
        const int c = G::col(j, lane), n = on ? cols - c : 0;
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < V; ++k) m = max_mag(m, k < n ? v[j * V + k] : 0.f);
#pragma unroll
        for (int d = 1; d < GL; d *= 2) m = max_mag(m, __shfl_xor(m, d, 64));
        if (n <= 0) continue;
        const uint32_t e = act8_exp(m);
        GMEM int8_t* p = gm(q.codes) + row * q.ld + c;
        if (q.vec && n >= V) {
            u32x2_t w = {0u, 0u};
#pragma unroll
            for (int k = 0; k < V; ++k) w[k >> 2] |= act8_code(v[j * V + k], e) << (8 * (k & 3));
            if constexpr (V == 8) *reinterpret_cast<GMEM u32x2_t*>(p) = w;
            else *reinterpret_cast<GMEM uint32_t*>(p) = w[0];
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k)
                if (k < n) p[k] = int8_t(act8_code(v[j * V + k], e));
        }
        if ((c & (kAct8Group - 1)) == 0) gm(q.exps)[row * q.lde + c / kAct8Group] = uint8_t(e);
    }
}

// Columns that wave w of a row holds.
template <class G>
__device__ __forceinline__ float wave_columns(int cols, int w) {
    int n = 0;
#pragma unroll
    for (int j = 0; j < G::C; ++j) {
        const int left = cols - G::col(j, w * 64);
        n += left < 0 ? 0 : (left > 64 * G::V ? 64 * G::V : left);
    }
    return float(n);
}

// 1 / sqrt(v), within two units in the last place; what the hardware's would flush
// goes the long way.
__device__ __forceinline__ float inverse_root(float v) {
#ifdef __HIP__
    if (!(v < 1e-37f)) return __builtin_amdgcn_rsqf(v);
#endif
    return 1.f / __builtin_sqrtf(v);
}

// v -> its normalised row (columns past the end become 0); mean and 1 / root.  A
// layer norm's mean and centred squares are one exchange between the row's waves:
// each centres its own columns (inv_here: one over their number) twice (the mean of what is left
// corrects the mean, so that equal values leave nothing, whatever their sum's
// rounding), and the waves' are joined as those of separate samples, means as
// differences from the first wave's: M2 = sum of M2_w + n_w (mean_w - mean)^2.
template <class G, int NW, int E, bool LAYER>
__device__ __forceinline__ void normalise(float (&v)[E], int kind, float eps, float inv_n, float inv_here,
                                          int cols, int lane, RowSums<NW>& sums, float& mu, float& r) {
    mu = 0.f;
    float q[2] = {0.f, 0.f};
    if (LAYER && kind == NORM_LAYER) {
#pragma unroll
        for (int i = 0; i < E; ++i) q[1] += v[i];
        float part = wave_total(q[1]) * inv_here;
        q[1] = 0.f;
#pragma unroll
        for (int j = 0; j < G::C; ++j)
#pragma unroll
            for (int k = 0; k < G::V; ++k) {
                const float t = G::col(j, lane) + k < cols ? v[j * G::V + k] - part : 0.f;
                q[0] = fmaf(t, t, q[0]);
                q[1] += t;
            }
        q[0] = wave_total(q[0]);
        q[1] = wave_total(q[1]);
        const float fix = q[1] * inv_here;
        part += fix;
        q[0] = fmaf(-fix, q[1], q[0]);
        q[0] = q[0] < 0.f ? 0.f : q[0];          // (a NaN stays one)
        if constexpr (NW > 1) {
            float w[2] = {q[0], part}, ref;
            sums.exchange(w, &ref);
            // lane i has wave i mod NW's squares and mean; its count from its place
            const float nw = wave_columns<G>(cols, int(threadIdx.x % NW));
            const float d = nw > 0.f ? w[1] - ref : 0.f, md = turn_total<NW>(nw * d) * inv_n, e = nw > 0.f ? d - md : 0.f;
            mu = ref + md;
            q[0] = turn_total<NW>(fmaf(nw * e, e, w[0]));
        } else {
            mu = part;
        }
#pragma unroll
        for (int j = 0; j < G::C; ++j)
#pragma unroll
            for (int k = 0; k < G::V; ++k) {
                float& t = v[j * G::V + k];
                t = G::col(j, lane) + k < cols ? t - mu : 0.f;
            }
    } else {
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < E; ++i) s[0] = fmaf(v[i], v[i], s[0]);
        sums(s);
        q[0] = s[0];
    }
    r = inverse_root(fmaf(q[0], inv_n, eps));
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] *= r;
}

// LAYER: one of the norms is a layer norm (means and biases).
template <class ST, class BT, int NW, bool LAYER>
__global__ __launch_bounds__(block_waves(NW) * 64, LAYER && sizeof(BT) == 4 && NW < 16 ? 2 : 4) void blocknorm_kernel(BlockNormArgs a) {
    constexpr int E = kRowElems, RB = block_waves(NW) / NW;
    using G = BlockRow<run_width<ST, BT>(), NW, E>;
    __shared__ float red[2][2][block_waves(NW)];
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6)), rg = wave / NW;   // (rows are scalar)
    const int lane = wave % NW * 64 + int(threadIdx.x & 63);
    const Philox m(a.drop);
    const float inv_n = 1.f / float(a.cols);
    const int64_t step = int64_t(gridDim.x) * RB;
    // two rows' loads are in flight under a third's arithmetic (the first two before
    // the parameters': a call of few rows waits once for all of them)
    typename G::template Raw<ST> rx[2];
    typename G::template Raw<BT> ro[2];
    int64_t r0 = int64_t(blockIdx.x) * RB;
    auto load = [&](int64_t row, typename G::template Raw<ST>& x, typename G::template Raw<BT>& o) {
        G::template load<ST, false>(a.x, row * a.ld_x, a.cols, lane, row < a.rows, x);
        if (a.branch) G::template load<BT, false>(a.branch, row * a.ld_branch, a.cols, lane, row < a.rows, o);
    };
    load(r0 + rg, rx[0], ro[0]);
    load(r0 + rg + step, rx[1], ro[1]);
    // post: the branch's factors and, with layer norm, addends, gate and scale folded in
    float wp[E], bp[LAYER ? E : 1], wn[E], bn[LAYER ? E : 1];
    if (a.branch) {
        G::param(a.post_gain, a.pdt, a.cols, lane, 1.f, wp);
        if (a.gate) {
            float g[E];
            G::param(a.gate, a.pdt, a.cols, lane, 1.f, g);
#pragma unroll
            for (int i = 0; i < E; ++i) wp[i] *= g[i];
            if constexpr (LAYER) {
                G::param(a.post_bias, a.pdt, a.cols, lane, 0.f, bp);
#pragma unroll
                for (int i = 0; i < E; ++i) bp[i] *= g[i];
            }
        } else if constexpr (LAYER) {
            G::param(a.post_bias, a.pdt, a.cols, lane, 0.f, bp);
        }
#pragma unroll
        for (int i = 0; i < E; ++i) {
            wp[i] *= a.beta;
            if constexpr (LAYER) bp[i] *= a.beta;
        }
    }
    G::param(a.pre_gain, a.pdt, a.cols, lane, 1.f, wn);
    if constexpr (LAYER) G::param(a.pre_bias, a.pdt, a.cols, lane, 0.f, bn);
    RowSums<NW> sums{red, wave};
    const float here = wave_columns<G>(a.cols, wave % NW), inv_here = here > 0.f ? 1.f / here : 0.f;
    auto one = [&](int64_t row, typename G::template Raw<ST>& x, typename G::template Raw<BT>& o) {
        const bool on = row < a.rows;
        float v[E], t[E], mu, r;
        G::decode(x, a.cols, lane, v);
        if (a.branch) G::decode(o, a.cols, lane, t);
        load(row + 2 * step, x, o);
        if (a.branch) {
            if (a.post) {
                normalise<G, NW, E, LAYER>(t, a.post, a.post_eps, inv_n, inv_here, a.cols, lane, sums, mu, r);
                if (on && lane == 0) {
                    if (a.post_mean) gm(a.post_mean)[row] = mu;
                    if (a.post_rstd) gm(a.post_rstd)[row] = r;
                }
            }
#pragma unroll
            for (int i = 0; i < E; ++i) {
                if constexpr (LAYER) t[i] = fmaf(t[i], wp[i], bp[i]);
                else t[i] *= wp[i];
            }
            if (m.cut) G::mask(m, uint32_t(row), lane, t);
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] = fmaf(a.alpha, v[i], t[i]);
            typename G::template Raw<ST> rs;
            G::encode(v, rs);
            if (on) G::template store<ST, false>(a.s, row * a.ld_s, a.cols, lane, rs);
            G::decode(rs, v);
        }
        if (!a.pre) return;
        normalise<G, NW, E, LAYER>(v, a.pre, a.pre_eps, inv_n, inv_here, a.cols, lane, sums, mu, r);
        if (on && lane == 0) {
            if (a.pre_mean) gm(a.pre_mean)[row] = mu;
            if (a.pre_rstd) gm(a.pre_rstd)[row] = r;
        }
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if constexpr (LAYER) v[i] = fmaf(v[i], wn[i], bn[i]);
            else v[i] *= wn[i];
        }
        typename G::template Raw<BT> ry;
        G::encode(v, ry);
        if (on) G::template store<BT, false>(a.y, row * a.ld_y, a.cols, lane, ry);
        if (a.y8.codes) store_act8<G, E>(a.y8, row, a.cols, lane, on, v);
    };
    for (; r0 < a.rows; r0 += 2 * step) {
        one(r0 + rg, rx[0], ro[0]);
        if (r0 + step < a.rows) one(r0 + step + rg, rx[1], ro[1]);
    }
}

// Rows longer than the registers hold, or shorter than a run: a workgroup walks rows, 8 columns a lane
// at a time, and passes over each as often as it needs (from the caches), element by
// element: far from its bytes (4096 x 12288 bf16, RMS 563 us, layer norms 656, where the
// bytes take 79; 65536 x 4, bound by the barriers of a row, 970).
__global__ __launch_bounds__(kNT) void blocknorm_long_kernel(BlockNormArgs a) {
    __shared__ float red[kWaves];
    const Philox m(a.drop);
    const float n = float(a.cols);
    auto stats = [&](const void* p, int64_t base, int dt, int kind, float eps, float& mu, float& r) {
        mu = 0.f;
        float v[8];
        if (kind == NORM_LAYER) {
            float s = 0.f;
            for (int c = threadIdx.x * 8; c < a.cols; c += kNT * 8) {
                get8(p, base + c, dt, a.cols - c, v);
#pragma unroll
                for (int k = 0; k < 8; ++k) s += v[k];
            }
            mu = block_add(s, red) / n;
        }
        float q = 0.f, left = 0.f;
        for (int c = threadIdx.x * 8; c < a.cols; c += kNT * 8) {
            get8(p, base + c, dt, a.cols - c, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float t = c + k < a.cols ? v[k] - mu : 0.f;
                q = fmaf(t, t, q);
                left += t;
            }
        }
        q = block_add(q, red);
        if (kind == NORM_LAYER) {        // the mean of what is left corrects the mean, as in normalise()
            left = block_add(left, red);
            const float fix = left / n;
            mu += fix;
            q = fmaf(-fix, left, q);
            q = q < 0.f ? 0.f : q;
        }
        r = 1.f / __builtin_sqrtf(q / n + eps);
    };
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        if (a.branch) {
            float mu = 0.f, r = 1.f;
            if (a.post) stats(a.branch, row * a.ld_branch, a.dt, a.post, a.post_eps, mu, r);
            if (a.post && threadIdx.x == 0) {
                if (a.post_mean) gm(a.post_mean)[row] = mu;
                if (a.post_rstd) gm(a.post_rstd)[row] = r;
            }
            for (int c = threadIdx.x * 8; c < a.cols; c += kNT * 8) {
                const int nv = a.cols - c;
                float t[8], w[8], b[8], g[8], x[8];
                get8(a.branch, row * a.ld_branch + c, a.dt, nv, t);
                par8(a.post_gain, c, a.pdt, nv, 1.f, w);
                par8(a.post_bias, c, a.pdt, nv, 0.f, b);
                par8(a.gate, c, a.pdt, nv, 1.f, g);
                get8(a.x, row * a.ld_x + c, a.sdt, nv, x);
#pragma unroll
                for (int k = 0; k < 8; ++k) t[k] = fmaf((t[k] - mu) * r, w[k], b[k]) * (g[k] * a.beta);
                if (m.cut) m.run<8>(uint32_t(row), uint32_t(c), t);
#pragma unroll
                for (int k = 0; k < 8; ++k) t[k] = fmaf(a.alpha, x[k], t[k]);
                store8(a.s, row * a.ld_s + c, a.sdt, false, nv, t);
            }
        }
        if (!a.pre) continue;
        // a lane reads back what it wrote itself
        const void* sp = a.branch ? a.s : a.x;
        const int64_t base = row * (a.branch ? a.ld_s : a.ld_x);
        float mu, r;
        stats(sp, base, a.sdt, a.pre, a.pre_eps, mu, r);
        if (threadIdx.x == 0) {
            if (a.pre_mean) gm(a.pre_mean)[row] = mu;
            if (a.pre_rstd) gm(a.pre_rstd)[row] = r;
        }
        for (int c0 = 0; c0 < a.cols; c0 += kNT * 8) {   // every lane runs every step: groups of 32 columns agree below
            const int c = c0 + threadIdx.x * 8, nv = a.cols - c;
            float v[8], w[8], b[8];
            get8(sp, base + c, a.sdt, nv, v);
            par8(a.pre_gain, c, a.pdt, nv, 1.f, w);
            par8(a.pre_bias, c, a.pdt, nv, 0.f, b);
            float mag = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                v[k] = fmaf((v[k] - mu) * r, w[k], b[k]);
                mag = max_mag(mag, k < nv ? v[k] : 0.f);
            }
            if (nv > 0) store8(a.y, row * a.ld_y + c, a.dt, false, nv, v);
            if (!a.y8.codes) continue;
            mag = max_mag(mag, __shfl_xor(mag, 1, 64));
            mag = max_mag(mag, __shfl_xor(mag, 2, 64));
            if (nv <= 0) continue;
            const uint32_t e = act8_exp(mag);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < nv) gm(a.y8.codes)[row * a.y8.ld + c + k] = int8_t(act8_code(v[k], e));
            if (c % kAct8Group == 0) gm(a.y8.exps)[row * a.y8.lde + c / kAct8Group] = uint8_t(e);
        }
    }
}

// Two workgroups a CU (8192 x 4096 bf16, RMS norms on both sides, of an earlier
// form of the kernel: 58.9 us; three 61.6, four 74).
constexpr int kMaxBlocks = 512;
constexpr int kMaxLongBlocks = 1024;

}  // namespace

hipError_t launch_blocknorm(const BlockNormArgs& a, hipStream_t s) {
    if (a.rows <= 0) return hipSuccess;
    if (!block_row_fits(a.cols)) {
        const int64_t nb = a.rows < kMaxLongBlocks ? a.rows : kMaxLongBlocks;
        hipLaunchKernelGGL(blocknorm_long_kernel, dim3(unsigned(nb)), dim3(kNT), 0, s, a);
        return hipGetLastError();
    }
    const bool layer = a.post == NORM_LAYER || a.pre == NORM_LAYER;
    pick_types(a.sdt, a.dt, [&](auto st, auto bt) {
        using ST = decltype(st);
        using BT = decltype(bt);
        pick_block_row(a.cols, [&](auto nw) {
            constexpr int NW = decltype(nw)::value, RB = block_waves(NW) / NW;
            const int64_t nb = (a.rows + RB - 1) / RB;
            const dim3 grid(unsigned(nb < kMaxBlocks ? nb : kMaxBlocks)), block(block_waves(NW) * 64);
            if (layer) hipLaunchKernelGGL((blocknorm_kernel<ST, BT, NW, true>), grid, block, 0, s, a);
            else hipLaunchKernelGGL((blocknorm_kernel<ST, BT, NW, false>), grid, block, 0, s, a);
        });
    });
    return hipGetLastError();
}

}  // namespace muon
