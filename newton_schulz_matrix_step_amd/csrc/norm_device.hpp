// Rows of a matrix in the registers of a workgroup's waves: loads, stores, row
// sums.  Shared by the layer norm's kernels (norm_kernels.hip) and the block
// norms' (blocknorm_kernels.hip).
#pragma once

#include <type_traits>

#include "layer_device.hpp"

namespace muon {
namespace {

using namespace layer;

constexpr int kNT = 512;                 // threads of a workgroup: 8 waves
constexpr int kWaves = kNT / 64;

template <class T>
struct Elem;
template <>
struct Elem<uint16_t> {
    static constexpr int dt = 0, V = 8;  // elements of a 16-byte run
};
template <>
struct Elem<float> {
    static constexpr int dt = 1, V = 4;
};

// A lane's share of a row: C runs of V consecutive elements, run j at column
// (j * lanes + lane) * V.  VEC: 16-byte runs; otherwise V = 1.
template <class T, bool VEC, int NW, int E>
struct RowGeom {
    static constexpr int V = VEC ? Elem<T>::V : 1;
    static constexpr int C = E / V;
    static constexpr int LANES = NW * 64;
    static __device__ __forceinline__ int col(int j, int lane) { return (j * LANES + lane) * V; }
};

template <class T, bool VEC, int NW, int E>
struct RowRaw {
    using G = RowGeom<T, VEC, NW, E>;
    u32x4_t w[VEC ? G::C : 1];
    T s[VEC ? 1 : G::C];
};

// A row exactly as loaded (decoded where it is used, so that the wait for the
// load falls there); columns past the end read as zeros.  STREAM: the row is not
// kept in the caches.  The backward streams what it reads (8192 x 4096 bf16 with
// an added gradient 64.4 -> 61.4 us; stores 63.6, both 63.8).
template <class T, bool VEC, int NW, int E, bool STREAM = false>
__device__ __forceinline__ void row_load(const void* p, int64_t base, int cols, int lane, bool on,
                                         RowRaw<T, VEC, NW, E>& r) {
    using G = RowGeom<T, VEC, NW, E>;
    const GMEM T* q = gm(static_cast<const T*>(p)) + base;
#pragma unroll
    for (int j = 0; j < G::C; ++j) {
        const int c = G::col(j, lane);
        if constexpr (VEC) {
            r.w[j] = u32x4_t{0u, 0u, 0u, 0u};
            if (on && c < cols) {
                const GMEM u32x4_t* w = reinterpret_cast<const GMEM u32x4_t*>(q + c);
                r.w[j] = STREAM ? __builtin_nontemporal_load(w) : *w;
            }
        } else {
            r.s[j] = T(0);
            if (on && c < cols) r.s[j] = q[c];
        }
    }
}

template <class T, bool VEC, int NW, int E>
__device__ __forceinline__ void row_decode(const RowRaw<T, VEC, NW, E>& r, float (&v)[E]) {
    using G = RowGeom<T, VEC, NW, E>;
#pragma unroll
    for (int j = 0; j < G::C; ++j) {
        if constexpr (!VEC) {
            if constexpr (Elem<T>::dt == 0) v[j] = bf16_bits_to_f32(r.s[j]);
            else v[j] = r.s[j];
        } else if constexpr (Elem<T>::dt == 0) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[8 * j + 2 * k] = __uint_as_float(r.w[j][k] << 16);
                v[8 * j + 2 * k + 1] = __uint_as_float(r.w[j][k] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) v[4 * j + k] = __uint_as_float(r.w[j][k]);
        }
    }
}

template <class T, bool VEC, int NW, int E, bool STREAM = false>
__device__ __forceinline__ void row_store(void* p, int64_t base, int cols, int lane, const float (&v)[E]) {
    using G = RowGeom<T, VEC, NW, E>;
    GMEM T* q = gm(static_cast<T*>(p)) + base;
#pragma unroll
    for (int j = 0; j < G::C; ++j) {
        const int c = G::col(j, lane);
        if (c >= cols) continue;
        if constexpr (!VEC) {
            if constexpr (Elem<T>::dt == 0) q[c] = uint16_t(f32_to_bf16_bits(v[j]));
            else q[c] = v[j];
        } else if constexpr (Elem<T>::dt == 0) {
            const u32x4_t w = {pack_bf16(v[8 * j], v[8 * j + 1]), pack_bf16(v[8 * j + 2], v[8 * j + 3]),
                               pack_bf16(v[8 * j + 4], v[8 * j + 5]), pack_bf16(v[8 * j + 6], v[8 * j + 7])};
            put16<STREAM>(q + c, w);
        } else {
            put16<STREAM>(q + c, f32x4_t{v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]});
        }
    }
}

// gain / bias of a lane's columns, in float32.
template <class T, bool VEC, int NW, int E>
__device__ __forceinline__ void param_load(const void* p, int dt, bool vec, int cols, int lane, float (&v)[E]) {
    using G = RowGeom<T, VEC, NW, E>;
#pragma unroll
    for (int j = 0; j < G::C; ++j) {
        const int c = G::col(j, lane);
        if constexpr (!VEC) {
            v[j] = c < cols ? load1(p, c, dt) : 0.f;
        } else {
            const int n = c < cols ? G::V : 0;   // cols is a multiple of V here
            if constexpr (G::V == 8) {
                float t[8];
                load8(p, c, dt, vec, n, t);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[8 * j + k] = t[k];
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) v[4 * j + k] = 0.f;
                if (n && vec && dt == 1) {
                    const f32x4_t t = *gm(reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + c));
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[4 * j + k] = t[k];
                } else if (n) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[4 * j + k] = load1(p, c + k, dt);
                }
            }
        }
    }
}

// Sums of K values over the NW waves that share a row.  `red` holds one slot per
// wave and value; callers alternate between two halves of it, so one barrier
// per sum is enough.
template <int NW, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float (*red)[2], int wave) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = wave_add(v[k]);
    if constexpr (NW > 1) {
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int k = 0; k < K; ++k) red[wave][k] = v[k];
        }
        __syncthreads();
        const int w0 = wave / NW * NW;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            v[k] = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) v[k] += red[w0 + w][k];
        }
    }
}

// 8-bit copy of the lane's share of a row: the lanes that hold a group of 32
// columns agree on its magnitude.
template <class T, bool VEC, int NW, int E>
__device__ __forceinline__ void row_store_act8(const Act8View& q, int64_t row, int cols, int lane, bool on,
                                               const float (&v)[E]) {
    using G = RowGeom<T, VEC, NW, E>;
    constexpr int GL = kAct8Group / G::V;   // lanes of a group
#pragma unroll
    for (int j = 0; j < G::C; ++j) {
        const int c = G::col(j, lane);
        const bool in = on && c < cols;
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < G::V; ++k) m = max_mag(m, in ? v[j * G::V + k] : 0.f);
#pragma unroll
        for (int d = 1; d < GL; d *= 2) m = max_mag(m, __shfl_xor(m, d, 64));
        if (!in) continue;
        const uint32_t e = act8_exp(m);
        GMEM int8_t* p = gm(q.codes) + row * q.ld + c;
        if (VEC && q.vec) {
            u32x2_t w = {0u, 0u};
#pragma unroll
            for (int k = 0; k < G::V; ++k) w[k >> 2] |= act8_code(v[j * G::V + k], e) << (8 * (k & 3));
            if constexpr (G::V == 8) *reinterpret_cast<GMEM u32x2_t*>(p) = w;
            else if constexpr (G::V == 4) *reinterpret_cast<GMEM uint32_t*>(p) = w[0];
        } else {
#pragma unroll
            for (int k = 0; k < G::V; ++k) p[k] = int8_t(act8_code(v[j * G::V + k], e));
        }
        if ((c & (kAct8Group - 1)) == 0) gm(q.exps)[row * q.lde + c / kAct8Group] = uint8_t(e);
    }
}

// Sum over a workgroup; red: kWaves floats.
__device__ __forceinline__ float block_add(float v, float* red) {
    v = wave_add(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += red[w];
    return v;
}

}  // namespace
}  // namespace muon
