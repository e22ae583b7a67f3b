// Device code of the norms around a block and of dropout: rows in registers in
// runs of 4 or 8 columns whatever their alignment, and the dropout mask.
#pragma once

#include "norm_device.hpp"

namespace muon {
namespace {

// ---- the dropout mask ----
// Philox 4x32 of ten rounds (Salmon, Moraes, Dror and Shaw 2011): the published
// multipliers and key increments.
struct Philox {
    uint32_t k0, k1, c2, c3;             // key; the call's half of the counter
    uint32_t cut;
    float scale;
    __device__ __forceinline__ explicit Philox(const DropMask& m) {
        const uint64_t n = m.offset + (m.step ? *gm(m.step) : 0);
        k0 = uint32_t(m.seed);
        k1 = uint32_t(m.seed >> 32);
        c2 = uint32_t(n);
        c3 = uint32_t(n >> 32);
        cut = m.cut;
        scale = m.scale;
    }
    // the four words of columns 8 block .. 8 block + 7 of a row
    __device__ __forceinline__ u32x4_t words(uint32_t row, uint32_t block) const {
        uint32_t x0 = block, x1 = row, x2 = c2, x3 = c3, a = k0, b = k1;
#pragma unroll
        for (int i = 0; i < 10; ++i) {
            const uint64_t p = uint64_t(x0) * 0xD2511F53u, q = uint64_t(x2) * 0xCD9E8D57u;
            x0 = uint32_t(q >> 32) ^ x1 ^ a;
            x1 = uint32_t(q);
            x2 = uint32_t(p >> 32) ^ x3 ^ b;
            x3 = uint32_t(p);
            a += 0x9E3779B9u;
            b += 0xBB67AE85u;
        }
        return u32x4_t{x0, x1, x2, x3};
    }
    // v under the mask: a select, so that what is dropped is 0 whatever it was
    __device__ __forceinline__ float keep(float v, uint32_t word, int half) const {
        return (half ? word >> 16 : word & 0xFFFFu) < cut ? 0.f : v * scale;
    }
    // the V values of the run at column c (a multiple of V)
    template <int V>
    __device__ __forceinline__ void run(uint32_t row, uint32_t c, float* v) const {
        const u32x4_t w = words(row, c >> 3);
        if constexpr (V == 8) {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = keep(v[k], w[k >> 1], k & 1);
        } else {
            const bool hi = (c & 4) != 0;
            const uint32_t w0 = hi ? w[2] : w[0], w1 = hi ? w[3] : w[1];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = keep(v[k], k < 2 ? w0 : w1, k & 1);
        }
    }
};

// ---- runs of V columns ----
// Vectors of their elements' alignment only: the memory takes them anywhere, so
// rows of any leading dimension move in whole runs; the run that a row's end
// cuts goes element by element.
typedef u32x4_t u32x4_any_t __attribute__((aligned(2)));
typedef u32x2_t u32x2_any_t __attribute__((aligned(2)));

template <class T, int V>
struct RunRaw {
    static_assert((sizeof(T) == 2 && (V == 4 || V == 8)) || (sizeof(T) == 4 && V == 4), "16 bytes a run at most");
    using vec = std::conditional_t<sizeof(T) * V == 16, u32x4_t, u32x2_t>;
    static constexpr int W = sizeof(T) * V / 4;
};

template <class T, int V, bool STREAM>
__device__ __forceinline__ typename RunRaw<T, V>::vec run_get(const GMEM T* p, int n) {
    using R = RunRaw<T, V>;
    typename R::vec w;
    if (n >= V) {
        if constexpr (R::W == 4) {       // (the alignment would be lost in a template's type)
            const GMEM u32x4_any_t* q = reinterpret_cast<const GMEM u32x4_any_t*>(p);
            return STREAM ? __builtin_nontemporal_load(q) : *q;
        } else {
            const GMEM u32x2_any_t* q = reinterpret_cast<const GMEM u32x2_any_t*>(p);
            return STREAM ? __builtin_nontemporal_load(q) : *q;
        }
    }
#pragma unroll
    for (int k = 0; k < R::W; ++k) w[k] = 0u;
    if (n <= 0) return w;
#pragma unroll
    for (int k = 0; k < V; ++k)
        if (k < n) {
            if constexpr (sizeof(T) == 2) w[k / 2] |= uint32_t(p[k]) << (16 * (k & 1));
            else w[k] = __float_as_uint(p[k]);
        }
    return w;
}
template <class T, int V>
__device__ __forceinline__ void run_decode(const typename RunRaw<T, V>::vec& w, float* v) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
        if constexpr (sizeof(T) == 2) v[k] = __uint_as_float(k & 1 ? w[k / 2] & 0xFFFF0000u : w[k / 2] << 16);
        else v[k] = __uint_as_float(w[k]);
    }
}
template <class T, int V>
__device__ __forceinline__ typename RunRaw<T, V>::vec run_encode(const float* v) {
    typename RunRaw<T, V>::vec w;
#pragma unroll
    for (int k = 0; k < RunRaw<T, V>::W; ++k) {
        if constexpr (sizeof(T) == 2) w[k] = pack_bf16(v[2 * k], v[2 * k + 1]);
        else w[k] = __float_as_uint(v[k]);
    }
    return w;
}
template <class T, int V, bool STREAM>
__device__ __forceinline__ void run_put(GMEM T* p, int n, const typename RunRaw<T, V>::vec& w) {
    using R = RunRaw<T, V>;
    if (n >= V) {
        if constexpr (R::W == 4) {
            GMEM u32x4_any_t* q = reinterpret_cast<GMEM u32x4_any_t*>(p);
            if constexpr (STREAM) __builtin_nontemporal_store(w, q);
            else *q = w;
        } else {
            GMEM u32x2_any_t* q = reinterpret_cast<GMEM u32x2_any_t*>(p);
            if constexpr (STREAM) __builtin_nontemporal_store(w, q);
            else *q = w;
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < V; ++k)
        if (k < n) {
            if constexpr (sizeof(T) == 2) p[k] = uint16_t(w[k / 2] >> (16 * (k & 1)));
            else p[k] = __uint_as_float(w[k]);
        }
}

// ---- rows: run j of a lane at column (j * LANES + lane) * V ----
template <int V_, int NW, int E>
struct BlockRow {
    static constexpr int V = V_, C = E / V_, LANES = NW * 64;
    static __device__ __forceinline__ int col(int j, int lane) { return (j * LANES + lane) * V; }

    template <class T>
    struct Raw {
        typename RunRaw<T, V>::vec w[C];
    };
    template <class T, bool STREAM>
    static __device__ __forceinline__ void load(const void* p, int64_t base, int cols, int lane, bool on, Raw<T>& r) {
        const GMEM T* q = gm(static_cast<const T*>(p)) + base;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c = col(j, lane);
            r.w[j] = run_get<T, V, STREAM>(q + c, on ? cols - c : 0);
        }
    }
    template <class T>
    static __device__ __forceinline__ void decode(const Raw<T>& r, float (&v)[E]) {
#pragma unroll
        for (int j = 0; j < C; ++j) run_decode<T, V>(r.w[j], v + j * V);
    }
    template <class T>
    static __device__ __forceinline__ void encode(const float (&v)[E], Raw<T>& r) {
#pragma unroll
        for (int j = 0; j < C; ++j) r.w[j] = run_encode<T, V>(v + j * V);
    }
    template <class T, bool STREAM>
    static __device__ __forceinline__ void store(void* p, int64_t base, int cols, int lane, const Raw<T>& r) {
        GMEM T* q = gm(static_cast<T*>(p)) + base;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c = col(j, lane);
            run_put<T, V, STREAM>(q + c, cols - c, r.w[j]);
        }
    }
    // a parameter's elements of the lane's columns; `absent` where there is none
    static __device__ __forceinline__ void param(const void* p, int dt, int cols, int lane, float absent, float (&v)[E]) {
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c = col(j, lane);
#pragma unroll
            for (int k = 0; k < V; ++k) v[j * V + k] = c + k < cols ? (p ? load1(p, c + k, dt) : absent) : 0.f;
        }
    }
    static __device__ __forceinline__ void mask(const Philox& m, uint32_t row, int lane, float (&v)[E]) {
#pragma unroll
        for (int j = 0; j < C; ++j) m.run<V>(row, uint32_t(col(j, lane)), v + j * V);
    }
};

// Sums of K values over the NW waves of a row; two halves of `red` in turn.
template <int NW, int K>
__device__ __forceinline__ void row_sum_turn(float (&v)[K], float (*red)[kWaves][2], int& turn, int wave) {
    row_sum<NW, K>(v, red[turn], wave);
    turn ^= 1;
}

// The types of a junction, and the widest row each variant holds: NW waves x 64
// lanes x E elements.
template <class F>
void pick_types(int sdt, int dt, F&& f) {
    if (sdt == 0) f(uint16_t{}, uint16_t{});
    else if (dt == 0) f(float{}, uint16_t{});
    else f(float{}, float{});
}
constexpr int kBlockRowCols = 8192;
template <class F>
void pick_block_row(int cols, F&& f) {
    if (cols <= 1024) f(std::integral_constant<int, 1>{});
    else if (cols <= 2048) f(std::integral_constant<int, 2>{});
    else if (cols <= 4096) f(std::integral_constant<int, 4>{});
    else f(std::integral_constant<int, 8>{});
}
inline int block_row_waves(int cols) { return cols <= 1024 ? 1 : cols <= 2048 ? 2 : cols <= 4096 ? 4 : 8; }
constexpr int kRowElems = 16;            // elements a lane holds of a row
template <class ST, class BT>
constexpr int run_width() { return sizeof(ST) == 2 && sizeof(BT) == 2 ? 8 : 4; }

// 8 columns of a row for the kernels of rows that the registers do not hold
__device__ __forceinline__ void get8(const void* p, int64_t i, int dt, int n, float (&v)[8]) { load8(p, i, dt, false, n, v); }
__device__ __forceinline__ void par8(const void* p, int c, int dt, int n, float absent, float (&v)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = k < n ? (p ? load1(p, c + k, dt) : absent) : 0.f;
}

}  // namespace
}  // namespace muon
