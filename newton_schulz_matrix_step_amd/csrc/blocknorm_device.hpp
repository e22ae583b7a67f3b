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
    __device__ __forceinline__ bool drops(uint32_t word, int half) const {
        return (half ? word >> 16 : word & 0xFFFFu) < cut;
    }
    // v under the mask: a select, so that what is dropped is 0 whatever it was
    __device__ __forceinline__ float keep(float v, uint32_t word, int half) const { return drops(word, half) ? 0.f : v * scale; }
    // the words of the run of V columns at column c (a multiple of V): half k & 1 of word k / 2
    template <int V>
    __device__ __forceinline__ u32x4_t run_words(uint32_t row, uint32_t c) const {
        const u32x4_t w = words(row, c >> 3);
        if constexpr (V == 8) return w;
        const bool hi = (c & 4) != 0;
        return u32x4_t{hi ? w[2] : w[0], hi ? w[3] : w[1], 0u, 0u};
    }
    // that run's V values
    template <int V>
    __device__ __forceinline__ void run(uint32_t row, uint32_t c, float* v) const {
        const u32x4_t w = run_words<V>(row, c);
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = keep(v[k], w[k >> 1], k & 1);
    }
    // and, unscaled, the values beside them (`beside`), of which what is dropped is 0 too
    template <int V>
    __device__ __forceinline__ void run(uint32_t row, uint32_t c, float* v, float* o, bool beside) const {
        const u32x4_t w = run_words<V>(row, c);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            v[k] = keep(v[k], w[k >> 1], k & 1);
            o[k] = beside && drops(w[k >> 1], k & 1) ? 0.f : o[k];
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
__device__ __forceinline__ typename RunRaw<T, V>::vec run_whole(const GMEM T* p, bool in) {   // zeros where not in
    typename RunRaw<T, V>::vec w;
#pragma unroll
    for (int k = 0; k < RunRaw<T, V>::W; ++k) w[k] = 0u;
    if (!in) return w;
    if constexpr (RunRaw<T, V>::W == 4) {    // (the alignment would be lost in a template's type)
        const GMEM u32x4_any_t* q = reinterpret_cast<const GMEM u32x4_any_t*>(p);
        w = STREAM ? __builtin_nontemporal_load(q) : *q;
    } else {
        const GMEM u32x2_any_t* q = reinterpret_cast<const GMEM u32x2_any_t*>(p);
        w = STREAM ? __builtin_nontemporal_load(q) : *q;
    }
    return w;
}
template <class T, int V, bool STREAM>
__device__ __forceinline__ typename RunRaw<T, V>::vec run_get(const GMEM T* p, int n) {
    using R = RunRaw<T, V>;
    typename R::vec w = run_whole<T, V, STREAM>(p, n >= V);
    if (n <= 0 || n >= V) return w;
    T t[V];                              // one wait for all: past the end the last one again
#pragma unroll
    for (int k = 0; k < V; ++k) t[k] = p[k < n ? k : n - 1];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        if constexpr (sizeof(T) == 2) w[k / 2] |= (k < n ? uint32_t(t[k]) : 0u) << (16 * (k & 1));
        else w[k] = k < n ? __float_as_uint(t[k]) : 0u;
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
    // element by element, the run's words moved down as they go (a short loop: the
    // row's last lane alone comes here)
    typename R::vec t = w;
#pragma unroll 1
    for (int k = 0; k < n; ++k) {
        if constexpr (sizeof(T) == 2) p[k] = uint16_t(t[0]);
        else p[k] = __uint_as_float(t[0]);
#pragma unroll
        for (int i = 0; i < R::W; ++i) {
            const uint32_t next = i + 1 < R::W ? t[i + 1] : 0u;
            if constexpr (sizeof(T) == 2) t[i] = (t[i] >> 16) | (next << 16);
            else t[i] = next;
        }
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
    // A run that the row's end cuts is loaded as the row's last V elements and moved
    // down where it is decoded: loaded element by element it would be put together,
    // and so waited for, where the loads are issued (8192 x 4095 bf16, backward: 161 us
    // so, 122 this way).
    template <class T, bool STREAM>
    static __device__ __forceinline__ void load(const void* p, int64_t base, int cols, int lane, bool on, Raw<T>& r) {
        const GMEM char* q = reinterpret_cast<const GMEM char*>(gm(static_cast<const T*>(p)) + base);
#pragma unroll
        for (int j = 0; j < C; ++j) {    // a scalar base and a 32-bit offset that stays the same from row to row
            const int c = col(j, lane), n = cols - c, back = n < V ? V - n : 0;
            r.w[j] = run_whole<T, V, STREAM>(reinterpret_cast<const GMEM T*>(q + uint32_t(c - back) * uint32_t(sizeof(T))),
                                             on && n > 0);
        }
    }
    template <class T>
    static __device__ __forceinline__ void decode(const Raw<T>& r, int cols, int lane, float (&v)[E]) {
#pragma unroll
        for (int j = 0; j < C; ++j) run_decode<T, V>(r.w[j], v + j * V);
        if (cols % V == 0) return;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int n = cols - col(j, lane), back = n > 0 && n < V ? V - n : 0;
            float* t = v + j * V;
#pragma unroll
            for (int s = 1; s < V; s *= 2)
#pragma unroll
                for (int k = 0; k < V; ++k) t[k] = back & s ? (k + s < V ? t[k + s] : 0.f) : t[k];
        }
    }
    template <class T>
    static __device__ __forceinline__ void decode(const Raw<T>& r, float (&v)[E]) {   // as encoded
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
        GMEM char* q = reinterpret_cast<GMEM char*>(gm(static_cast<T*>(p)) + base);
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c = col(j, lane);
            run_put<T, V, STREAM>(reinterpret_cast<GMEM T*>(q + uint32_t(c) * uint32_t(sizeof(T))), cols - c, r.w[j]);
        }
    }
    // float32 values of the lane's columns to a row of them
    static __device__ __forceinline__ void store_f32(GMEM float* p, int cols, int lane, const float (&v)[E]) {
        GMEM char* q = reinterpret_cast<GMEM char*>(p);
#pragma unroll
        for (int i = 0; i < E; i += 4) {
            const int c = col(i / V, lane) + i % V;
            run_put<float, 4, false>(reinterpret_cast<GMEM float*>(q + uint32_t(c) * 4u), cols - c, run_encode<float, 4>(v + i));
        }
    }
    // a parameter's elements of the lane's columns; `absent` where there is none
    static __device__ __forceinline__ void param(const void* p, int dt, int cols, int lane, float absent, float (&v)[E]) {
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int c = col(j, lane), n = cols - c;
            float* o = v + j * V;
            if (!p) {
#pragma unroll
                for (int k = 0; k < V; ++k) o[k] = k < n ? absent : 0.f;
            } else if (dt == 0) {
                run_decode<uint16_t, V>(run_get<uint16_t, V, false>(gm(static_cast<const uint16_t*>(p)) + c, n), o);
            } else {
#pragma unroll
                for (int h = 0; h < V; h += 4)
                    run_decode<float, 4>(run_get<float, 4, false>(gm(static_cast<const float*>(p)) + c + h, n - h), o + h);
            }
        }
    }
    static __device__ __forceinline__ void mask(const Philox& m, uint32_t row, int lane, float (&v)[E]) {
#pragma unroll
        for (int j = 0; j < C; ++j) m.run<V>(row, uint32_t(col(j, lane)), v + j * V);
    }
    static __device__ __forceinline__ void mask(const Philox& m, uint32_t row, int lane, float (&v)[E], float (&o)[E], bool beside) {
#pragma unroll
        for (int j = 0; j < C; ++j) m.run<V>(row, uint32_t(col(j, lane)), v + j * V, o + j * V, beside);
    }
};

// Waves of a workgroup whose rows take NW waves each.
constexpr int block_waves(int nw) { return nw > 8 ? nw : 8; }

// x + x of the lane N places on in its row of 16 (cyclic).
template <int N>
__device__ __forceinline__ float add_ror(float x) {
#ifdef __HIP__
    return x + __uint_as_float(uint32_t(__builtin_amdgcn_mov_dpp(int(__float_as_uint(x)), 0x120 + N, 0xF, 0xF, true)));
#else   // a host build for checking runs one lane at a time
    return x + x;
#endif
}
// Sum over a wave's lanes in every lane, without LDS: rotations within rows of 16,
// then swaps of rows.  Each step adds two values in either order, so all lanes
// hold the same bits.
__device__ __forceinline__ float wave_total(float v) {
    v = add_ror<1>(add_ror<2>(add_ror<4>(add_ror<8>(v))));
    typedef unsigned u2 __attribute__((ext_vector_type(2)));
    const u2 s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    const u2 t = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(t[0]) + __uint_as_float(t[1]);
}
// Sum of N (a power of two up to 16) values that lanes hold in turn: lane i value i mod N.
template <int N>
__device__ __forceinline__ float turn_total(float v) {
    if constexpr (N >= 16) v = add_ror<8>(v);
    if constexpr (N >= 8) v = add_ror<4>(v);
    if constexpr (N >= 4) v = add_ror<2>(v);
    if constexpr (N >= 2) v = add_ror<1>(v);
    return v;
}

// Sums over the NW waves of a row: `red` holds K values a wave, its two halves
// used in turn, so that one barrier a sum is enough.
template <int NW>
struct RowSums {
    float (*red)[2][block_waves(NW)];
    int wave, turn = 0;
    // exchange of each wave's K values: lane i gets those of wave i mod NW of its row,
    // and every lane in `ref` the first wave's last one
    template <int K>
    __device__ __forceinline__ void exchange(float (&v)[K], float* ref = nullptr) {
        if constexpr (NW > 1) {
            float(*r)[block_waves(NW)] = red[turn];
            turn ^= 1;
            if ((threadIdx.x & 63) == 0) {
#pragma unroll
                for (int k = 0; k < K; ++k) r[k][wave] = v[k];
            }
            __syncthreads();
            const int w = wave / NW * NW + int(threadIdx.x % NW);
#pragma unroll
            for (int k = 0; k < K; ++k) v[k] = r[k][w];
            if (ref) *ref = r[K - 1][wave / NW * NW];
        }
    }
    template <int K>
    __device__ __forceinline__ void operator()(float (&v)[K]) {
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = wave_total(v[k]);
        exchange(v);
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = turn_total<NW>(v[k]);
    }
};

// The types of a junction, and the widest row each variant holds: NW waves x 64
// lanes x E elements.
template <class F>
void pick_types(int sdt, int dt, F&& f) {
    if (sdt == 0) f(uint16_t{}, uint16_t{});
    else if (dt == 0) f(float{}, uint16_t{});
    else f(float{}, float{});
}
constexpr int kBlockRowCols = 8192;
constexpr int kBlockRowLeast = 8;        // columns: a run of any type
template <class F>
void pick_block_row(int cols, F&& f) {
    if (cols <= 512) f(std::integral_constant<int, 1>{});
    else if (cols <= 1024) f(std::integral_constant<int, 2>{});
    else if (cols <= 2048) f(std::integral_constant<int, 4>{});
    else if (cols <= 4096) f(std::integral_constant<int, 8>{});
    else f(std::integral_constant<int, 16>{});
}
inline int block_row_waves(int cols) { return cols <= 512 ? 1 : cols <= 1024 ? 2 : cols <= 2048 ? 4 : cols <= 4096 ? 8 : 16; }
constexpr int kRowElems = 8;             // elements a lane holds of a row
template <class ST, class BT>
constexpr int run_width() { return sizeof(ST) == 2 && sizeof(BT) == 2 ? 8 : 4; }

inline bool block_row_fits(int cols) { return cols >= kBlockRowLeast && cols <= kBlockRowCols; }

// 8 columns of a row for the kernels of rows that the registers do not hold
__device__ __forceinline__ void get8(const void* p, int64_t i, int dt, int n, float (&v)[8]) { load8(p, i, dt, false, n, v); }
__device__ __forceinline__ void par8(const void* p, int c, int dt, int n, float absent, float (&v)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = k < n ? (p ? load1(p, c + k, dt) : absent) : 0.f;
}

}  // namespace
}  // namespace muon
