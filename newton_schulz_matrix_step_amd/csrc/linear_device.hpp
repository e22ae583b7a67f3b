// Device code of products on the matrix cores, shared by the linear layer's
// kernels (linear_kernels.hip) and the gated feed-forward's (gated_kernels.hip):
// operands from global memory to LDS and into fragments, the tile kernels, and
// the epilogues of the linear layer's three products.
#pragma once

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "layer_device.hpp"

namespace muon {
namespace {

using namespace layer;

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));
#ifndef LDS_AS
#define LDS_AS __attribute__((address_space(3)))
#endif

// ---------------------------------------------------------------------------
// global -> LDS
// ---------------------------------------------------------------------------
constexpr uint32_t kFar = 0x80000000u;        // beyond every buffer below: such a lane reads zeros
constexpr uint32_t kMaxRecords = 0x7FFFFFFFu;

__device__ __forceinline__ i32x4_t buffer_at(const char* p, uint32_t bytes) {
    const uint64_t u = reinterpret_cast<uint64_t>(p);
    i32x4_t r;
    r[0] = __builtin_amdgcn_readfirstlane(int(uint32_t(u)));
    r[1] = __builtin_amdgcn_readfirstlane(int(uint32_t(u >> 32) & 0xFFFFu));
    r[2] = __builtin_amdgcn_readfirstlane(int(bytes));
    r[3] = 0x00020000;                        // raw buffer of 32-bit data
    return r;
}

#ifndef MUON_BUFFER_TO_LDS
__device__ __forceinline__ uint32_t lds_base(const char* smem) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((LDS_AS const char*)smem));
}
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// 16 bytes per lane from the buffer straight into LDS: lane L's bytes land at
// LDS address lds + 16 L (lds wave-uniform); a lane whose offset lies past the
// buffer's end stores zeros.  Nothing is returned in registers; completion
// counts in vmcnt.
__device__ __forceinline__ void buffer_to_lds(i32x4_t buf, uint32_t voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(voff), "s"(buf)
                 : "memory", "m0");
}
#pragma clang diagnostic pop
#else
#define lds_base MUON_LDS_BASE
#define buffer_to_lds MUON_BUFFER_TO_LDS
#endif

template <int N>
__device__ __forceinline__ void vm_wait() {   // s_waitcnt vmcnt(N), no wait on the other counters
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

template <class T>
struct Num;
template <>
struct Num<uint16_t> {
    static constexpr int dt = 0, BK = 64, EPC = 8;   // k per stage, elements of a 16-byte chunk
};
template <>
struct Num<float> {
    static constexpr int dt = 1, BK = 32, EPC = 4;
};

// Where an operand comes from: S_DMA whole aligned 16-byte chunks straight into
// LDS; S_ANY any alignment and size, element by element through registers;
// S_ACT8 8-bit codes, decoded on their way through registers.
enum Src { S_DMA, S_ANY, S_ACT8 };

// One stage of one operand is 128 bytes of LDS per tile row: 16 KB for a
// 128-wide tile.  Row-contiguous operands (KC) lie as [row][8 chunks of 16 bytes
// along k], chunk XOR row & 7; k-strided ones as [k][W elements] (W the tile
// edge) with their own chunk swizzle.  Both feed the fragment reads below
// without bank conflicts.
constexpr int kOpBytes = 16384;

// bf16 [k][128]: a ds_read_b64_tr_b16 group of 16 lanes reads 4 k rows x 32
// bytes (bits 1-2 spread them over a 128-byte window, bit 3 moves the
// neighbouring group to the other half); [k][64]: two of the four rows share a
// 256-byte window's half, so bit 1 goes by k >> 1, and bit 2 moves the
// neighbouring group; [k][32]: the four rows lie in different 64-byte windows,
// and bit 1 moves the neighbouring group to the windows' other halves.  float32
// [k][W]: the four lane groups read rows 4 apart, which bits 2-3 put on different
// 64-byte windows (W = 32: two of them, bit 2).
template <class T, int W>
__device__ __forceinline__ int ks_swizzle(int k) {
    if constexpr (Num<T>::dt == 1) return ((k >> 2) & (W == 32 ? 1 : 3)) << 2;
    else if constexpr (W == 32) return (k >> 2) & 2;
    else if constexpr (W == 64) return (k & 2) | ((k >> 1) & 4);
    else return ((2 * k) & 6) | ((((k >> 3) ^ (k >> 2)) & 1) << 3);
}

// The operand's rows (KC) or columns (KS) [e0, e0 + W) of the tile, `ext`
// existing in all; k runs to kend.  Four waves load it.
template <class T, bool KC, int SRC, int W>
struct Loader {
    using N = Num<T>;
    static constexpr int ES = sizeof(T);
    static constexpr int NQ = W / 32;                    // 1 KB blocks a wave loads of a stage
    static constexpr int CPR = KC ? 8 : W * ES / 16;     // chunks of an LDS row
    static constexpr int RPB = 64 / CPR;                 // LDS rows of 1 KB
    const char* base;
    int64_t ld, ext, kend, e0;
    const uint8_t* exps;
    int64_t lde;
    bool vec8;
    uint32_t voff[NQ];
    u32x4_t reg[SRC == S_DMA ? 1 : NQ];
    int wave, lane;

    // LDS row and logical chunk of this lane's part of 1 KB block q
    __device__ __forceinline__ int lrow(int q) const { return (wave * NQ + q) * RPB + lane / CPR; }
    __device__ __forceinline__ int lchunk(int q) const {
        const int r = lrow(q), c = lane % CPR;
        return KC ? c ^ (r & 7) : c ^ ks_swizzle<T, W>(r);
    }

    __device__ __forceinline__ void init(const void* p, int64_t ld_, int64_t ext_, int64_t e0_, int64_t kend_, int wave_,
                                         int lane_) {
        ld = ld_;
        ext = ext_;
        e0 = e0_;
        kend = kend_;
        wave = wave_;
        lane = lane_;
        base = static_cast<const char*>(p);
        if constexpr (SRC == S_DMA) {
            base += (KC ? e0 * ld : e0) * ES;
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                const int r = lrow(q), c = lchunk(q);
                const bool in = KC ? e0 + r < ext : e0 + c * N::EPC < ext;
                voff[q] = in ? uint32_t(r * ld * ES + c * 16) : kFar;
            }
        }
    }

    // S_DMA: enqueue block q of the stage at k0 into LDS at address st, or all of it
    // (`from`: this operand's base, or that of another one laid out alike)
    __device__ __forceinline__ void issue(const char* from, int64_t k0, uint32_t st, int q) {
        if constexpr (SRC == S_DMA) {
            const uint32_t at = st + (wave * NQ + q) * 1024;
            if constexpr (KC) {
                const bool in = k0 + lchunk(q) * N::EPC < kend;   // a whole chunk is in or out
                buffer_to_lds(buffer_at(from + k0 * ES, kMaxRecords), in ? voff[q] : kFar, at);
            } else {
                int64_t n = (kend - k0) * ld * ES;   // rows past kend lie past the buffer
                n = n < 0 ? 0 : (n > int64_t(kMaxRecords) ? int64_t(kMaxRecords) : n);
                buffer_to_lds(buffer_at(from + k0 * ld * ES, uint32_t(n)), voff[q], at);
            }
        }
    }
    __device__ __forceinline__ void issue(int64_t k0, uint32_t st, int q) { issue(base, k0, st, q); }
    __device__ __forceinline__ void issue(int64_t k0, uint32_t st) {
#pragma unroll
        for (int q = 0; q < NQ; ++q) issue(k0, st, q);
    }

    // S_ANY, S_ACT8: load the stage at k0 into registers
    __device__ __forceinline__ void fetch(int64_t k0) {
        if constexpr (SRC == S_ANY) {
            const GMEM T* p = gm(reinterpret_cast<const T*>(base));
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                const int64_t r = KC ? e0 + lrow(q) : k0 + lrow(q);
                const int64_t c = (KC ? k0 : e0) + lchunk(q) * N::EPC;
                const int64_t rn = KC ? ext : kend, cn = KC ? kend : ext;
                uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int e = 0; e < N::EPC; ++e) {
                    if (r < rn && c + e < cn) {
                        if constexpr (N::dt == 0) w[e / 2] |= uint32_t(p[r * ld + c + e]) << (16 * (e & 1));
                        else w[e] = __float_as_uint(p[r * ld + c + e]);
                    }
                }
                reg[q] = u32x4_t{w[0], w[1], w[2], w[3]};
            }
        } else if constexpr (SRC == S_ACT8) {
            static_assert(!KC, "checkpoints are stored by rows of k here");
            const GMEM int8_t* p = gm(reinterpret_cast<const int8_t*>(base));
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                const int64_t k = k0 + lrow(q);
                const int64_t c = e0 + lchunk(q) * N::EPC;
                u32x4_t r = {0u, 0u, 0u, 0u};   // codes in [0..1], the exponent byte in [2]
                if (k < kend && c < ext) {
                    if (vec8 && c + N::EPC <= ext) {
                        if constexpr (N::EPC == 8) {
                            const u32x2_t t = *reinterpret_cast<const GMEM u32x2_t*>(p + k * ld + c);
                            r[0] = t[0];
                            r[1] = t[1];
                        } else {
                            r[0] = *reinterpret_cast<const GMEM uint32_t*>(p + k * ld + c);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < N::EPC; ++e)
                            if (c + e < ext) r[e / 4] |= uint32_t(uint8_t(p[k * ld + c + e])) << (8 * (e & 3));
                    }
                    r[2] = gm(exps)[k * lde + c / kAct8Group];
                }
                reg[q] = r;
            }
        }
    }
    // and store them to LDS.  code * 2^k has at most 7 significant bits, so the
    // bf16 value is its float32 value's upper half, exactly.
    __device__ __forceinline__ void put(char* st) {
        if constexpr (SRC == S_ANY) {
#pragma unroll
            for (int q = 0; q < NQ; ++q) *reinterpret_cast<u32x4_t*>(st + (wave * NQ + q) * 1024 + lane * 16) = reg[q];
        } else if constexpr (SRC == S_ACT8) {
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                const float step = act8_step(reg[q][2]);
                float v[8];
                act8_dec4(reg[q][0], step, v);
                u32x4_t w;
                if constexpr (N::EPC == 8) {
                    act8_dec4(reg[q][1], step, v + 4);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = (__float_as_uint(v[2 * e]) >> 16) | (__float_as_uint(v[2 * e + 1]) & 0xFFFF0000u);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(v[e]);
                }
                *reinterpret_cast<u32x4_t*>(st + (wave * NQ + q) * 1024 + lane * 16) = w;
            }
        }
    }
};

// ---------------------------------------------------------------------------
// LDS -> fragments.  bf16: 8 k values k = 32 s + 8 (lane >> 4) + e of row or
// column rc + (lane & 15).  float32: 4 values k = 16 s + 4 (lane >> 4) + e, one
// for each of four MFMAs; both operands use the same k for the same lane group
// and e, which is all a sum over k asks for.
// ---------------------------------------------------------------------------
template <class T, bool KC, int W>
__device__ __forceinline__ auto frag(const char* lds, int rc, int s, int lane) {
    const int g = lane >> 4, i = lane & 15;
    if constexpr (KC) {
        const int r = rc + i;
        const u32x4_t w = *reinterpret_cast<const u32x4_t*>(lds + r * 128 + (((4 * s + g) ^ (r & 7)) << 4));
        if constexpr (Num<T>::dt == 0) return __builtin_bit_cast(bf16x8_t, w);
        else return __builtin_bit_cast(f32x4_t, w);
    } else if constexpr (Num<T>::dt == 0) {
        const int n = rc + 4 * (i & 3);
        i16x4_t h[2];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const int k = 32 * s + 8 * g + 4 * hh + (i >> 2);
            const char* p = lds + k * (W * 2) + (((n >> 3) ^ ks_swizzle<T, W>(k)) << 4) + (n & 7) * 2;
            h[hh] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS i16x4_t*)(p));
        }
        return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
        f32x4_t v;
        const int n = rc + i;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int k = 16 * s + 4 * g + e;
            v[e] = *reinterpret_cast<const float*>(lds + k * (W * 4) + (((n >> 2) ^ ks_swizzle<T, W>(k)) << 4) + (n & 3) * 4);
        }
        return v;
    }
}

__device__ __forceinline__ f32x4_t mma(bf16x8_t a, bf16x8_t b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t mma(f32x4_t a, f32x4_t b, f32x4_t c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
}
template <class F>
__device__ __forceinline__ F ones() {
    F f;
    if constexpr (std::is_same_v<F, bf16x8_t>) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = (__bf16)1.f;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = 1.f;
    }
    return f;
}

// ---------------------------------------------------------------------------
// epilogue
// ---------------------------------------------------------------------------
// Two neighbouring 16 x 16 accumulators hold, per lane, 4 consecutive output
// elements of each tile (elements 4 g .. 4 g + 3, g = lane >> 4).  After the two
// swaps lane group g holds the 8 consecutive elements 8 g .. 8 g + 7 of the 32.
__device__ __forceinline__ void join_tiles(f32x4_t a, f32x4_t b, float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        typedef unsigned u2 __attribute__((ext_vector_type(2)));
        const u2 s = __builtin_amdgcn_permlane32_swap(__float_as_uint(a[e]), __float_as_uint(b[e]), false, false);
        const u2 t = __builtin_amdgcn_permlane16_swap(s[0], s[1], false, false);
        v[e] = __uint_as_float(t[0]);
        v[4 + e] = __uint_as_float(t[1]);
    }
}

// Where a run of 8 consecutive output elements lies: row r + rl, columns c + cl ..
// of the output, r and c the same for all lanes.  An address is then a scalar
// base plus a 32-bit lane offset that stays the same from run to run.
struct RunAt {
    int64_t r, c;
    int rl, cl;
};
// Byte address of that run in a matrix of `es`-byte elements.
template <class B>
__device__ __forceinline__ GMEM B* run_ptr(B* p, int64_t ld, const RunAt& t, int es) {
    return gm(reinterpret_cast<B*>(const_cast<char*>(reinterpret_cast<const char*>(p)) + (t.r * ld + t.c) * es)) +
           (uint32_t(t.rl) * uint32_t(ld) + uint32_t(t.cl)) * uint32_t(es);
}
template <int DT>
__device__ __forceinline__ void run_load(const void* p, int64_t ld, const RunAt& t, int dt_arg, float (&v)[8]) {
    const int dt = DT >= 0 ? DT : dt_arg;
    const GMEM char* q = run_ptr(static_cast<const char*>(p), ld, t, dt == 0 ? 2 : 4);
    if (dt == 0) {
        unpack_bf16x8(*reinterpret_cast<const GMEM u32x4_t*>(q), v);
    } else {
        const f32x4_t a = *reinterpret_cast<const GMEM f32x4_t*>(q), b = *reinterpret_cast<const GMEM f32x4_t*>(q + 16);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[k] = a[k];
            v[4 + k] = b[k];
        }
    }
}
template <int DT, bool STREAM = false>
__device__ __forceinline__ void run_store(void* p, int64_t ld, const RunAt& t, int dt_arg, const float (&v)[8]) {
    const int dt = DT >= 0 ? DT : dt_arg;
    GMEM char* q = run_ptr(static_cast<char*>(p), ld, t, dt == 0 ? 2 : 4);
    if (dt == 0) {
        put16<STREAM>(q, u32x4_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                 pack_bf16(v[6], v[7])});
    } else {
        put16<STREAM>(q, f32x4_t{v[0], v[1], v[2], v[3]});
        put16<STREAM>(q + 16, f32x4_t{v[4], v[5], v[6], v[7]});
    }
}
template <int SH>
__device__ __forceinline__ float group_max(const float (&v)[8], int nv) {
    float m = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max_mag(m, k < nv ? v[k] : 0.f);
    if constexpr (SH == 16) {            // lanes 16 and 32 apart: swapped, without LDS
        typedef unsigned u2 __attribute__((ext_vector_type(2)));
        const u2 s = __builtin_amdgcn_permlane16_swap(__float_as_uint(m), __float_as_uint(m), false, false);
        m = max_mag(__uint_as_float(s[0]), __uint_as_float(s[1]));
        const u2 t = __builtin_amdgcn_permlane32_swap(__float_as_uint(m), __float_as_uint(m), false, false);
        return max_mag(__uint_as_float(t[0]), __uint_as_float(t[1]));
    } else {
        m = max_mag(m, __shfl_xor(m, SH, 64));
        return max_mag(m, __shfl_xor(m, 2 * SH, 64));
    }
}
// act8_code of 8 values as bytes.  1.5 * 2^23 + x, |x| <= 127, is rounded to an
// integer (nearest, halves to even), whose two's complement is its low bits.
__device__ __forceinline__ u32x2_t act8_pack(const float (&v)[8], uint32_t e, int nv) {
    const bool bad = e == 255u;
    const float inv = bad ? 0.f : act8_inv(e);
    u32x2_t w;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t b[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            b[k] = __float_as_uint(fmaf(4 * h + k < nv ? v[4 * h + k] : 0.f, inv, 12582912.f)) & 0xFFu;
        w[h] = bad ? 0u : b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24);   // (a NaN's product is one)
    }
    return w;
}
__device__ __forceinline__ void act_all(float (&v)[8], int act) {
    if (act == ACT_GELU) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = act_value(v[k], ACT_GELU);
    } else if (act == ACT_RELU_SQ) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = act_value(v[k], ACT_RELU_SQ);
    }
}
// Gates: act(z), and its value and derivative.  The logistic and its limits as
// in act_value and act_both; beyond |z| = 80 it is 0 or 1 (e^-80 = 2e-35).
__device__ __forceinline__ float logistic(float z) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
}
template <int ACT>
__device__ __forceinline__ float gate_value(float z) {
    if (ACT == GATE_SILU) return mul_zero(z, logistic(z));
    if (ACT == GATE_GELU) return act_value(z, ACT_GELU);
    if (ACT == GATE_SIGMOID) return logistic(z);
    return z <= 0.f ? 0.f : z;                        // a NaN stays one
}
template <int ACT>
__device__ __forceinline__ void gate_both(float z, float& v, float& d) {
    if (ACT == GATE_GELU) {
        act_both(z, ACT_GELU, v, d);
    } else if (ACT == GATE_RELU) {
        v = z <= 0.f ? 0.f : z;
        d = z <= 0.f ? 0.f : (z > 0.f ? 1.f : z);
    } else {
        const float c = __builtin_elementwise_maximum(__builtin_elementwise_minimum(z, 80.f), -80.f);
        const float e = __builtin_amdgcn_exp2f(-1.4426950408889634f * c);
        const float s = z < -80.f ? 0.f : __builtin_amdgcn_rcpf(1.f + e), r = e * s;   // r = 1 - s
        v = ACT == GATE_SILU ? mul_zero(z, s) : s;
        d = ACT == GATE_SILU ? fmaf(c * s, r, s) : s * r;
    }
}
// g = act(g) u
template <int ACT>
__device__ __forceinline__ void gate_each(float (&g)[8], const float (&u)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) g[k] = gate_value<ACT>(g[k]) * u[k];
}
__device__ __forceinline__ void gate_all(float (&g)[8], const float (&u)[8], int act) {
    if (act == GATE_SILU) gate_each<GATE_SILU>(g, u);
    else if (act == GATE_GELU) gate_each<GATE_GELU>(g, u);
    else if (act == GATE_SIGMOID) gate_each<GATE_SIGMOID>(g, u);
    else gate_each<GATE_RELU>(g, u);
}
// From dh in v: v = dh u act'(g), g = dh act(g), u = act(g) u
template <int ACT>
__device__ __forceinline__ void gate_grad_each(float (&v)[8], float (&g)[8], float (&u)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        float f, d;
        gate_both<ACT>(g[k], f, d);
        g[k] = v[k] * f;
        v[k] = v[k] * u[k] * d;
        u[k] = f * u[k];
    }
}
__device__ __forceinline__ void gate_grad_all(float (&v)[8], float (&g)[8], float (&u)[8], int act) {
    if (act == GATE_SILU) gate_grad_each<GATE_SILU>(v, g, u);
    else if (act == GATE_GELU) gate_grad_each<GATE_GELU>(v, g, u);
    else if (act == GATE_SIGMOID) gate_grad_each<GATE_SIGMOID>(v, g, u);
    else gate_grad_each<GATE_RELU>(v, g, u);
}
// v *= act'(z), h = act(z)
__device__ __forceinline__ void act_grad_all(float (&v)[8], const float (&z)[8], float (&h)[8], int act) {
    float d[8];
    if (act == ACT_GELU) {
#pragma unroll
        for (int k = 0; k < 8; ++k) act_both(z[k], ACT_GELU, h[k], d[k]);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) act_both(z[k], act, h[k], d[k]);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= d[k];
}

// The run's 8 elements, all inside, every buffer of the epilogue allowing
// vectors and 32-bit offsets (fast_epilogue).  The four lanes of a group of 32
// columns lie 16 apart, in the same row (so a row past the end leaves them out
// together).
template <int KIND, int DT>
__device__ __forceinline__ void epilogue_run(const LinArgs& a, const RunAt& t, float (&v)[8]) {
    if (KIND == LIN_FWD) {
        if (a.bias) {
            float b[8];
            const RunAt tb{0, t.c, 0, t.cl};
            if (a.bias_dt == 0) run_load<0>(a.bias, 0, tb, 0, b);
            else run_load<1>(a.bias, 0, tb, 1, b);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] += b[k];
        }
        if (a.z) run_store<DT>(a.z, a.ld_z, t, DT, v);
        if (a.z8.codes) {
            const uint32_t e = act8_exp(group_max<16>(v, 8));
            *reinterpret_cast<GMEM u32x2_t*>(run_ptr(a.z8.codes, a.z8.ld, t, 1)) = act8_pack(v, e, 8);
            if ((t.cl & (kAct8Group - 1)) == 0)
                *run_ptr(a.z8.exps, a.z8.lde, RunAt{t.r, t.c / kAct8Group, t.rl, t.cl / kAct8Group}, 1) = uint8_t(e);
        }
        act_all(v, a.act);
    } else if (KIND == LIN_DX) {
        if (a.z || a.z8.codes) {
            float z[8], h[8];
            if (a.z) {
                run_load<DT>(a.z, a.ld_z, t, DT, z);
            } else {
                const float step =
                    act8_step(*run_ptr(a.z8.exps, a.z8.lde, RunAt{t.r, t.c / kAct8Group, t.rl, t.cl / kAct8Group}, 1));
                const u32x2_t w = *reinterpret_cast<const GMEM u32x2_t*>(run_ptr(a.z8.codes, a.z8.ld, t, 1));
                act8_dec4(w[0], step, z);
                act8_dec4(w[1], step, z + 4);
            }
            act_grad_all(v, z, h, a.act);
            if (a.act_out) {
                if (a.act_stream) {
                    asm volatile("");    // or both stores become one that does not stream
                    run_store<DT, true>(a.act_out, a.ld_act, t, DT, h);
                    asm volatile("");
                } else {
                    run_store<DT>(a.act_out, a.ld_act, t, DT, h);
                }
            }
        }
    } else if (a.accumulate) {
        float o[8];
        run_load<-1>(a.out, a.ld_out, t, a.out_dt, o);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += o[k];
    }
    if (KIND != LIN_DW && a.add) {
        float b[8];
        run_load<DT>(a.add, a.ld_add, t, DT, b);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += b[k];
    }
    run_store<KIND == LIN_DW ? -1 : DT>(a.out, a.ld_out, t, a.out_dt, v);
}

// ---- the gated feed-forward's epilogues ----
// Both pre-activations of a run as loaded (full, or codes and exponent byte), and
// the values they stand for.
template <int DT>
struct ZRaw {
    u32x4_t g, u, g1, u1;      // g1, u1: the second halves of float32 runs
};
template <int DT>
__device__ __forceinline__ void z_fetch(const GatedArgs& a, const RunAt& t, ZRaw<DT>& w) {
    if (a.z) {
        const GMEM char* g = run_ptr(static_cast<const char*>(a.z), a.ld_z, t, DT == 0 ? 2 : 4);
        const GMEM char* u = run_ptr(static_cast<const char*>(a.z2), a.ld_z, t, DT == 0 ? 2 : 4);
        w.g = *reinterpret_cast<const GMEM u32x4_t*>(g);
        w.u = *reinterpret_cast<const GMEM u32x4_t*>(u);
        if constexpr (DT == 1) {
            w.g1 = *reinterpret_cast<const GMEM u32x4_t*>(g + 16);
            w.u1 = *reinterpret_cast<const GMEM u32x4_t*>(u + 16);
        }
        return;
    }
    auto get = [&](const Act8View& q) {
        const u32x2_t c = *reinterpret_cast<const GMEM u32x2_t*>(run_ptr(q.codes, q.ld, t, 1));
        return u32x4_t{c[0], c[1], *run_ptr(q.exps, q.lde, RunAt{t.r, t.c / kAct8Group, t.rl, t.cl / kAct8Group}, 1), 0u};
    };
    w.g = get(a.z8);
    w.u = get(a.z8_2);
}
template <int DT>
__device__ __forceinline__ void z_values(bool full, u32x4_t w, u32x4_t w1, float (&v)[8]) {
    if (!full) {
        const float step = act8_step(w[2]);
        act8_dec4(w[0], step, v);
        act8_dec4(w[1], step, v + 4);
    } else if constexpr (DT == 0) {
        unpack_bf16x8(w, v);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[k] = __uint_as_float(w[k]);
            v[4 + k] = __uint_as_float(w1[k]);
        }
    }
}
template <int DT>
__device__ __forceinline__ void z_store(void* z, int64_t ld, const Act8View& z8, const RunAt& t, const float (&v)[8]) {
    if (z) run_store<DT>(z, ld, t, DT, v);
    if (z8.codes) {
        const uint32_t e = act8_exp(group_max<16>(v, 8));
        *reinterpret_cast<GMEM u32x2_t*>(run_ptr(z8.codes, z8.ld, t, 1)) = act8_pack(v, e, 8);
        if ((t.cl & (kAct8Group - 1)) == 0)
            *run_ptr(z8.exps, z8.lde, RunAt{t.r, t.c / kAct8Group, t.rl, t.cl / kAct8Group}, 1) = uint8_t(e);
    }
}
// h = act(zg) zu from the two projections' sums; the run is all inside, and the
// four lanes of a group of 32 columns lie 16 apart where z8 is written.
template <int DT>
__device__ __forceinline__ void gated_run(const GatedArgs& a, const RunAt& t, float (&g)[8], float (&u)[8]) {
    const RunAt tb{0, t.c, 0, t.cl};
    if (a.bias) {
        float b[8];
        if (a.bias_dt == 0) run_load<0>(a.bias, 0, tb, 0, b);
        else run_load<1>(a.bias, 0, tb, 1, b);
#pragma unroll
        for (int k = 0; k < 8; ++k) g[k] += b[k];
    }
    if (a.bias2) {
        float b[8];
        if (a.bias_dt == 0) run_load<0>(a.bias2, 0, tb, 0, b);
        else run_load<1>(a.bias2, 0, tb, 1, b);
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] += b[k];
    }
    z_store<DT>(a.z, a.ld_z, a.z8, t, g);
    z_store<DT>(a.z2, a.ld_z, a.z8_2, t, u);
    gate_all(g, u, a.gate_act);
    run_store<DT>(a.out, a.ld_out, t, DT, g);
}
// From dh: the gradients at both pre-activations, and h again.  Their stores stay
// in the caches for the products that read them next: streamed past them the call
// itself is faster (4001 x 2816, 68 MB written: 57 -> 50 us), a whole feed-forward
// block slower (4096 x 1024 x 2816, forward and backward: 392 -> 405).
template <int DT>
__device__ __forceinline__ void gated_dh_run(const GatedArgs& a, const RunAt& t, const ZRaw<DT>& w, float (&v)[8]) {
    float g[8], u[8];
    z_values<DT>(a.z != nullptr, w.g, w.g1, g);
    z_values<DT>(a.z != nullptr, w.u, w.u1, u);
    gate_grad_all(v, g, u, a.gate_act);      // v: dzg, g: dzu, u: h
    run_store<DT>(a.out, a.ld_out, t, DT, v);
    run_store<DT>(a.out2, a.ld_out, t, DT, g);
    if (a.act_out) run_store<DT>(a.act_out, a.ld_act, t, DT, u);
}
// The same for any run, nv of its 8 elements inside; the four lanes of a group
// of 32 columns are neighbours.
__device__ __forceinline__ void z_store_any(void* z, int64_t ld, int dt, bool vec, const Act8View& z8, int64_t r, int64_t c,
                                            int nv, const float (&v)[8]) {
    if (z && nv > 0) store8(z, r * ld + c, dt, vec, nv, v);
    if (!z8.codes) return;
    const uint32_t e = act8_exp(group_max<1>(v, nv));
    if (nv <= 0) return;
    const u32x2_t w = act8_pack(v, e, nv);
    GMEM int8_t* p = gm(z8.codes) + r * z8.ld + c;
    if (z8.vec && nv >= 8) {
        *reinterpret_cast<GMEM u32x2_t*>(p) = w;
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < nv) p[k] = int8_t(w[k >> 2] >> (8 * (k & 3)));
    }
    if ((c & (kAct8Group - 1)) == 0) gm(z8.exps)[r * z8.lde + c / kAct8Group] = uint8_t(e);
}
__device__ __forceinline__ void z_load_any(const void* z, int64_t ld, int dt, bool vec, const Act8View& z8, int64_t r,
                                           int64_t c, int nv, float (&v)[8]) {
    if (z) {
        load8(z, r * ld + c, dt, vec, nv, v);
        return;
    }
    const float step = act8_step(gm(z8.exps)[r * z8.lde + c / kAct8Group]);
    const GMEM int8_t* p = gm(z8.codes) + r * z8.ld + c;
    if (z8.vec && nv >= 8) {
        const u32x2_t w = *reinterpret_cast<const GMEM u32x2_t*>(p);
        act8_dec4(w[0], step, v);
        act8_dec4(w[1], step, v + 4);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = k < nv ? float(p[k]) * step : 0.f;
    }
}
__device__ __forceinline__ void gated_any(const GatedArgs& a, int64_t r, int64_t c, int nv, float (&g)[8], float (&u)[8]) {
    if (a.bias) {
        float b[8];
        load8(a.bias, c, a.bias_dt, a.bias_vec, nv, b);
#pragma unroll
        for (int k = 0; k < 8; ++k) g[k] += b[k];
    }
    if (a.bias2) {
        float b[8];
        load8(a.bias2, c, a.bias_dt, a.bias_vec, nv, b);
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] += b[k];
    }
    z_store_any(a.z, a.ld_z, a.dt, a.z_vec, a.z8, r, c, nv, g);
    z_store_any(a.z2, a.ld_z, a.dt, a.z_vec, a.z8_2, r, c, nv, u);
    if (nv <= 0) return;
    gate_all(g, u, a.gate_act);
    store8(a.out, r * a.ld_out + c, a.dt, a.out_vec, nv, g);
}
__device__ __forceinline__ void gated_dh_any(const GatedArgs& a, int64_t r, int64_t c, int nv, float (&v)[8]) {
    if (nv <= 0) return;
    float g[8], u[8];
    z_load_any(a.z, a.ld_z, a.dt, a.z_vec, a.z8, r, c, nv, g);
    z_load_any(a.z2, a.ld_z, a.dt, a.z_vec, a.z8_2, r, c, nv, u);
    gate_grad_all(v, g, u, a.gate_act);
    store8(a.out, r * a.ld_out + c, a.dt, a.out_vec, nv, v);
    store8(a.out2, r * a.ld_out + c, a.dt, a.out_vec, nv, g);
    if (a.act_out) store8(a.act_out, r * a.ld_act + c, a.dt, a.act_vec, nv, u);
}

// Any run: 8 elements from (r, c) on, nv of them inside (0: none), any
// alignment.  The four lanes of a group of 32 columns are neighbours.
__device__ __forceinline__ void epilogue_any(const LinArgs& a, int64_t r, int64_t c, int nv, float (&v)[8]) {
    if (a.kind == LIN_FWD) {
        if (a.bias) {
            float b[8];
            load8(a.bias, c, a.bias_dt, a.bias_vec, nv, b);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] += b[k];
        }
        if (a.z && nv > 0) store8(a.z, r * a.ld_z + c, a.dt, a.z_vec, nv, v);
        if (a.z8.codes) {
            const uint32_t e = act8_exp(group_max<1>(v, nv));
            if (nv > 0) {
                const u32x2_t w = act8_pack(v, e, nv);
                GMEM int8_t* p = gm(a.z8.codes) + r * a.z8.ld + c;
                if (a.z8.vec && nv >= 8) {
                    *reinterpret_cast<GMEM u32x2_t*>(p) = w;
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k < nv) p[k] = int8_t(w[k >> 2] >> (8 * (k & 3)));
                }
                if ((c & (kAct8Group - 1)) == 0) gm(a.z8.exps)[r * a.z8.lde + c / kAct8Group] = uint8_t(e);
            }
        }
        if (nv <= 0) return;
        act_all(v, a.act);
    } else if (a.kind == LIN_DX) {
        if (nv <= 0) return;
        if (a.z || a.z8.codes) {
            float z[8], h[8];
            if (a.z) {
                load8(a.z, r * a.ld_z + c, a.dt, a.z_vec, nv, z);
            } else {
                const float step = act8_step(gm(a.z8.exps)[r * a.z8.lde + c / kAct8Group]);
                const GMEM int8_t* p = gm(a.z8.codes) + r * a.z8.ld + c;
                if (a.z8.vec && nv >= 8) {
                    const u32x2_t w = *reinterpret_cast<const GMEM u32x2_t*>(p);
                    act8_dec4(w[0], step, z);
                    act8_dec4(w[1], step, z + 4);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) z[k] = k < nv ? float(p[k]) * step : 0.f;
                }
            }
            act_grad_all(v, z, h, a.act);
            if (a.act_out) store8(a.act_out, r * a.ld_act + c, a.dt, a.act_vec, nv, h);
        }
    } else {
        if (nv <= 0) return;
        if (a.accumulate) {
            float o[8];
            load8(a.out, r * a.ld_out + c, a.out_dt, a.out_vec, nv, o);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] += o[k];
        }
    }
    if (a.kind != LIN_DW && a.add) {
        float b[8];
        load8(a.add, r * a.ld_add + c, a.dt, a.add_vec, nv, b);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += b[k];
    }
    store8(a.out, r * a.ld_out + c, a.out_dt, a.out_vec, nv, v);
}

// Every buffer that the epilogue touches allows vectors, and lane offsets of
// up to 16 rows fit 32 bits.
__device__ __forceinline__ bool fast_epilogue(const LinArgs& a) {
    constexpr int64_t kMost = int64_t(1) << 25;   // 16 rows x 4 bytes x this < 2^32
    return a.out_vec && a.ld_out <= kMost && (!a.bias || a.bias_vec) && (!a.add || (a.add_vec && a.ld_add <= kMost)) &&
           (!a.z || (a.z_vec && a.ld_z <= kMost)) &&
           (!a.z8.codes || (a.z8.vec && a.z8.ld <= kMost && a.z8.lde <= kMost)) &&
           (!a.act_out || (a.act_vec && a.ld_act <= kMost));
}
__device__ __forceinline__ bool fast_epilogue(const GatedArgs& a) {
    constexpr int64_t kMost = int64_t(1) << 25;
    return fast_epilogue(static_cast<const LinArgs&>(a)) && (!a.bias2 || a.bias_vec) &&
           (!a.z8_2.codes || (a.z8_2.vec && a.z8_2.ld <= kMost && a.z8_2.lde <= kMost));
}

// Shape of the output as stored, and of the split sums (rows padded to whole groups).
struct OutShape {
    int64_t rows, cols, ldp;
};
__host__ __device__ inline OutShape out_shape(const LinArgs& a) {
    OutShape o;
    o.rows = a.out_trans ? a.N : a.M;
    o.cols = a.out_trans ? a.M : a.N;
    o.ldp = (o.cols + kAct8Group - 1) / kAct8Group * kAct8Group;
    return o;
}

// 8 elements of a split's sums, kept in the caches for the join (1024 x 4096 in
// four splits, 8192 tokens: 89 us; streamed past them 101).
__device__ __forceinline__ void put_partial(const LinArgs& a, const OutShape& o, int split, const RunAt& t,
                                            const float (&v)[8]) {
    if (t.r + t.rl >= o.rows || t.c + t.cl >= o.cols) return;   // a run that begins inside may end in the row's padding
    GMEM char* p = run_ptr(reinterpret_cast<char*>(a.partial) + int64_t(split) * o.rows * o.ldp * 4, o.ldp, t, 4);
    *reinterpret_cast<GMEM f32x4_t*>(p) = f32x4_t{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<GMEM f32x4_t*>(p + 16) = f32x4_t{v[4], v[5], v[6], v[7]};
}

// The output tile (ROWS x COLS at r0, c0, in the output's orientation) lies in
// LDS as float32 rows: through the general epilogue, 8 elements a lane.  One
// copy of its code, for tiles past the last column and buffers without vectors.
__device__ __forceinline__ int stage_at(int cols, int r, int c) {   // float index of 4 elements; chunks XOR row
    return r * cols + (((c >> 2) ^ (r & 15)) << 2);
}
__device__ __forceinline__ void run_any(const LinArgs& a, int64_t r, int64_t c, int nv, float (&v)[8]) {
    epilogue_any(a, r, c, nv, v);
}
__device__ __forceinline__ void run_any(const GatedArgs& a, int64_t r, int64_t c, int nv, float (&v)[8]) {
    if (a.kind == LIN_GATED_DH) gated_dh_any(a, r, c, nv, v);
    else epilogue_any(a, r, c, nv, v);
}
template <int THREADS, class Args>
__device__ __forceinline__ void staged_epilogue(const Args& a, const OutShape& o, const float* stage, int rows,
                                                int cols, int64_t r0, int64_t c0) {
#pragma unroll 1
    for (int i = threadIdx.x; i < rows * cols / 8; i += THREADS) {
        const int r = i / (cols / 8), c = i % (cols / 8) * 8;
        const f32x4_t x = *reinterpret_cast<const f32x4_t*>(stage + stage_at(cols, r, c));
        const f32x4_t y = *reinterpret_cast<const f32x4_t*>(stage + stage_at(cols, r, c + 4));
        float v[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
        int64_t n = o.cols - (c0 + c);
        n = r0 + r < o.rows ? (n > 8 ? 8 : n) : 0;
        run_any(a, r0 + r, c0 + c, n > 0 ? int(n) : 0, v);
    }
}
// Both projections' tiles in LDS, `cols` columns of the gate's and then as many
// of the up projection's.
template <int THREADS>
__device__ __forceinline__ void staged_gated(const GatedArgs& a, const OutShape& o, const float* stage, int rows, int cols,
                                             int64_t r0, int64_t c0) {
#pragma unroll 1
    for (int i = threadIdx.x; i < rows * cols / 8; i += THREADS) {
        const int r = i / (cols / 8), c = i % (cols / 8) * 8;
        float v[2][8];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const f32x4_t x = *reinterpret_cast<const f32x4_t*>(stage + stage_at(2 * cols, r, w * cols + c));
            const f32x4_t y = *reinterpret_cast<const f32x4_t*>(stage + stage_at(2 * cols, r, w * cols + c + 4));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[w][k] = x[k];
                v[w][4 + k] = y[k];
            }
        }
        int64_t n = o.cols - (c0 + c);
        n = r0 + r < o.rows ? (n > 8 ? 8 : n) : 0;
        gated_any(a, r0 + r, c0 + c, n > 0 ? int(n) : 0, v[0], v[1]);
    }
}
__device__ __forceinline__ void stage_put(float* stage, int cols, int r, int c, const float (&v)[8]) {
    *reinterpret_cast<f32x4_t*>(stage + stage_at(cols, r, c)) = f32x4_t{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<f32x4_t*>(stage + stage_at(cols, r, c + 4)) = f32x4_t{v[4], v[5], v[6], v[7]};
}

__device__ __forceinline__ void emit_db(const LinArgs& a, int split, int64_t n, float v) {
    if (n >= a.N) return;
    if (a.splits > 1) {
        gm(a.db_partial)[int64_t(split) * a.N + n] = v;
        return;
    }
    if (a.accumulate) v += load1(a.db, n, a.db_dt);
    store1(a.db, n, a.db_dt, v);
}

// Workgroup -> (split, tile).  Workgroup b runs on XCD b % 8 and each XCD has
// its own L2: an XCD takes one contiguous eighth of the tiles, in groups of 8
// tile rows across all tile columns, so that the tiles it runs at one time
// share few operand panels.
struct TileAt {
    int64_t tm, tn;
    int split;
    bool in;
};
template <int PAIR = PAIR_NONE>
__device__ __forceinline__ TileAt tile_at(const LinArgs& a, int edge) {   // at most 2^31 workgroups
    const int ce = PAIR == PAIR_COLS ? edge / 2 : edge;   // columns of a tile
    const uint32_t nm = uint32_t((a.M + edge - 1) / edge), n1 = uint32_t((a.N + ce - 1) / ce);
    const uint32_t nn = PAIR == PAIR_OUT ? 2 * n1 : n1, tiles = nm * nn;
    const uint32_t all = tiles * uint32_t(a.splits), chunk = (all + 7) / 8;
    const uint32_t t = (blockIdx.x & 7) * chunk + (blockIdx.x >> 3);
    TileAt o;
    o.in = t < all && (blockIdx.x >> 3) < chunk;
    const uint32_t split = t / tiles, u = t - split * tiles, g = u / (8 * nn), w = u - g * 8 * nn;
    const uint32_t rows = nm - 8 * g < 8 ? nm - 8 * g : 8, c = w / rows;
    o.split = int(split);
    o.tm = 8 * g + (w - c * rows);
    o.tn = c;
    return o;
}

template <int KIND, int PAIR>
using ArgsOf = std::conditional_t<(KIND >= LIN_GATED || PAIR != PAIR_NONE), GatedArgs, LinArgs>;

// PAIR_OUT: the tile columns past the first output's are the second's.
__device__ __forceinline__ void pick_output(GatedArgs& a, TileAt& t, int edge) {
    const int64_t n1 = (a.N + edge - 1) / edge;
    if (t.tn < n1) return;
    t.tn -= n1;
    a.b = a.b2;
    a.out = a.out2;
    a.db = a.db2;
    if (a.splits > 1) {
        const OutShape o = out_shape(a);
        a.partial += a.splits * o.rows * o.ldp;
        if (a.db_partial) a.db_partial += a.splits * a.N;
    }
}

// ---------------------------------------------------------------------------
// W x W tiles: 4 waves of W/2 x W/2 and a ring of NST LDS stages.  With W = 128
// and two stages (64 KB) two workgroups share a CU and one's epilogue and waits
// overlap the other's MFMAs.  Where there are no more workgroups than CUs, four
// stages (128 KB) let the fragments be read half a block ahead (below): 2048 x
// 2048 -> 1408 28 -> 23 us.  W = 64 serves outputs of few tiles, with four stages
// (64 KB), or eight where a CU has only one workgroup: a few rows' product is as
// fast as the weight arrives, and that takes 7 blocks in flight on each CU
// (1 token 4096 -> 14336: 25.3 us, 4.65 TB/s).
// TR: the accumulators hold runs along M (the output is stored transposed).
// ---------------------------------------------------------------------------
template <class T, bool AKC, bool BKC, int ASRC, int BSRC, int KIND, bool TR, int W, int NST, int PAIR = PAIR_NONE>
__global__ __launch_bounds__(256, 2) void linear_tile_kernel(ArgsOf<KIND, PAIR> a) {
    using N = Num<T>;
    constexpr int OPB = W * 128;         // LDS bytes of an operand's stage
    constexpr int TI = W / 32;           // 16-wide fragments of a wave's edge
    constexpr bool COLS = PAIR == PAIR_COLS;
    constexpr int WB = COLS ? W / 2 : W; // columns of a tile
    constexpr int PW = COLS ? OPB / 2 : 0;   // LDS bytes from the gate's columns to the up projection's
    static_assert(PAIR == PAIR_NONE || (ASRC == S_DMA && BSRC == S_DMA), "pairs come by whole chunks");
    __shared__ __align__(1024) char smem[NST * 2 * OPB];
    static_assert(NST == 2 || (ASRC == S_DMA && BSRC == S_DMA), "registers stage one block ahead");
    const uint32_t lds0 = lds_base(smem);
    TileAt t = tile_at<PAIR>(a, W);
    if (!t.in) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    if constexpr (PAIR == PAIR_OUT) pick_output(a, t, W);
    const int64_t nk1 = (a.K + N::BK - 1) / N::BK, nkb = PAIR == PAIR_K ? 2 * nk1 : nk1;
    const int64_t kbs = (nkb + a.splits - 1) / a.splits;
    const int64_t kb0 = t.split * kbs, kb1 = kb0 + kbs < nkb ? kb0 + kbs : nkb;
    const int64_t kend = PAIR != PAIR_K && kb1 * N::BK < a.K ? kb1 * N::BK : a.K;
    Loader<T, AKC, ASRC, W> la;
    Loader<T, BKC, BSRC, WB> lb;
    la.init(a.a, a.lda, a.M, t.tm * W, kend, wave, lane);
    lb.init(a.b, a.ldb, a.N, t.tn * WB, kend, wave, lane);
    const char *a2 = nullptr, *b2 = nullptr;   // the pair's second operands, from the same tile on
    if constexpr (PAIR == PAIR_K) a2 = static_cast<const char*>(a.a2) + (la.base - static_cast<const char*>(a.a));
    if constexpr (PAIR == PAIR_K || COLS) b2 = static_cast<const char*>(a.b2) + (lb.base - static_cast<const char*>(a.b));
    if constexpr (ASRC == S_ACT8) {
        la.exps = a.a_exps;
        la.lde = a.lda_exps;
        la.vec8 = a.a8_vec != 0;
    }
    const int wr = (wave >> 1) * (W / 2), wc = (wave & 1) * (W / 2);
    f32x4_t acc[TI][TI];
    f32x4_t dbs[TI];
#pragma unroll
    for (int i = 0; i < TI; ++i) {
        dbs[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < TI; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    // the column sums of B: a product with a row of ones, in the tiles of the first tile row
    const bool sum_b = !AKC && a.db != nullptr && t.tm == 0 && wr == 0;

    using F = decltype(frag<T, AKC, W>(smem, 0, 0, 0));
    auto read = [&](const char* st, int s, F(&fa)[TI], F(&fb)[TI]) {
#pragma unroll
        for (int i = 0; i < TI; ++i) fa[i] = frag<T, AKC, W>(st, wr + 16 * i, s, lane);
#pragma unroll
        for (int j = 0; j < TI; ++j) {
            if constexpr (COLS) {        // a wave's columns: a quarter of the tile's edge of each projection
                const int up = j >= TI / 2;
                fb[j] = frag<T, BKC, WB>(st + OPB + up * PW, wc / 2 + 16 * (j - up * (TI / 2)), s, lane);
            } else {
                fb[j] = frag<T, BKC, W>(st + OPB, wc + 16 * j, s, lane);
            }
        }
    };
    // beside(i): loads issued between the rows' MFMAs
    auto mul = [&](const F(&fa)[TI], const F(&fb)[TI], auto&& beside) {
#pragma unroll
        for (int i = 0; i < TI; ++i) {
#pragma unroll
            for (int j = 0; j < TI; ++j) acc[i][j] = TR ? mma(fa[i], fb[j], acc[i][j]) : mma(fb[j], fa[i], acc[i][j]);
            beside(i);
        }
        if (sum_b) {
            const F one = ones<F>();
#pragma unroll
            for (int j = 0; j < TI; ++j) dbs[j] = mma(fb[j], one, dbs[j]);
        }
    };
    const int nk = int(kb1 - kb0);
    auto k_of = [&](int kb) { return (kb0 + kb) * N::BK; };
    // part q (of TI) of block kb's loads into the stage at LDS address st; past
    // the end of k: zeros
    auto load = [&](int kb, uint32_t st, int q) {
        if constexpr (PAIR == PAIR_K) {
            const int64_t b = kb0 + kb;
            const bool second = b >= nk1;
            const int64_t k0 = b >= kb1 ? nk1 * N::BK : (second ? b - nk1 : b) * N::BK;
            la.issue(second ? a2 : la.base, k0, st, q);
            lb.issue(second ? b2 : lb.base, k0, st + OPB, q);
        } else if constexpr (COLS) {
            la.issue(k_of(kb), st, q);
            if (q < TI / 2) lb.issue(lb.base, k_of(kb), st + OPB, q);
            else lb.issue(b2, k_of(kb), st + OPB + PW, q - TI / 2);
        } else {
            la.issue(k_of(kb), st, q);
            lb.issue(k_of(kb), st + OPB, q);
        }
    };
    auto load_all = [&](int kb, uint32_t st) {
        if constexpr (PAIR == PAIR_NONE) {
            la.issue(k_of(kb), st);
            lb.issue(k_of(kb), st + OPB);
        } else {
#pragma unroll
            for (int q = 0; q < TI; ++q) load(kb, st, q);
        }
    };
    if constexpr (NST >= 4) {
        // Stage kb of the ring is kb mod NST.  At the top of block kb its stage and
        // the next one are whole in LDS, the NST - 3 after them are in flight.
        // Fragments are read half a block (one step s) ahead of their MFMAs,
        // across blocks too.
        static_assert((NST & (NST - 1)) == 0, "ring");
        constexpr int kFlight = (NST - 3) * (W / 16);   // a wave's loads of those blocks
        auto stage = [&](int kb) { return (kb & (NST - 1)) * 2 * OPB; };
        auto issue = [&](int kb) { load_all(kb, lds0 + stage(kb)); };   // past the end too: it keeps the count of loads
        if (nk > 0) {
#pragma unroll
            for (int p = 0; p < NST - 1; ++p) issue(p);
            vm_wait<kFlight>();
            __syncthreads();
            F fa0[TI], fb0[TI], fa1[TI], fb1[TI];
            read(smem + stage(0), 0, fa0, fb0);
            for (int kb = 0; kb < nk; ++kb) {
                // Pinned in this order: the compiler would move each read down to
                // its use.  The loads of block kb + NST - 1 go into the stage of
                // block kb - 1, which every wave has read: between the MFMAs, or
                // (eight stages: bound by memory) before them.
                constexpr bool kFirst = NST == 8;
                if (kFirst) issue(kb + NST - 1);
                read(smem + stage(kb), 1, fa1, fb1);
                __builtin_amdgcn_sched_barrier(0);
                mul(fa0, fb0, [&](int i) {
                    if (kFirst) return;
                    load(kb + NST - 1, lds0 + stage(kb + NST - 1), i);
                    __builtin_amdgcn_sched_barrier(0);
                });
                read(smem + stage(kb + 1), 0, fa0, fb0);
                __builtin_amdgcn_sched_barrier(0);
                mul(fa1, fb1, [](int) {});
                vm_wait<kFlight>();      // this wave's part of block kb + 2 has landed
                __syncthreads();         // and every other wave's
            }
            vm_wait<0>();                // no load may land after the epilogue reuses LDS or gives it away
        }
    } else {
        if (nk > 0) {
            load_all(0, lds0);
            la.fetch(k_of(0));
            lb.fetch(k_of(0));
            la.put(smem);
            lb.put(smem + OPB);
        }
        for (int kb = 0; kb < nk; ++kb) {
            const int at = (kb & 1) * 2 * OPB, into = 2 * OPB - at;
            vm_wait<0>();                // this wave's part of the stage has landed
            __syncthreads();             // and every other wave's; the other stage has been read
            const bool more = kb + 1 < nk;
            if (more) {
                load_all(kb + 1, lds0 + into);
                la.fetch(k_of(kb + 1));
                lb.fetch(k_of(kb + 1));
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                F fa[TI], fb[TI];
                read(smem + at, s, fa, fb);
                mul(fa, fb, [](int) {});
            }
            if (more) {
                la.put(smem + into);
                lb.put(smem + into + OPB);
            }
        }
    }

    const OutShape o = out_shape(a);
    const int g = lane >> 4, i16 = lane & 15;
    const int64_t r0 = (TR ? t.tn : t.tm) * W, c0 = (TR ? t.tm : t.tn) * WB;
    if constexpr (COLS) {
        // f(row, column, lane's row, lane's column, gate, up): with two fragments of
        // each projection a run's 32 columns lie in one row tile; with one of each,
        // two row tiles' 16 columns make a run of their own
        auto runs2 = [&](auto&& f) {
            if constexpr (TI == 4) {
#pragma unroll
                for (int i = 0; i < TI; ++i) {
                    float v[8], u[8];
                    join_tiles(acc[i][0], acc[i][1], v);
                    join_tiles(acc[i][2], acc[i][3], u);
                    f(wr + 16 * i, wc / 2, i16, 8 * g, v, u);
                }
            } else {
                float v[8], u[8];
                join_tiles(acc[0][0], acc[1][0], v);
                join_tiles(acc[0][1], acc[1][1], u);
                f(wr, wc / 2, 16 * (g >> 1) + i16, 8 * (g & 1), v, u);
            }
        };
        if (a.splits > 1) {
            runs2([&](int r, int c, int rl, int cl, float(&v)[8], float(&u)[8]) {
                put_partial(a, o, 2 * t.split, RunAt{r0 + r, c0 + c, rl, cl}, v);
                put_partial(a, o, 2 * t.split + 1, RunAt{r0 + r, c0 + c, rl, cl}, u);
            });
        } else if (c0 + WB <= o.cols && fast_epilogue(a) && (TI == 4 || !a.z8.codes)) {
            runs2([&](int r, int c, int rl, int cl, float(&v)[8], float(&u)[8]) {
                if (r0 + r + rl < o.rows) gated_run<N::dt>(a, RunAt{r0 + r, c0 + c, rl, cl}, v, u);
            });
        } else {
            float* stage = reinterpret_cast<float*>(smem);
            __syncthreads();             // every wave has read its last fragments
            runs2([&](int r, int c, int rl, int cl, float(&v)[8], float(&u)[8]) {
                stage_put(stage, W, r + rl, c + cl, v);
                stage_put(stage, W, r + rl, WB + c + cl, u);
            });
            __syncthreads();
            staged_gated<256>(a, o, stage, W, WB, r0, c0);
        }
        return;
    }
    // f(row, column, values): runs of 8 of this wave's part of the output tile; a
    // lane's own is i16 rows and 8 g columns on
    auto runs = [&](auto&& f) {
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
            for (int p = 0; p < TI / 2; ++p) {
                float v[8];
                if constexpr (TR) {
                    join_tiles(acc[2 * p][i], acc[2 * p + 1][i], v);
                    f(wc + 16 * i, wr + 32 * p, v);
                } else {
                    join_tiles(acc[i][2 * p], acc[i][2 * p + 1], v);
                    f(wr + 16 * i, wc + 32 * p, v);
                }
            }
    };
    if constexpr (KIND == LIN_GATED_DH) {
        if (a.splits == 1 && c0 + W <= o.cols && fast_epilogue(a)) {
            // the next fragment row's pre-activations are in flight under this one's arithmetic
            ZRaw<N::dt> z[2][TI / 2];
            auto at = [&](int i, int p) { return RunAt{r0 + wr + 16 * i, c0 + wc + 32 * p, i16, 8 * g}; };
            auto fetch = [&](int i) {
#pragma unroll
                for (int p = 0; p < TI / 2; ++p)
                    if (r0 + wr + 16 * i + i16 < o.rows) z_fetch<N::dt>(a, at(i, p), z[i & 1][p]);
            };
            fetch(0);
#pragma unroll
            for (int i = 0; i < TI; ++i) {
                if (i + 1 < TI) fetch(i + 1);
#pragma unroll
                for (int p = 0; p < TI / 2; ++p) {
                    float v[8];
                    join_tiles(acc[i][2 * p], acc[i][2 * p + 1], v);
                    if (r0 + wr + 16 * i + i16 < o.rows) gated_dh_run<N::dt>(a, at(i, p), z[i & 1][p], v);
                }
            }
            return;
        }
    }
    if (a.splits > 1) {
        runs([&](int r, int c, float(&v)[8]) { put_partial(a, o, t.split, RunAt{r0 + r, c0 + c, i16, 8 * g}, v); });
    } else if (KIND >= 0 && c0 + W <= o.cols && fast_epilogue(a)) {
        runs([&](int r, int c, float(&v)[8]) {
            if (r0 + r + i16 < o.rows) epilogue_run<KIND, N::dt>(a, RunAt{r0 + r, c0 + c, i16, 8 * g}, v);
        });
    } else {
        float* stage = reinterpret_cast<float*>(smem);
        __syncthreads();                 // every wave has read its last fragments
        runs([&](int r, int c, float(&v)[8]) { stage_put(stage, W, r + i16, c + 8 * g, v); });
        __syncthreads();
        staged_epilogue<256>(a, o, stage, W, W, r0, c0);
    }
    if (sum_b && i16 == 0) {   // every column of the product with ones is the same
#pragma unroll
        for (int j = 0; j < TI; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) emit_db(a, t.split, t.tn * W + wc + 16 * j + 4 * g + e, dbs[j][e]);
    }
}

// ---------------------------------------------------------------------------
// 256 x 256 tiles of bf16, one workgroup of 8 waves per CU.
//
// The tile is cut into halves of 128 rows (A0, A1) and columns (B0, B1); a wave
// owns a 64 x 32 block of each of the four quadrants, so a k block of 64 is four
// phases of 16 MFMAs:  A0 B0, A0 B1, A1 B1, A1 B0.  A phase has a load section
// (fragments of the operand half that the phase needs new, and the global loads
// of one half of the k block after next) and an MFMA section, each ended by a
// barrier.  The two waves that share a SIMD run half a phase apart (waves 4-7
// pass one barrier more at the start): one issues MFMAs while the other reads
// LDS, so the matrix cores see no LDS latency and no wait at a barrier.
//
// LDS holds two k blocks (128 KB), each as four halves of 16 KB that are
// refilled one by one as soon as they have been read: B0 is read in phase 3 of
// the block before, A0 in phase 0, B1 in 1, A1 in 2, and the loads of the block
// after next go out in phases 0 (B0), 1 (A0), 2 (B1) and 3 (A1), one phase
// after the half's last read by either group of waves.  A half is needed 7
// phases after its loads were issued; at the end of a load section everything
// but the 6 halves issued last (2 loads a wave each) has landed.  Loads past the
// end of k are issued too and read as zeros, which keeps that count.
//
// Long k is MFMA bound (pipes busy about 70 % of the time, no LDS bank conflict):
// 4096 tokens 14336 -> 4096 with a residual 335 us, 1.44 PFLOP/s.  Short k is
// carried by prologue and epilogue: 8192 tokens 1024 -> 4096 with bias and GELU
// 75-80 us, 0.86-0.91 PFLOP/s, pipes busy 41 % (one workgroup a CU: nothing
// overlaps its epilogue).
// ---------------------------------------------------------------------------
constexpr int kPpThreads = 512;

// PAIR: the halves are the same rows or columns of two operands laid out alike
// (base2: the second's).
template <bool KC, bool PAIR = false>
struct HalfLoader {
    const char* base;
    const char* base2;
    int64_t ld, kend;
    uint32_t voff[PAIR ? 1 : 2][2];       // [half][1 KB block]
    int wave, lane;

    static constexpr int CPR = KC ? 8 : 16;
    __device__ __forceinline__ int lrow(int q) const { return (wave * 2 + q) * (64 / CPR) + lane / CPR; }
    __device__ __forceinline__ int lchunk(int q) const {
        const int r = lrow(q), c = lane % CPR;
        return KC ? c ^ (r & 7) : c ^ ks_swizzle<uint16_t, 128>(r);
    }
    __device__ __forceinline__ void init(const void* p, int64_t ld_, int64_t ext, int64_t e0, int64_t kend_, int wave_,
                                         int lane_) {
        ld = ld_;
        kend = kend_;
        wave = wave_;
        lane = lane_;
        base = static_cast<const char*>(p) + (KC ? e0 * ld : e0) * 2;
#pragma unroll
        for (int hf = 0; hf < (PAIR ? 1 : 2); ++hf)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int r = lrow(q), c = lchunk(q);
                if (KC) voff[hf][q] = e0 + hf * 128 + r < ext ? uint32_t((hf * 128 + r) * ld * 2 + c * 16) : kFar;
                else voff[hf][q] = e0 + hf * 128 + c * 8 < ext ? uint32_t(r * ld * 2 + hf * 256 + c * 16) : kFar;
            }
    }
    __device__ __forceinline__ void issue(int hf, int64_t k0, uint32_t lds) const {
        issue(PAIR && hf ? base2 : base, PAIR ? 0 : hf, k0, lds);
    }
    __device__ __forceinline__ void issue(const char* from, int hf, int64_t k0, uint32_t lds) const {
        if (KC) {
            const i32x4_t buf = buffer_at(from + k0 * 2, kMaxRecords);
#pragma unroll
            for (int q = 0; q < 2; ++q)
                buffer_to_lds(buf, k0 + lchunk(q) * 8 < kend ? voff[hf][q] : kFar, lds + (wave * 2 + q) * 1024);
        } else {
            int64_t n = (kend - k0) * ld * 2;
            n = n < 0 ? 0 : (n > int64_t(kMaxRecords) ? int64_t(kMaxRecords) : n);
            const i32x4_t buf = buffer_at(from + k0 * ld * 2, uint32_t(n));
#pragma unroll
            for (int q = 0; q < 2; ++q) buffer_to_lds(buf, voff[hf][q], lds + (wave * 2 + q) * 1024);
        }
    }
};

// Fragments of a half with few registers for addresses: one base per operand
// (the lane's part of the address of the wave's first row or column), from
// which every read differs by constants, some of them XORed (the swizzles only
// flip address bits: rows and columns step by 16 within a wave's aligned part).
// The base is made opaque at every use, so that the addresses are formed where
// they are used (one xor a read, beside the other waves' MFMAs) instead of all
// being kept in registers across the loop.
template <bool KC>
__device__ __forceinline__ uint32_t frag_base(int w0, int lane) {
    const int g = lane >> 4, i = lane & 15;
    if constexpr (KC) return uint32_t((w0 + i) * 128 + ((g ^ (i & 7)) << 4));
    const int k = 8 * g + (i >> 2), n = w0 + 4 * (i & 3);
    return uint32_t(k * 256 + (((n >> 3) ^ ks_swizzle<uint16_t, 128>(k)) << 4) + (n & 7) * 2);
}
template <bool KC>
__device__ __forceinline__ bf16x8_t frag_at(const char* smem, uint32_t base, int rc, int s, int region) {
    if constexpr (KC) {
        const u32x4_t w = *reinterpret_cast<const u32x4_t*>(smem + region + ((s ? base ^ 64u : base) + rc * 128));
        return __builtin_bit_cast(bf16x8_t, w);
    } else {
        i16x4_t h[2];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const char* p = smem + region + ((base ^ uint32_t((rc / 8 * 16) ^ (hh * 128))) + hh * 1024 + s * 8192);
            h[hh] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS i16x4_t*)(p));
        }
        return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
    }
}
__device__ __forceinline__ uint32_t opaque(uint32_t v) {
    asm volatile("" : "+v"(v));
    return v;
}

__device__ __forceinline__ void mem_fence() { asm volatile("" ::: "memory"); }
__device__ __forceinline__ void pp_barrier() {
    mem_fence();
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    mem_fence();
}
// End of a load section: its LDS reads are done, all but the last 12 loads have landed.
template <int VM>
__device__ __forceinline__ void pp_wait() {
    mem_fence();
    __builtin_amdgcn_s_waitcnt((VM & 15) | ((VM >> 4) << 14) | (7 << 4) | (0 << 8));
    pp_barrier();
}

template <bool AKC, bool BKC, int KIND, bool TR, int PAIR = PAIR_NONE>
__global__ __launch_bounds__(kPpThreads, 2) void linear_pp_kernel(ArgsOf<KIND, PAIR> a) {
    __shared__ __align__(1024) char smem[8 * kOpBytes];
    const uint32_t lds0 = lds_base(smem);
    constexpr bool COLS = PAIR == PAIR_COLS;
    constexpr int WB = COLS ? 128 : 256;     // columns of a tile: with pairs, B0 is the gate's and B1 the up projection's
    TileAt t = tile_at<PAIR>(a, 256);
    if (!t.in) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    if constexpr (PAIR == PAIR_OUT) pick_output(a, t, 256);
    const int64_t nk1 = (a.K + 63) / 64, nkb = PAIR == PAIR_K ? 2 * nk1 : nk1, kbs = (nkb + a.splits - 1) / a.splits;
    const int64_t kb0 = t.split * kbs, kb1 = kb0 + kbs < nkb ? kb0 + kbs : nkb;
    const int64_t kend = PAIR != PAIR_K && kb1 * 64 < a.K ? kb1 * 64 : a.K;
    const int nk = int(kb1 - kb0);
    const int64_t k00 = kb0 * 64;
    HalfLoader<AKC> la;
    HalfLoader<BKC, COLS> lb;
    la.init(a.a, a.lda, a.M, t.tm * 256, kend, wave, lane);
    lb.init(a.b, a.ldb, a.N, t.tn * WB, kend, wave, lane);
    if constexpr (PAIR == PAIR_K) la.base2 = static_cast<const char*>(a.a2) + (la.base - static_cast<const char*>(a.a));
    if constexpr (PAIR == PAIR_K || COLS)
        lb.base2 = static_cast<const char*>(a.b2) + (lb.base - static_cast<const char*>(a.b));
    // half hf of block kb of this split (past its end: zeros)
    auto issue_a = [&](int hf, int kb, uint32_t at) {
        if constexpr (PAIR == PAIR_K) {
            const int64_t b = kb0 + kb;
            const bool second = b >= nk1;
            la.issue(second ? la.base2 : la.base, hf, b >= kb1 ? nk1 * 64 : (second ? b - nk1 : b) * 64, at);
        } else {
            la.issue(hf, k00 + int64_t(kb) * 64, at);
        }
    };
    auto issue_b = [&](int hf, int kb, uint32_t at) {
        if constexpr (PAIR == PAIR_K) {
            const int64_t b = kb0 + kb;
            const bool second = b >= nk1;
            lb.issue(second ? lb.base2 : lb.base, hf, b >= kb1 ? nk1 * 64 : (second ? b - nk1 : b) * 64, at);
        } else {
            lb.issue(hf, k00 + int64_t(kb) * 64, at);
        }
    };
    const int wr = (wave >> 2) * 64, wc = (wave & 3) * 32;
    const bool sum_b = KIND == LIN_DW && a.db != nullptr && t.tm == 0 && wr == 0;

    f32x4_t acc[2][2][4][2], dbs[2][2];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            dbs[x][y] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[x][y][i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
    bf16x8_t fa[2][4], fb[2][2][2];      // [s][i]; [set][s][j]

    auto half_a = [&](int par, int hf) { return (par * 4 + hf) * kOpBytes; };
    auto half_b = [&](int par, int hf) { return (par * 4 + 2 + hf) * kOpBytes; };
    const uint32_t base_a = frag_base<AKC>(wr, lane), base_b = frag_base<BKC>(wc, lane);
    auto read_a = [&](int par, int hf) {
        const uint32_t b = opaque(base_a);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) fa[s][i] = frag_at<AKC>(smem, b, 16 * i, s, half_a(par, hf));
    };
    auto read_b = [&](int par, int hf, auto set) {
        constexpr int S = decltype(set)::value;
        const uint32_t b = opaque(base_b);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int j = 0; j < 2; ++j) fb[S][s][j] = frag_at<BKC>(smem, b, 16 * j, s, half_b(par, hf));
    };
    auto mul = [&](auto hh, auto gg, auto set, auto sum) {
        constexpr int H = decltype(hh)::value, G = decltype(gg)::value, S = decltype(set)::value;
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[H][G][i][j] = TR ? mma(fa[s][i], fb[S][s][j], acc[H][G][i][j])
                                         : mma(fb[S][s][j], fa[s][i], acc[H][G][i][j]);
        if constexpr (KIND == LIN_DW && decltype(sum)::value) {
            if (sum_b) {
                const bf16x8_t one = ones<bf16x8_t>();
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int j = 0; j < 2; ++j) dbs[G][j] = mma(fb[S][s][j], one, dbs[G][j]);
            }
        }
        __builtin_amdgcn_s_setprio(0);
        pp_barrier();
    };
    constexpr std::integral_constant<int, 0> c0_{};
    constexpr std::integral_constant<int, 1> c1_{};
    // one k block: PAR its LDS buffer, and the register set that holds its B0
    auto block = [&](auto par, int kb) {
        constexpr int P = decltype(par)::value;
        constexpr std::integral_constant<int, P> s0{};
        constexpr std::integral_constant<int, 1 - P> s1{};
        read_a(P, 0);
        issue_b(0, kb + 2, lds0 + half_b(P, 0));
        pp_wait<12>();
        mul(c0_, c0_, s0, std::true_type{});
        read_b(P, 1, s1);
        issue_a(0, kb + 2, lds0 + half_a(P, 0));
        pp_wait<12>();
        mul(c0_, c1_, s1, std::true_type{});
        read_a(P, 1);
        issue_b(1, kb + 2, lds0 + half_b(P, 1));
        pp_wait<12>();
        mul(c1_, c1_, s1, std::false_type{});
        read_b(1 - P, 0, s1);            // the next block's B0
        issue_a(1, kb + 2, lds0 + half_a(P, 1));
        pp_wait<12>();
        mul(c1_, c0_, s0, std::false_type{});
    };

    if (nk > 0) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            issue_b(0, p, lds0 + half_b(p, 0));
            issue_a(0, p, lds0 + half_a(p, 0));
            issue_b(1, p, lds0 + half_b(p, 1));
            issue_a(1, p, lds0 + half_a(p, 1));
        }
        pp_wait<14>();                   // B0 of the first block
        read_b(0, 0, c0_);
        pp_wait<12>();                   // and A0
        if (wave >= 4) pp_barrier();     // half a phase behind from here on
        for (int kb = 0; kb < nk; kb += 2) {
            block(c0_, kb);
            if (kb + 1 < nk) block(c1_, kb + 1);
        }
        if (wave < 4) pp_barrier();
        vm_wait<0>();                    // no load may land after the workgroup's LDS is given away
    }

    const OutShape o = out_shape(a);
    const int g = lane >> 4, i16 = lane & 15;
    const int64_t r0 = (TR ? t.tn : t.tm) * 256, c0 = (TR ? t.tm : t.tn) * WB;
    if constexpr (COLS) {
        const bool fast2 = c0 + WB <= o.cols && fast_epilogue(a);
        auto half2 = [&](auto hh) {
            constexpr int H = decltype(hh)::value;
            const int64_t rh = r0 + 128 * H;
            auto runs2 = [&](auto&& f) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v[8], u[8];
                    join_tiles(acc[H][0][i][0], acc[H][0][i][1], v);
                    join_tiles(acc[H][1][i][0], acc[H][1][i][1], u);
                    f(wr + 16 * i, wc, v, u);
                }
            };
            if (a.splits > 1) {
                runs2([&](int r, int c, float(&v)[8], float(&u)[8]) {
                    put_partial(a, o, 2 * t.split, RunAt{rh + r, c0 + c, i16, 8 * g}, v);
                    put_partial(a, o, 2 * t.split + 1, RunAt{rh + r, c0 + c, i16, 8 * g}, u);
                });
            } else if (fast2) {
                runs2([&](int r, int c, float(&v)[8], float(&u)[8]) {
                    if (rh + r + i16 < o.rows) gated_run<0>(a, RunAt{rh + r, c0 + c, i16, 8 * g}, v, u);
                });
            } else {
                float* stage = reinterpret_cast<float*>(smem);
                __syncthreads();
                runs2([&](int r, int c, float(&v)[8], float(&u)[8]) {
                    stage_put(stage, 256, r + i16, c + 8 * g, v);
                    stage_put(stage, 256, r + i16, 128 + c + 8 * g, u);
                });
                __syncthreads();
                staged_gated<kPpThreads>(a, o, stage, 128, 128, rh, c0);
            }
        };
        half2(c0_);
        half2(c1_);
        return;
    }
    // f(row, column, values): runs of 8 of this wave's part of half h (128 rows) of the output tile
    auto runs = [&](auto hh, auto&& f) {
        constexpr int H = decltype(hh)::value;
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float v[8];
                if constexpr (TR) {      // i: column tile i & 1, row pair i >> 1
                    join_tiles(acc[y][H][2 * (i >> 1)][i & 1], acc[y][H][2 * (i >> 1) + 1][i & 1], v);
                    f(wc + 16 * (i & 1), y * 128 + wr + 32 * (i >> 1), v);
                } else {
                    join_tiles(acc[H][y][i][0], acc[H][y][i][1], v);
                    f(wr + 16 * i, y * 128 + wc, v);
                }
            }
    };
    const bool fast = c0 + 256 <= o.cols && fast_epilogue(a);
    if constexpr (KIND == LIN_GATED_DH) {
        if (a.splits == 1 && fast) {
            // four runs' pre-activations are in flight under the four before: loaded
            // where they are used, each run would wait out its own loads (nothing
            // else runs on the CU)
            ZRaw<0> z[2][4];
            auto at = [&](int b, int i) {
                return RunAt{r0 + (b >> 1) * 128 + wr + 16 * i, c0 + (b & 1) * 128 + wc, i16, 8 * g};
            };
            auto in = [&](int b, int i) { return r0 + (b >> 1) * 128 + wr + 16 * i + i16 < o.rows; };
            auto fetch = [&](int b) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (in(b, i)) z_fetch<0>(a, at(b, i), z[b & 1][i]);
            };
            fetch(0);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                if (b < 3) fetch(b + 1);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v[8];
                    join_tiles(acc[b >> 1][b & 1][i][0], acc[b >> 1][b & 1][i][1], v);
                    if (in(b, i)) gated_dh_run<0>(a, at(b, i), z[b & 1][i], v);
                }
            }
            return;
        }
    }
    auto half = [&](auto hh) {
        const int64_t rh = r0 + 128 * decltype(hh)::value;
        if (a.splits > 1) {
            runs(hh, [&](int r, int c, float(&v)[8]) { put_partial(a, o, t.split, RunAt{rh + r, c0 + c, i16, 8 * g}, v); });
        } else if (fast) {
            runs(hh, [&](int r, int c, float(&v)[8]) {
                if (rh + r + i16 < o.rows) epilogue_run<KIND, 0>(a, RunAt{rh + r, c0 + c, i16, 8 * g}, v);
            });
        } else {
            float* stage = reinterpret_cast<float*>(smem);
            __syncthreads();
            runs(hh, [&](int r, int c, float(&v)[8]) { stage_put(stage, 256, r + i16, c + 8 * g, v); });
            __syncthreads();
            staged_epilogue<kPpThreads>(a, o, stage, 128, 256, rh, c0);
        }
    };
    half(c0_);
    half(c1_);
    if (sum_b && i16 == 0) {
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    emit_db(a, t.split, t.tn * 256 + y * 128 + wc + 16 * j + 4 * g + e, dbs[y][j][e]);
    }
}

}  // namespace
}  // namespace muon
